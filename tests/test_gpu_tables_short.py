"""Block tables when something runs out or is wrong: a slot map too small for the new tokens.
Whatever a row does not get, its length must not count: the decode reads every position
that a length counts."""

import pytest
import torch

import decode_attention_flash_gb300 as da
from test_gpu_tables import case, engine, i32

pytestmark = pytest.mark.gpu


def plain(old, new, page, table, free, cap, slot_capacity):
    """The definition, one token at a time: a row takes the tokens that its capacity and the slot
    map hold, and the pages for those; a row that misses a page takes none, nor does a later row
    that needs one."""
    table = [list(r) for r in table]
    free = list(free)
    out, slots, cu, closed = [], [], [0], False
    for b, (o, n) in enumerate(zip(old, new)):
        fits = min(n, cap - o, max(0, slot_capacity - len(slots)))
        need = -(-(o + fits) // page) - -(-o // page)
        ok = need == 0 or (not closed and need <= len(free))
        closed = closed or not ok
        if ok:
            for k in range(need):
                table[b][-(-o // page) + k] = free.pop()
        for i in range(n):
            p = o + i
            slots.append(table[b][p // page] * page + p % page if ok and i < fits else -1)
        out.append(o + fits if ok else o)
        cu.append(len(slots))
    return table, free, out, slots[:slot_capacity], cu


def call(eng, old, new, table, free, slots, in_place):
    t = dict(seq_lens=i32(old), new_lens=i32(new), free_pages=i32(free + [-5]), num_free=i32([len(free)]),
             block_table=i32(table), slot_map=torch.full((slots,), 77, device="cuda"), cu_new=i32([77] * (len(old) + 1)))
    t["seq_lens_out"] = t["seq_lens"] if in_place else i32([77] * len(old))
    t["num_free_out"] = t["num_free"] if in_place else i32([77])
    eng.build_tables(t)
    torch.cuda.synchronize()
    return t, eng.errors()


def same(t, want):
    assert t["seq_lens_out"].tolist() == want[2]
    assert t["block_table"].tolist() == want[0]
    assert t["num_free_out"].item() == len(want[1])
    assert t["slot_map"].tolist() == want[3]
    assert t["cu_new"].tolist() == want[4]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,new_hi,spare", [(1, 50, 3), (7, 300, 5), (61, 90, 5), (61, 90, -20), (700, 20, 5), (1500, 2, 9)])
@pytest.mark.parametrize("part", [0.0, 0.3, 0.99])
def test_lengths_leave_out_what_the_slot_map_does_not_hold(batch, new_hi, spare, part, in_place):
    old, new, table, free, cols, pages = case(batch, batch, 16, 40, new_hi, spare)
    new[-1] = max(new[-1], 1)
    slots = max(1, int(sum(new) * part))
    eng = engine(batch, 16, cols, pages + 3)
    want = plain(old, new, 16, table, free, cols * 16, slots)
    t, err = call(eng, old, new, table, free, slots, in_place)
    assert err & da.DA_DEVERR_SLOT or sum(new) <= slots
    same(t, want)
    # the tokens left over, in calls of their own: as if all had come at once
    if spare > 0:
        got, have, tab, left = want[2], want[1], want[0], [o + n for o, n in zip(old, new)]
        while got != left:
            rest = [a - b for a, b in zip(left, got)]
            t, err = call(eng, got, rest, tab, have, max(slots, 200), in_place)
            assert err in (0, da.DA_DEVERR_SLOT)
            want = plain(got, rest, 16, tab, have, cols * 16, max(slots, 200))
            want = (*want[:3], want[3] + [-1] * (max(slots, 200) - len(want[3])), want[4])
            same(t, want)
            assert want[2] != got
            got, have, tab = want[2], want[1], want[0]
        assert len(have) == len(free) - sum(-(-(o + n) // 16) - -(-o // 16) for o, n in zip(old, new))


def test_no_slots_at_all_leave_the_state_as_it_was():
    eng = engine(3, 16, 4, 10)
    t = dict(seq_lens=i32([5, 0, 64]), new_lens=i32([1, 20, 0]), free_pages=i32([1, 2, 3]), num_free=i32([3]),
             num_free_out=i32([9]), seq_lens_out=i32([9] * 3), block_table=i32([[6, 7, 8, 9]] * 3),
             slot_map=torch.zeros(0, dtype=torch.int64, device="cuda"))
    eng.build_tables(t)
    assert eng.errors() == da.DA_DEVERR_SLOT
    assert t["seq_lens_out"].tolist() == [5, 0, 64] and t["num_free_out"].item() == 3
    assert t["block_table"].tolist() == [[6, 7, 8, 9]] * 3


def test_a_contiguous_cache_counts_what_it_holds():
    eng = engine(3, 0, 0, 0, contiguous=100)
    t = dict(seq_lens=i32([0, 98, 50]), new_lens=i32([2, 2, 4]), seq_lens_out=i32([0] * 3),
             slot_map=torch.zeros(3, dtype=torch.int64, device="cuda"))
    eng.build_tables(t)
    assert eng.errors() == da.DA_DEVERR_SLOT
    assert t["slot_map"].tolist() == [0, 1, 198] and t["seq_lens_out"].tolist() == [2, 99, 50]


def test_the_definition_by_hand():
    # 3 tokens of row 0 fit its page, row 1 takes a page and 2 of its 5 tokens, row 2 nothing
    table, free, out, slots, cu = plain([13, 16, 4], [3, 5, 9], 16, [[4, 0], [5, 0], [6, 0]], [1, 2], 32, 5)
    assert (table, free, out) == ([[4, 0], [5, 2], [6, 0]], [1], [16, 18, 4])
    assert slots == [77, 78, 79, 32, 33] and cu == [0, 3, 8, 17]
