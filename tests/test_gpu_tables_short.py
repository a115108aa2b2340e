"""Block tables when something runs out or is wrong: a slot map too small for the new tokens,
ids outside the pool on the stack of free pages.
Whatever a row does not get, its length must not count: the decode reads every position
that a length counts."""

import pytest
import torch

import decode_attention_flash_gb300 as da
from test_gpu_tables import case, engine, i32

pytestmark = pytest.mark.gpu


def plain(old, new, page, table, free, cap, slot_capacity, pages=1 << 30):
    """The definition, one token at a time: a row takes the tokens that its capacity and the slot
    map hold, and the pages for those; a row that misses a page, or would get one that is none,
    takes nothing, nor does a later row that needs a page."""
    table = [list(r) for r in table]
    free = list(free)
    out, slots, cu, closed = [], [], [0], False
    for b, (o, n) in enumerate(zip(old, new)):
        fits = min(n, cap - o, max(0, slot_capacity - len(slots)))
        need = -(-(o + fits) // page) - -(-o // page)
        ok = need == 0 or (not closed and need <= len(free) and all(0 <= x < pages for x in free[-need:]))
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


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,new_hi,spare", [(1, 50, 3), (1, 40000, 700), (7, 300, 5), (61, 90, 5), (61, 900, -20), (700, 40, 5)])
@pytest.mark.parametrize("where", [0.0, 0.2, 0.7, 1.0])
@pytest.mark.parametrize("bad", [-1, 1 << 30, "pool"])
def test_an_id_outside_the_pool_ends_the_stack(batch, new_hi, spare, where, bad, in_place):
    old, new, table, free, cols, pages = case(batch, batch, 16, 40, new_hi, spare)
    new[0] = new[0] or 1
    need = sum(-(-(o + n) // 16) - -(-o // 16) for o, n in zip(old, new))
    depth = min(int(where * need), len(free) - 1)  # (at 1.0 nobody asks for it, or it is the last there is)
    free[len(free) - 1 - depth] = pages if bad == "pool" else bad
    eng = engine(batch, 16, cols, pages)
    want = plain(old, new, 16, table, free, cols * 16, sum(new), pages)
    t, err = call(eng, old, new, table, free, sum(new), in_place)
    ask = depth < min(need, len(free))
    assert err == (da.DA_DEVERR_PAGE_INDEX if ask else 0) | (da.DA_DEVERR_NO_PAGES if need > len(free) else 0)
    same(t, want)
    if not ask and need <= len(free):
        assert want[2] == [o + n for o, n in zip(old, new)]


def test_a_decode_behind_a_bad_id_reads_no_other_row():
    """Row 1's new page is no page: its table entry, of an earlier request, must not be read."""
    eng = da.DecodeAttention(device=0, batch=2, num_q_heads=1, num_kv_heads=1, head_dim_qk=128, head_dim_v=128,
                             kv_layout=da.DA_KV_PAGED, page_size=16, num_pages=8, max_pages_per_seq=2, max_seq_len=32,
                             q_dtype=da.DA_DTYPE_BF16, kv_dtype=da.DA_DTYPE_BF16)
    lens, table = i32([0, 0]), i32([[3, 3], [3, 3]])
    t = dict(seq_lens=lens, seq_lens_out=lens, new_lens=i32([1, 1]), free_pages=i32([5, 8, 4]), num_free=i32([3]),
             num_free_out=i32([0]), block_table=table, slot_map=torch.zeros(2, dtype=torch.int64, device="cuda"))
    eng.build_tables(t)
    assert eng.errors() == da.DA_DEVERR_PAGE_INDEX
    assert lens.tolist() == [1, 0] and table[:, 0].tolist() == [4, 3] and t["num_free_out"].item() == 2
    assert t["slot_map"].tolist() == [64, -1]
    kv = torch.full((8, 1, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = eng.run(dict(q=torch.ones(2, 1, 128, dtype=torch.bfloat16, device="cuda"), k=kv, v=kv, seq_lens=lens,
                       block_table=table), 1.0)
    assert eng.errors() == 0 and (out[0] == 7).all() and (out[1] == 0).all()


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
