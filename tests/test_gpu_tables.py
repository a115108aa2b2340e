"""Block tables and slots from request lengths, on the GPU, against a plain loop."""

import ctypes
import random

import pytest
import torch

import decode_attention_flash_gb300 as da

pytestmark = pytest.mark.gpu


def engine(batch, page, cols, pages, contiguous=0):
    kw = dict(batch=batch, num_q_heads=1, num_kv_heads=1, head_dim_qk=128, head_dim_v=128,
              q_dtype=da.DA_DTYPE_BF16, kv_dtype=da.DA_DTYPE_BF16)
    if contiguous:
        kw |= dict(kv_layout=da.DA_KV_CONTIGUOUS, max_seq_len=contiguous)
    else:
        kw |= dict(kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=pages, max_pages_per_seq=cols,
                   max_seq_len=cols * page)
    return da.DecodeAttention(device=0, **kw)


def plain(old, new, page, table, free, cap):
    """The definition, one token at a time."""
    table = [list(r) for r in table]
    free = list(free)
    out, slots, pos, row, cu = [], [], [], [], [0]
    full = False
    for b, (o, n) in enumerate(zip(old, new)):
        fits = min(n, cap - o)
        need = -(-(o + fits) // page) - -(-o // page)
        ok = need == 0 or (not full and need <= len(free))
        full = full or not ok
        if ok:
            for k in range(need):
                table[b][-(-o // page) + k] = free.pop()
        for i in range(n):
            p = o + i
            slots.append(table[b][p // page] * page + p % page if ok and i < fits else -1)
            pos.append(p)
            row.append(b)
        out.append(o + fits if ok else o)
        cu.append(len(slots))
    return table, free, out, slots, pos, row, cu


def case(seed, batch, page, old_hi, new_hi, spare, cols_extra=2):
    r = random.Random(seed)
    old = [r.randint(0, old_hi) for _ in range(batch)]
    new = [r.randint(0, new_hi) for _ in range(batch)]
    cols = max(-(-(o + n) // page) for o, n in zip(old, new)) + cols_extra
    have = sum(-(-o // page) for o in old)
    need = sum(-(-(o + n) // page) - -(-o // page) for o, n in zip(old, new))
    ids = list(range(have + max(0, need + spare)))
    r.shuffle(ids)
    table, at = [], 0
    for o in old:
        k = -(-o // page)
        table.append(ids[at:at + k] + [-9] * (cols - k))
        at += k
    return old, new, table, ids[at:], cols, len(ids)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(seed, batch, page, old_hi, new_hi, spare=5, in_place=False, extra_slots=0):
    old, new, table, free, cols, pages = case(seed, batch, page, old_hi, new_hi, spare)
    eng = engine(batch, page, cols, pages)
    want = plain(old, new, page, table, free, cols * page)
    n = sum(new) + extra_slots
    t = dict(seq_lens=i32(old), new_lens=i32(new), free_pages=i32(free + [-5, -5]), num_free=i32([len(free)]),
             block_table=i32(table), slot_map=torch.full((n,), 77, device="cuda"), positions=i32([77] * n),
             token_row=i32([77] * n), cu_new=i32([77] * (batch + 1)))
    t["seq_lens_out"] = t["seq_lens"] if in_place else i32([77] * batch)
    t["num_free_out"] = t["num_free"] if in_place else i32([77])
    eng.build_tables(t)
    torch.cuda.synchronize()
    short = want[2] != [o + k for o, k in zip(old, new)]
    assert eng.errors() == (da.DA_DEVERR_NO_PAGES if short else 0)
    assert t["block_table"].tolist() == want[0]
    assert t["num_free_out"].item() == len(want[1])
    assert t["seq_lens_out"].tolist() == want[2]
    assert t["slot_map"].tolist() == want[3] + [-1] * extra_slots
    assert t["positions"].tolist() == want[4] + [0] * extra_slots
    assert t["token_row"].tolist() == want[5] + [-1] * extra_slots
    assert t["cu_new"].tolist() == want[6]
    assert t["free_pages"].tolist() == free + [-5, -5]
    if not in_place:
        assert t["seq_lens"].tolist() == old and t["num_free"].item() == len(free)
    return eng, t


@pytest.mark.parametrize("batch", [1, 2, 33, 511, 512, 513, 1500])
@pytest.mark.parametrize("page", [16, 64, 192])
def test_decode_step(batch, page):
    check(batch + page, batch, page, 500, 1)


@pytest.mark.parametrize("batch,new_hi", [(1, 5000), (7, 3000), (61, 700), (600, 60), (3, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_prefill(batch, new_hi, in_place):
    for _ in range(2):  # the block counter is back at zero
        check(batch, batch, 16, 300, new_hi, in_place=in_place, extra_slots=13)


@pytest.mark.parametrize("spare", [-1, -3, -20, -1000])
@pytest.mark.parametrize("batch", [5, 700])
def test_pages_run_out(spare, batch):
    check(spare + batch, batch, 16, 40, 40, spare=spare)


def test_without_allocation_and_contiguous():
    old, new, table, free, cols, pages = case(1, 9, 16, 100, 0, 0)
    lens = old
    eng = engine(9, 16, cols, pages)
    n = sum(lens)
    t = dict(seq_lens=i32([0] * 9), new_lens=i32(lens), block_table=i32(table), seq_lens_out=i32([5] * 9),
             slot_map=torch.zeros(n, dtype=torch.int64, device="cuda"))
    eng.build_tables(t)  # the slots of everything that the rows hold
    assert eng.errors() == 0 and t["seq_lens_out"].tolist() == lens
    want = [table[b][p // 16] * 16 + p % 16 for b in range(9) for p in range(lens[b])]
    assert t["slot_map"].tolist() == want and t["block_table"].tolist() == table
    eng = engine(3, 0, 0, 0, contiguous=100)
    t = dict(seq_lens=i32([0, 98, 50]), new_lens=i32([2, 2, 0]), seq_lens_out=i32([0] * 3),
             slot_map=torch.zeros(5, dtype=torch.int64, device="cuda"))
    eng.build_tables(t)
    assert eng.errors() == 0 and t["slot_map"].tolist() == [0, 1, 198, 199, -1]


def test_bad_lengths_pages_and_too_few_slots():
    eng = engine(3, 16, 4, 10)
    base = dict(free_pages=i32([1, 2, 3, 4, 5]), num_free=i32([5]), num_free_out=i32([0]), seq_lens_out=i32([0] * 3))

    def run(old, new, n, **more):
        t = base | dict(seq_lens=i32(old), new_lens=i32(new), block_table=i32([[6, 7, 8, 9]] * 3),
                        slot_map=torch.full((n,), 77, device="cuda")) | more
        eng.build_tables(t)
        torch.cuda.synchronize()
        return eng.errors(), t
    err, t = run([-4, 70, 10], [1, 1, 1], 3)
    assert err == da.DA_DEVERR_SEQ_LEN and t["seq_lens_out"].tolist() == [1, 64, 11]
    assert t["slot_map"].tolist() == [5 * 16, -1, 6 * 16 + 10]
    err, t = run([0, 60, 10], [-2, 10, 1], 11)  # past the row's capacity: no slot
    assert err == da.DA_DEVERR_SEQ_LEN and t["seq_lens_out"].tolist() == [0, 64, 11]
    assert t["slot_map"].tolist() == [9 * 16 + 12 + i for i in range(4)] + [-1] * 6 + [6 * 16 + 10]
    err, t = run([0, 0, 0], [16, 16, 16], 20)
    assert err == da.DA_DEVERR_SLOT and t["slot_map"].tolist() == [80 + i for i in range(16)] + [64 + i for i in range(4)]
    err, t = run([0, 8, 0], [1, 1, 1], 3, free_pages=i32([1, 2, 3, 10, -1]), block_table=i32([[6] * 4, [12] * 4, [6] * 4]))
    assert err == da.DA_DEVERR_PAGE_INDEX and t["slot_map"].tolist() == [-1, -1, -1]
    assert t["block_table"].tolist() == [[6] * 4, [12] * 4, [6] * 4]
    err, t = run([0, 0, 0], [1, 0, 0], 1, num_free=i32([6]))
    assert err == da.DA_DEVERR_NO_PAGES and t["slot_map"].tolist() == [80]


def test_captured_decode_steps_in_place():
    batch, page, cols = 6, 16, 8
    eng = engine(batch, page, cols, 60)
    free = list(range(59, -1, -1))
    t = dict(seq_lens=i32([0] * batch), new_lens=i32([3, 1, 0, 7, 16, 5]), free_pages=i32(free), num_free=i32([60]),
             block_table=i32([[-1] * cols] * batch), slot_map=torch.zeros(32, dtype=torch.int64, device="cuda"))
    t |= dict(seq_lens_out=t["seq_lens"], num_free_out=t["num_free"])
    state = ([0] * batch, [[-1] * cols] * batch, list(free))
    eng.build_tables(t)
    torch.cuda.synchronize()
    old, table, free = state
    w = plain(old, [3, 1, 0, 7, 16, 5], page, table, free, cols * page)
    table, free, old = w[0], w[1], w[2]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eng.build_tables(t)
    for _ in range(4):
        g.replay()
        w = plain(old, [3, 1, 0, 7, 16, 5], page, table, free, cols * page)
        table, free, old = w[0], w[1], w[2]
        assert t["seq_lens"].tolist() == old and t["block_table"].tolist() == table
        assert t["num_free"].item() == len(free) and t["slot_map"].tolist() == w[3]
    assert eng.errors() == 0


def test_refusals():
    eng = engine(2, 16, 4, 8)
    t = dict(seq_lens=i32([0, 0]), new_lens=i32([1, 1]), free_pages=i32([1, 2]), num_free=i32([2]), num_free_out=i32([0]),
             block_table=i32([[0] * 4] * 2), seq_lens_out=i32([0, 0]), slot_map=torch.zeros(2, dtype=torch.int64, device="cuda"))
    ws = eng.workspace

    def status(**change):
        a = da.make_table_args(t)
        for k, v in change.items():
            setattr(a, k, v)
        return da.load().decode_attn_build_tables(eng.ctx, ctypes.byref(a), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                                  da._stream(None))
    for change in (dict(seq_lens=None), dict(new_lens=None), dict(block_table=None), dict(seq_lens_out=None),
                   dict(slot_map=None), dict(num_free=None), dict(num_free_out=None), dict(free_pages=None),
                   dict(slot_capacity=-1), dict(free_capacity=-1)):
        assert status(**change) == da.DA_ERR_INVALID_ARG, change
    a = da.make_table_args(t)
    assert da.load().decode_attn_build_tables(eng.ctx, ctypes.byref(a), ctypes.c_void_p(ws.data_ptr()), 255,
                                              da._stream(None)) == da.DA_ERR_WORKSPACE
    for bad in (dict(seq_lens=t["seq_lens"].long()), dict(cu_new=i32([0, 0])), dict(block_table=i32([0] * 7)),
                dict(seq_lens=i32([0]), new_lens=i32([0]), seq_lens_out=i32([0]))):
        with pytest.raises(ValueError):
            eng.build_tables(t | bad)
    assert eng.errors() == 0
