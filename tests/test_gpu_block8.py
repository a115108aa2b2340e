"""Decode attention over the 8-bit block cache (DA_DTYPE_FP8_E4M3_BLOCKS, DA_DTYPE_INT8_BLOCKS) on
the GPU, against a plain definition in 64 bits. The kernel's roundings are those of the 4-bit float
cache's (codes and scales are exact, weights f16, sums fp32), so the bounds are fp4_ref's."""

import math

import pytest
import torch

import block8_ref as B
import decode_attention_flash_gb300 as da
import fp4_ref as R

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
both = pytest.mark.parametrize("kind", ["e4m3", "int8"])


def engine(t, *, hq, hkv, kind, block, page=0, q_len=1, splits=0, host_lens=True, **more):
    kw = dict(batch=t["seq_lens"].numel(), num_q_heads=hq, num_kv_heads=hkv, head_dim_qk=128,
              head_dim_v=128, q_dtype=da.DA_DTYPE_BF16, kv_dtype=B.KINDS[kind], kv_groups=block, q_len=q_len)
    if page:
        cols = t["block_table"].shape[1]
        kw |= dict(kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=t["k"].shape[0],
                   max_pages_per_seq=cols, max_seq_len=cols * page)
    else:
        kw |= dict(kv_layout=da.DA_KV_CONTIGUOUS, max_seq_len=t["k"].shape[2])
    kw |= more
    return da.DecodeAttention(device=0, seq_lens_host=t["seq_lens"] if host_lens else None,
                              num_splits_override=splits, **kw)


def run(eng, t, scale=SCALE, softcap=0.0):
    dev = {k: v.cuda() for k, v in t.items()}
    lse = torch.full(t["q"].shape[:-1], 12345.0, device="cuda")
    out = torch.full(t["q"].shape, 777.0, dtype=torch.bfloat16, device="cuda")
    eng.run(dev, scale, out=out, lse=lse, softcap=softcap)
    torch.cuda.synchronize()
    return out, lse


def check(t, *, hq, hkv, kind, block, page=0, q_len=1, splits=0, scale=SCALE, softcap=0.0, sparse_block=0, **more):
    eng = engine(t, hq=hq, hkv=hkv, kind=kind, block=block, page=page, q_len=q_len, splits=splits, **more)
    out, lse = run(eng, t, scale, softcap)
    assert eng.errors() == 0
    R.check(out, lse, B.reference(t, scale, block=block, hq=hq, hkv=hkv, q_len=q_len, page=page, softcap=softcap,
                                  sparse_block=sparse_block))
    again, lse2 = run(eng, t, scale, softcap)  # same workspace, and the same bits
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    assert torch.equal(lse2.view(torch.int32), lse.view(torch.int32))
    return eng, out, lse


LENS = [1, 0, 15, 16, 17, 31, 33, 64, 700]


@both
@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (32, 32), (64, 64), (128, 32), (192, 64), (256, 256)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_paged_ragged(kind, page, block, splits):
    t = B.make(lens=LENS, hq=8, hkv=2, kind=kind, block=block, page=page, seed=page)
    check(t, hq=8, hkv=2, kind=kind, block=block, page=page, splits=splits)


@both
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 16])
def test_group_sizes_contiguous(kind, group):
    t = B.make(lens=[208, 97, 3], hq=2 * group, hkv=2, kind=kind, block=16, length=208, seed=group)
    check(t, hq=2 * group, hkv=2, kind=kind, block=16)


@both
@pytest.mark.parametrize("block", [16, 32, 64, 128, 256])
def test_contiguous_blocks(kind, block):
    t = B.make(lens=[1000, 300, 256, 1], hq=4, hkv=2, kind=kind, block=block, seed=block)
    check(t, hq=4, hkv=2, kind=kind, block=block)


@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [0, 5, 0]])
def test_smallest(lens):
    t = B.make(lens=lens, hq=4, hkv=1, kind="e4m3", block=16, page=16, seed=4)
    check(t, hq=4, hkv=1, kind="e4m3", block=16, page=16)


@pytest.mark.parametrize("n,splits", [(5000, 0), (5000, 7), (9001, 9), (9001, 64), (40000, 0), (40000, 5000)])
def test_one_long_row_over_many_ctas(n, splits):
    t = B.make(lens=[n], hq=4, hkv=1, kind="int8", block=64, page=64, seed=n)
    check(t, hq=4, hkv=1, kind="int8", block=64, page=64, splits=splits)


@both
@pytest.mark.parametrize("hq,hkv", [(32, 1), (40, 2), (128, 1)])
@pytest.mark.parametrize("page,splits", [(16, 0), (0, 0), (16, 3)])
def test_more_than_16_queries_a_head(kind, hq, hkv, page, splits):
    t = B.make(lens=[300, 0, 17, 1, 1900], hq=hq, hkv=hkv, kind=kind, block=16, page=page, seed=hq)
    check(t, hq=hq, hkv=hkv, kind=kind, block=16, page=page, splits=splits)
    t["mask_window"] = torch.tensor([50, -1, 7, 200] * (hq // 4), dtype=torch.int32)
    t["alibi_slopes"] = torch.linspace(0.01, 0.2, hq)
    check(t, hq=hq, hkv=hkv, kind=kind, block=16, page=page, splits=splits)


@pytest.mark.parametrize("group", [5, 16])
@pytest.mark.parametrize("splits", [33, 61, 0])
def test_two_long_rows_merged_in_one_and_two_levels(group, splits):
    t = B.make(lens=[4100, 3999], hq=group, hkv=1, kind="e4m3", block=32, page=64, seed=group)
    check(t, hq=group, hkv=1, kind="e4m3", block=32, page=64, splits=splits)


@both
@pytest.mark.parametrize("rows,hi", [(70, 40), (150, 3), (40, 500)])
def test_many_short_rows(kind, rows, hi):
    gen = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, hi + 1, (rows,), generator=gen).tolist()
    t = B.make(lens=lens, hq=16, hkv=8, kind=kind, block=16, page=16, seed=rows)
    check(t, hq=16, hkv=8, kind=kind, block=16, page=16)
    check(t, hq=16, hkv=8, kind=kind, block=16, page=16, splits=1)


@pytest.mark.parametrize("splits", [1, 2])
def test_few_ctas_for_many_units(splits):
    t = B.make(lens=[333, 64, 1200, 31, 95, 2, 800], hq=8, hkv=1, kind="int8", block=32, page=32, seed=5)
    check(t, hq=8, hkv=1, kind="int8", block=32, page=32, splits=splits)


@both
@pytest.mark.parametrize("q_len,group", [(2, 1), (4, 4), (16, 1), (5, 3)])
@pytest.mark.parametrize("tree", [False, True])
def test_several_query_tokens(kind, q_len, group, tree):
    t = B.make(lens=[300, q_len, 1, 33, 0], hq=2 * group, hkv=2, kind=kind, block=16, page=16, q_len=q_len, seed=q_len)
    if tree:
        gen = torch.Generator().manual_seed(1)
        t["spec_mask"] = torch.randint(0, 1 << q_len, (5, q_len), generator=gen).int()
    check(t, hq=2 * group, hkv=2, kind=kind, block=16, page=16, q_len=q_len)


@pytest.mark.parametrize("cap", [0.5, 30.0])
def test_softcap(cap):
    t = B.make(lens=[300, 17], hq=8, hkv=2, kind="e4m3", block=16, page=16, seed=8)
    check(t, hq=8, hkv=2, kind="e4m3", block=16, page=16, softcap=cap)


@both
@pytest.mark.parametrize("group", [4, 12])
def test_window_sink_and_alibi(kind, group):
    t = B.make(lens=[300, 17, 64], hq=group, hkv=1, kind=kind, block=16, page=16, seed=9)
    t["mask_window"] = torch.tensor([(-1, 1, 40, 0, 7, 100)[i % 6] for i in range(group)], dtype=torch.int32)
    check(t, hq=group, hkv=1, kind=kind, block=16, page=16)
    t["mask_sink"] = torch.tensor([i % 5 for i in range(group)], dtype=torch.int32)
    t["alibi_slopes"] = torch.tensor([2.0 ** -(i % 8) for i in range(group)])
    check(t, hq=group, hkv=1, kind=kind, block=16, page=16)


@both
@pytest.mark.parametrize("full", [False, True])
def test_block_sparse(kind, full):
    t = B.make(lens=[1000, 130, 64, 0], hq=8, hkv=2, kind=kind, block=64, length=1024, seed=10)
    gen = torch.Generator().manual_seed(2)
    t["kv_idx"] = torch.stack([torch.randperm(16, generator=gen)[:12] for _ in range(8)]).reshape(4, 2, 12).int()
    t["kv_num_blks"] = torch.randint(0, 13, (4, 2), generator=gen).int()
    if full:
        t["kv_full_idx"] = torch.stack([torch.randperm(16, generator=gen)[:12] for _ in range(8)]).reshape(4, 2, 12).int()
        t["kv_full_num_blks"] = torch.randint(0, 13, (4, 2), generator=gen).int()
        t["mask_window"] = torch.tensor([50] * 8, dtype=torch.int32)
    check(t, hq=8, hkv=2, kind=kind, block=64, sparse_block=64, sparse_block_size=64, max_sparse_blocks=12)


@both
@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_any_scale(kind, scale):
    t = B.make(lens=[200, 9], hq=4, hkv=1, kind=kind, block=16, page=16, seed=11)
    check(t, hq=4, hkv=1, kind=kind, block=16, page=16, scale=scale)


@both
def test_every_code(kind):
    # one key per row: the output is its value row, exact but for the bf16 rounding
    t = B.make(lens=[1] * 16, hq=1, hkv=1, kind=kind, block=16, page=16, seed=12)
    raw = t["v"].view(torch.uint8)
    for i in range(16):
        p = int(t["block_table"][i, 0])
        c = (torch.arange(128) + 128 * (i % 2)).roll(i).to(torch.uint8)
        raw[p, 0, 0] = torch.where((c & 0x7F) == 0x7F, c - 1, c) if kind == "e4m3" else c
        t["v_scale"][p] = 2.0 ** (9 * i - 60)
    _, out, _ = check(t, hq=1, hkv=1, kind=kind, block=16, page=16)
    want = torch.stack([B.values(t["v"][int(p)][None], t["v_scale"][int(p)][None], 16)[0, 0, 0] for p in t["block_table"][:, 0]])
    assert ((out.double().cpu()[:, 0] - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -14)).all()


def test_scales_of_any_size():
    """Values far outside f16's range: only the fp32 sums see the scales."""
    for f in (2.0 ** 60, 2.0 ** -60):
        t = B.make(lens=[300, 40], hq=4, hkv=2, kind="int8", block=32, page=64, seed=14)
        t["v_scale"] *= f
        check(t, hq=4, hkv=2, kind="int8", block=32, page=64)
        t["k_scale"] *= f
        check(t, hq=4, hkv=2, kind="int8", block=32, page=64, scale=SCALE / f)
        t["k_scale"][:, :, ::2] = 0.0  # an all-zero block may have the scale 0
        t["v_scale"][:, :, ::2] = 0.0
        check(t, hq=4, hkv=2, kind="int8", block=32, page=64, scale=SCALE / f)


@both
@pytest.mark.parametrize("group", [4, 12])
def test_scales_that_differ_and_negative_ones(kind, group):
    """Value scales from 2^-40 to 2^6 of one another, some negative: a block far below the largest keeps its
    weights' bits."""
    t = B.make(lens=[700, 90], hq=group, hkv=1, kind=kind, block=16, page=64, seed=23)
    gen = torch.Generator().manual_seed(24)
    n = t["v_scale"].numel()
    f = torch.exp2(torch.randint(-40, 7, (n,), generator=gen).float()) * (torch.randint(0, 2, (n,), generator=gen) * 2 - 1)
    t["v_scale"] = (t["v_scale"].flatten() * f).reshape(t["v_scale"].shape)
    check(t, hq=group, hkv=1, kind=kind, block=16, page=64)
    t["v_scale"] = t["v_scale"].abs() * -1
    check(t, hq=group, hkv=1, kind=kind, block=16, page=64)
    t["v_scale"] *= 2.0 ** 100
    check(t, hq=group, hkv=1, kind=kind, block=16, page=64)


def test_misaligned_scales_are_refused():
    t = B.make(lens=[20], hq=4, hkv=1, kind="e4m3", block=16, page=16, seed=25)
    eng = engine(t, hq=4, hkv=1, kind="e4m3", block=16, page=16)
    dev = {k: v.cuda() for k, v in t.items()}
    out = torch.zeros_like(dev["q"])
    for name in ("k_scale", "v_scale"):
        a = da.make_args(dev, SCALE, out)
        setattr(a, name, getattr(a, name) + 2)
        with pytest.raises(da.DecodeAttnError) as e:
            da.decode_attn_run(eng.ctx, a, eng.workspace)
        assert e.value.status == da.DA_ERR_INVALID_ARG
        setattr(a, name, None)
        with pytest.raises(da.DecodeAttnError) as e:
            da.decode_attn_run(eng.ctx, a, eng.workspace)
        assert e.value.status == da.DA_ERR_INVALID_ARG


@both
def test_nan_reaches_the_rows_that_read_it(kind):
    t = B.make(lens=[90, 90], hq=4, hkv=2, kind=kind, block=16, page=16, seed=13)
    p = int(t["block_table"][1, 3])
    clean = {k: v.clone() for k, v in t.items()}
    if kind == "e4m3":
        t["v"].view(torch.uint8)[p, 1, 5, 40] = 0xFF
    else:
        t["v_scale"][p, 1, 0] = float("nan")
    eng = engine(t, hq=4, hkv=2, kind=kind, block=16, page=16)
    out, lse = run(eng, t)
    want = torch.zeros(2, 4, 128, dtype=torch.bool)
    want[1, 2:, 40 if kind == "e4m3" else slice(None)] = True
    assert torch.equal(torch.isnan(out.cpu()), want) and torch.isfinite(lse).all()
    if kind == "e4m3":
        clean["k"].view(torch.uint8)[p, 1, 5, 40] = 0x7F
    else:
        clean["k_scale"][p, 1, 0] = float("nan")
    out, lse = run(eng, clean)
    assert torch.isnan(out.cpu()[1, 2:]).all() and torch.isnan(lse.cpu()[1, 2:]).all()
    assert torch.isfinite(out.cpu()[0]).all() and torch.isfinite(out.cpu()[1, :2]).all()


@both
@pytest.mark.parametrize("group", [2, 5])
@pytest.mark.parametrize("where", ["draft", "window", "tree"])
def test_nan_where_a_mask_hides_it(kind, group, where):
    """A token that some query rows see and others do not holds NaN: only those that see it have it."""
    q_len = 1 if where == "window" else 3
    t = B.make(lens=[66, 35], hq=group, hkv=1, kind=kind, block=16, page=16, q_len=q_len, seed=21)
    if where == "window":
        t["mask_window"] = torch.tensor([(20, -1, 3)[i % 3] for i in range(group)], dtype=torch.int32)
        at = 40
    elif where == "draft":
        at = 64  # the second query token's own position (a block that only it and the third see)
    else:
        t["spec_mask"] = torch.tensor([[1, 3, 5]] * 2, dtype=torch.int32)
        at = 64  # new token 1: seen by itself alone
    p, o = int(t["block_table"][0, at // 16]), at % 16
    for s in ("k", "v"):
        if kind == "e4m3":
            t[s].view(torch.uint8)[p, 0, o, 7] = 0x7F
        elif where != "window":
            t[s + "_scale"][p, 0, 0] = float("nan")
    ref = B.reference(t, SCALE, block=16, hq=group, hkv=1, q_len=q_len, page=16)
    assert torch.isnan(ref[0]).any() == (kind == "e4m3" or where != "window") and not torch.isnan(ref[0]).all()
    eng = engine(t, hq=group, hkv=1, kind=kind, block=16, page=16, q_len=q_len)
    out, lse = run(eng, t)
    R.check(out, lse, ref)


def test_a_bad_page_is_reported_and_skipped():
    t = B.make(lens=[100, 64], hq=4, hkv=1, kind="e4m3", block=16, page=16, seed=15)
    bad = dict(t, block_table=t["block_table"].clone())
    bad["block_table"][0, 2] = t["k"].shape[0]
    bad["block_table"][1, 1] = -1
    eng = engine(t, hq=4, hkv=1, kind="e4m3", block=16, page=16)
    out, _ = run(eng, bad)
    assert eng.errors() == da.DA_DEVERR_PAGE_INDEX and torch.isfinite(out).all()
    out, lse = run(eng, t)
    assert eng.errors() == 0
    R.check(out, lse, B.reference(t, SCALE, block=16, hq=4, hkv=1, page=16))


def test_lengths_may_change_under_one_plan_and_are_clamped():
    t = B.make(lens=[3000, 2000, 10], hq=8, hkv=2, kind="int8", block=16, page=16, seed=17)
    eng = engine(t, hq=8, hkv=2, kind="int8", block=16, page=16)
    for lens in ([3000, 2000, 10], [1, 1, 1], [0, 0, 0], [2999, 0, 9], [17, 1500, 10]):
        u = dict(t, seq_lens=torch.tensor(lens, dtype=torch.int32))
        out, lse = run(eng, u)
        assert eng.errors() == 0
        R.check(out, lse, B.reference(u, SCALE, block=16, hq=8, hkv=2, page=16))
    out, lse = run(eng, dict(t, seq_lens=torch.tensor([-3, 2000, 1 << 30], dtype=torch.int32)))
    assert eng.errors() & da.DA_DEVERR_SEQ_LEN


def test_captured_and_replayed():
    t = B.make(lens=[500, 60], hq=8, hkv=2, kind="e4m3", block=16, page=16, seed=18)
    eng = engine(t, hq=8, hkv=2, kind="e4m3", block=16, page=16)
    dev = {k: v.cuda() for k, v in t.items()}
    out, lse = torch.zeros_like(dev["q"]), torch.zeros(2, 8, device="cuda")
    eng.run(dev, SCALE, out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eng.run(dev, SCALE, out=out, lse=lse)
    dev["seq_lens"].copy_(torch.tensor([123, 7]))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    R.check(out, lse, B.reference(dict(t, seq_lens=torch.tensor([123, 7])), SCALE, block=16, hq=8, hkv=2, page=16))
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    da.decode_attn_run_noalloc(eng.ctx, da.make_args(dev, SCALE, o2, l2))
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_stalled_wait_reports_timeout_then_the_context_recovers():
    t = B.make(lens=[3000, 70], hq=8, hkv=2, kind="int8", block=16, page=16, seed=20)
    eng = engine(t, hq=8, hkv=2, kind="int8", block=16, page=16)
    assert da.load().decode_attn_test_set_stall(eng.ctx, 200_000) == da.DA_OK  # 0.2 ms
    run(eng, t)
    assert eng.errors() & da.DA_DEVERR_TIMEOUT
    out, lse = run(eng, t)
    assert eng.errors() == 0
    R.check(out, lse, B.reference(t, SCALE, block=16, hq=8, hkv=2, page=16))


def test_a_cache_past_four_gigabytes():
    """Pages behind 2^32 bytes of keys, and of values (one pool of 4.3 GB each)."""
    page, hkv = 64, 8
    pages = (1 << 32) // (page * hkv * 128) + 300
    t = B.make(lens=[200, 70], hq=16, hkv=hkv, kind="int8", block=64, page=page, seed=22)
    few = t["k"].shape[0]
    dev = {k: v.cuda() for k, v in t.items()}
    for s in ("k", "v"):
        big = torch.zeros(pages, hkv, page, 128, dtype=torch.int8, device="cuda")
        big[pages - few:] = dev[s]
        sc = torch.zeros(pages, hkv, 1, device="cuda")
        sc[pages - few:] = dev[s + "_scale"]
        dev[s], dev[s + "_scale"] = big, sc
    dev["block_table"] = torch.where(dev["block_table"] >= 0, dev["block_table"] + (pages - few), dev["block_table"])
    eng = engine(dict(t, k=dev["k"]), hq=16, hkv=hkv, kind="int8", block=64, page=page)
    out, lse = torch.zeros_like(dev["q"]), torch.zeros(2, 16, device="cuda")
    eng.run(dev, SCALE, out=out, lse=lse)
    assert eng.errors() == 0
    R.check(out, lse, B.reference(t, SCALE, block=64, hq=16, hkv=hkv, page=page))
    assert math.isfinite(float(lse.sum()))
