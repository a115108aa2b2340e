"""Decode attention over the 4-bit float cache (DA_DTYPE_FP4_E2M1_BLOCKS) on the
GPU, against a plain definition in 64 bits. The tolerances are the sums of the
roundings that the kernel makes (tests/fp4_ref.py, attend_row)."""

import math

import pytest
import torch

import decode_attention_flash_gb300 as da
import fp4_ref as R

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def engine(t, *, hq, hkv, page=0, q_len=1, splits=0, host_lens=True, **more):
    kw = dict(batch=t["seq_lens"].numel(), num_q_heads=hq, num_kv_heads=hkv, head_dim_qk=128,
              head_dim_v=128, q_dtype=da.DA_DTYPE_BF16, kv_dtype=da.DA_DTYPE_FP4_E2M1_BLOCKS, q_len=q_len)
    if page:
        cols = t["block_table"].shape[1]
        kw |= dict(kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=t["k"].shape[0],
                   max_pages_per_seq=cols, max_seq_len=cols * page)
    else:
        kw |= dict(kv_layout=da.DA_KV_CONTIGUOUS, max_seq_len=t["k"].shape[2] * 16)
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


def check(t, *, hq, hkv, page=0, q_len=1, splits=0, scale=SCALE, softcap=0.0, sparse_block=0, **more):
    eng = engine(t, hq=hq, hkv=hkv, page=page, q_len=q_len, splits=splits, **more)
    out, lse = run(eng, t, scale, softcap)
    assert eng.errors() == 0
    R.check(out, lse, R.reference(t, scale, hq=hq, hkv=hkv, q_len=q_len, page=page, softcap=softcap,
                                  sparse_block=sparse_block))
    again, lse2 = run(eng, t, scale, softcap)  # same workspace, and the same bits
    assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(lse2, lse)
    return eng, out, lse


LENS = [1, 0, 15, 16, 17, 31, 33, 64, 700]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 192])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_paged_ragged(page, splits):
    check(R.make(lens=LENS, hq=8, hkv=2, page=page, seed=page), hq=8, hkv=2, page=page, splits=splits)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 16])
def test_group_sizes_contiguous(group):
    t = R.make(lens=[208, 97, 3], hq=2 * group, hkv=2, length=208, seed=group)
    check(t, hq=2 * group, hkv=2)


@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [0, 5, 0]])
def test_smallest(lens):
    check(R.make(lens=lens, hq=4, hkv=1, page=16, seed=4), hq=4, hkv=1, page=16)


@pytest.mark.parametrize("n,splits", [(5000, 0), (5000, 7), (9001, 8), (9001, 9), (9001, 64), (40000, 0)])
def test_one_long_row_over_many_ctas(n, splits):
    check(R.make(lens=[n], hq=4, hkv=1, page=64, seed=n), hq=4, hkv=1, page=64, splits=splits)


@pytest.mark.parametrize("hq,hkv", [(32, 1), (40, 2), (72, 3), (128, 1)])
@pytest.mark.parametrize("page,splits", [(16, 0), (64, 0), (0, 0), (16, 3)])
def test_more_than_16_queries_a_head(hq, hkv, page, splits):
    t = R.make(lens=[300, 0, 17, 1, 1900], hq=hq, hkv=hkv, page=page, length=0 if page else 1904, seed=hq)
    check(t, hq=hq, hkv=hkv, page=page, splits=splits)
    t["mask_window"] = torch.tensor([50, -1, 7, 200] * (hq // 4), dtype=torch.int32)
    t["alibi_slopes"] = torch.linspace(0.01, 0.2, hq)
    check(t, hq=hq, hkv=hkv, page=page, splits=splits)


@pytest.mark.parametrize("group", [1, 5, 8, 12, 16])
@pytest.mark.parametrize("splits", [33, 61, 0])
def test_two_long_rows_merged_in_one_and_two_levels(group, splits):
    # 33 and 61 pieces of a row, and the number that the planned lengths give
    check(R.make(lens=[4100, 3999], hq=group, hkv=1, page=64, seed=group), hq=group, hkv=1, page=64, splits=splits)


@pytest.mark.parametrize("splits", [1000, 5000])
def test_as_many_pieces_as_two_levels_merge(splits):
    check(R.make(lens=[40000], hq=4, hkv=1, page=64, seed=6), hq=4, hkv=1, page=64, splits=splits)


@pytest.mark.parametrize("rows,hi", [(70, 40), (150, 3), (40, 500)])
def test_many_short_rows(rows, hi):
    # warps whose range holds several whole units, and pieces of two others
    gen = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, hi + 1, (rows,), generator=gen).tolist()
    t = R.make(lens=lens, hq=16, hkv=8, page=16, seed=rows)
    check(t, hq=16, hkv=8, page=16)
    check(t, hq=16, hkv=8, page=16, splits=1)


@pytest.mark.parametrize("splits", [1, 2])
def test_few_ctas_for_many_units(splits):
    # one CTA for everything: pieces of a unit between warps, heads and tails of every kind
    t = R.make(lens=[333, 64, 1200, 31, 95, 2, 800], hq=8, hkv=1, page=32, seed=5)
    eng = engine(t, hq=8, hkv=1, page=32)
    # the planner takes splits x units CTAs; fewer CTAs come from a batch of its own per row
    check(t, hq=8, hkv=1, page=32, splits=splits)
    assert eng.plan["num_units"] == 7


@pytest.mark.parametrize("q_len,group", [(2, 1), (3, 2), (4, 4), (16, 1), (5, 3)])
@pytest.mark.parametrize("tree", [False, True])
def test_several_query_tokens(q_len, group, tree):
    t = R.make(lens=[300, q_len, 1, 33, 0], hq=2 * group, hkv=2, page=16, q_len=q_len, seed=q_len)
    if tree:
        gen = torch.Generator().manual_seed(1)
        t["spec_mask"] = torch.randint(0, 1 << q_len, (5, q_len), generator=gen).int()
    check(t, hq=2 * group, hkv=2, page=16, q_len=q_len)


@pytest.mark.parametrize("cap", [0.5, 30.0])
def test_softcap(cap):
    check(R.make(lens=[300, 17], hq=8, hkv=2, page=16, seed=8), hq=8, hkv=2, page=16, softcap=cap)


@pytest.mark.parametrize("group", [4, 12])
def test_window_sink_and_alibi(group):
    t = R.make(lens=[300, 17, 64], hq=group, hkv=1, page=16, seed=9)
    t["mask_window"] = torch.tensor([(-1, 1, 40, 0, 7, 100)[i % 6] for i in range(group)], dtype=torch.int32)
    check(t, hq=group, hkv=1, page=16)
    t["mask_sink"] = torch.tensor([i % 5 for i in range(group)], dtype=torch.int32)
    t["alibi_slopes"] = torch.tensor([2.0 ** -(i % 8) for i in range(group)])
    check(t, hq=group, hkv=1, page=16)


@pytest.mark.parametrize("full", [False, True])
def test_block_sparse(full):
    lens = [1000, 130, 64, 0]
    t = R.make(lens=lens, hq=8, hkv=2, length=1024, seed=10)
    gen = torch.Generator().manual_seed(2)
    t["kv_idx"] = torch.stack([torch.randperm(16, generator=gen)[:12] for _ in range(8)]).reshape(4, 2, 12).int()
    t["kv_num_blks"] = torch.randint(0, 13, (4, 2), generator=gen).int()
    if full:
        t["kv_full_idx"] = torch.stack([torch.randperm(16, generator=gen)[:12] for _ in range(8)]).reshape(4, 2, 12).int()
        t["kv_full_num_blks"] = torch.randint(0, 13, (4, 2), generator=gen).int()
        t["mask_window"] = torch.tensor([50] * 8, dtype=torch.int32)
    check(t, hq=8, hkv=2, sparse_block=64, sparse_block_size=64, max_sparse_blocks=12)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_any_scale(scale):
    check(R.make(lens=[200, 9], hq=4, hkv=1, page=16, seed=11), hq=4, hkv=1, page=16, scale=scale)


def test_every_code_and_scale_of_the_format():
    # one key per row: the output is its value row, exact but for the bf16 rounding
    t = R.make(lens=[1] * 64, hq=1, hkv=1, page=16, seed=12)
    codes, scales = R.unpack(t["v"])
    for i in range(64):
        p = int(t["block_table"][i, 0])
        codes[p, 0, 0] = torch.arange(64) * 4 + i % 4
        codes[p, 0, 0] = codes[p, 0, 0].roll(i)
        scales[p, 0, 0] = torch.tensor([(8 * i + j) % 0x7F for j in range(8)], dtype=torch.uint8)
    t["v"] = R.pack(codes, scales)
    eng, out, _ = check(t, hq=1, hkv=1, page=16)
    want = torch.stack([R.cache_values(t["v"][int(p)][None], t["v_scale"])[0, 0, 0] for p in t["block_table"][:, 0]])
    assert ((out.double().cpu()[:, 0] - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -14)).all()


def test_a_nan_scale_reaches_the_rows_that_read_it():
    t = R.make(lens=[90, 90], hq=4, hkv=2, page=16, seed=13)
    codes, scales = R.unpack(t["v"])
    p = int(t["block_table"][1, 3])
    scales[p, 1, 5, 2] = 0x7F  # row 1, kv head 1, elements 32..47 of position 53
    t["v"] = R.pack(codes, scales)
    eng = engine(t, hq=4, hkv=2, page=16)
    out, lse = run(eng, t)
    nan = torch.isnan(out.cpu())
    want = torch.zeros_like(nan)
    want[1, 2:, 32:48] = True
    assert torch.equal(nan, want) and torch.isfinite(lse).all()
    codes, scales = R.unpack(t["k"])
    scales[p, 1, 5, 2] = 0xFF
    t["k"] = R.pack(codes, scales)
    out, lse = run(eng, t)
    assert torch.isnan(out.cpu()[1, 2:]).all() and torch.isnan(lse.cpu()[1, 2:]).all()
    assert torch.isfinite(out.cpu()[0]).all() and torch.isfinite(out.cpu()[1, :2]).all()


def test_queries_of_any_size():
    t = R.make(lens=[300], hq=8, hkv=2, page=16, seed=14)
    for f in (2.0 ** 40, 2.0 ** -40, 0.0):
        u = dict(t, q=(t["q"].float() * f).to(torch.bfloat16))
        check(u, hq=8, hkv=2, page=16, scale=SCALE / f if f else SCALE)


def test_a_bad_page_is_reported_and_skipped():
    t = R.make(lens=[100, 64], hq=4, hkv=1, page=16, seed=15)
    bad = dict(t, block_table=t["block_table"].clone())
    bad["block_table"][0, 2] = t["k"].shape[0]
    bad["block_table"][1, 1] = -1
    eng = engine(t, hq=4, hkv=1, page=16)
    out, _ = run(eng, bad)
    assert eng.errors() == da.DA_DEVERR_PAGE_INDEX and torch.isfinite(out).all()
    out, lse = run(eng, t)
    assert eng.errors() == 0
    R.check(out, lse, R.reference(t, SCALE, hq=4, hkv=1, page=16))


def test_bad_lengths_are_clamped():
    t = R.make(lens=[64, 32], hq=4, hkv=1, page=16, seed=16)
    eng = engine(t, hq=4, hkv=1, page=16, host_lens=False)
    bad = dict(t, seq_lens=torch.tensor([65, -3], dtype=torch.int32))
    out, lse = run(eng, bad)
    assert eng.errors() == da.DA_DEVERR_SEQ_LEN
    R.check(out, lse, R.reference(dict(t, seq_lens=torch.tensor([64, 0])), SCALE, hq=4, hkv=1, page=16))


def test_lengths_may_change_under_one_plan():
    t = R.make(lens=[3000, 2000, 10], hq=8, hkv=2, page=16, seed=17)
    eng = engine(t, hq=8, hkv=2, page=16)
    for lens in ([3000, 2000, 10], [1, 1, 1], [0, 0, 0], [2999, 0, 9], [17, 1500, 10]):
        u = dict(t, seq_lens=torch.tensor(lens, dtype=torch.int32))
        out, lse = run(eng, u)
        assert eng.errors() == 0
        R.check(out, lse, R.reference(u, SCALE, hq=8, hkv=2, page=16))


def test_captured_and_replayed():
    t = R.make(lens=[500, 60], hq=8, hkv=2, page=16, seed=18)
    eng = engine(t, hq=8, hkv=2, page=16)
    dev = {k: v.cuda() for k, v in t.items()}
    out = torch.zeros_like(dev["q"])
    lse = torch.zeros(2, 8, device="cuda")
    eng.run(dev, SCALE, out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eng.run(dev, SCALE, out=out, lse=lse)
    dev["seq_lens"].copy_(torch.tensor([123, 7]))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    R.check(out, lse, R.reference(dict(t, seq_lens=torch.tensor([123, 7])), SCALE, hq=8, hkv=2, page=16))


def test_noalloc_matches():
    t = R.make(lens=[700, 60], hq=8, hkv=2, page=16, seed=19)
    eng, out, lse = check(t, hq=8, hkv=2, page=16)
    dev = {k: v.cuda() for k, v in t.items()}
    o2, l2 = torch.zeros_like(dev["q"]), torch.zeros(2, 8, device="cuda")
    da.decode_attn_run_noalloc(eng.ctx, da.make_args(dev, SCALE, o2, l2))
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_stalled_wait_reports_timeout_then_the_context_recovers():
    t = R.make(lens=[3000, 70], hq=8, hkv=2, page=16, seed=20)
    eng = engine(t, hq=8, hkv=2, page=16)
    assert da.load().decode_attn_test_set_stall(eng.ctx, 200_000) == da.DA_OK  # 0.2 ms
    run(eng, t)
    assert eng.errors() & da.DA_DEVERR_TIMEOUT
    out, lse = run(eng, t)
    assert eng.errors() == 0
    R.check(out, lse, R.reference(t, SCALE, hq=8, hkv=2, page=16))


def test_one_great_weight_before_many_small_ones():
    """The first token weighs 2^24 / 1.49 times every other: f16 alone would take each of the
    others for 2/3 of its weight. More units than warps, so a warp sees a row in one piece; the
    rows share their pages. The bound, as in fp4_ref: bf16 2^-8, f16 weights 2^-11 (2^-25 of the
    reference for the smallest, which is 2^-5 of the greatest), the weight's own error."""
    n, batch, page = 131072, 304, 64
    k = torch.zeros(n // page, 8, page // 16, 1152, dtype=torch.uint8)
    v = torch.full((n // page, 8, page // 16, 1152), 0xFF, dtype=torch.uint8)  # -6
    k[..., 1024:] = 0x38
    v[..., 1024:] = 0x38
    k[0, :, 0, :64] = 0x22  # 1
    v[0, :, 0, :64] = 0x11  # 0.5
    t = dict(k=k, v=v, k_scale=torch.ones(8), v_scale=torch.ones(8), q=torch.ones(batch, 8, 128, dtype=torch.bfloat16),
             seq_lens=torch.full((batch,), n, dtype=torch.int32),
             block_table=torch.arange(n // page, dtype=torch.int32).repeat(batch, 1))
    scale = float(torch.tensor(math.log(2 ** 24 / 1.49) / 128))
    small = math.exp(-128 * scale)
    total = 1 + (n - 1) * small
    want = (0.5 - 6 * (n - 1) * small) / total
    spread = (0.5 + 6 * (n - 1) * small) / total
    tol = 2.0 ** -8 * abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + 6 * (n - 1) * 2.0 ** -30 / total
    eng = engine(t, hq=8, hkv=8, page=page)
    out, lse = run(eng, t, scale)
    assert eng.errors() == 0
    assert (out.double() - want).abs().max().item() <= tol
    assert (lse.double() - (128 * scale + math.log(total))).abs().max().item() <= 2.0 ** -12
