"""Queries, keys and latent rows normed head by head on their way into the cache
(decode_attn_append_normed), against the definition in 64 bits.

The bound: y = x rsqrt(mean x^2 + eps) w in fp32. The mean of 128 (512) squares is off by at most
24 half steps of 2^-24 (sums of 16 to 20 terms, then 4 or 5 additions), of which the root takes half;
rsqrt itself by 2 units (4 half steps), two products one each: 20. The turn adds 3 (two products, a
sum). Then bf16, 2^-8."""

import pytest
import torch

import decode_attention_flash_gb300 as da
from test_gpu_cache_rows import Cache, make_inputs, rotate

pytestmark = pytest.mark.gpu
EPS = 1e-6


def norm(x, w, eps=EPS):
    if w is None:
        return x
    return x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w.cpu().double()


def near(got, want, size):
    tol = 2.0 ** -8 * want.abs() + 23 * 2.0 ** -24 * size * (1 + 2.0 ** -8) + 2.0 ** -133
    bad = (got.cpu().double() - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {((got.cpu().double() - want).abs() / tol).max():.2f}"


def turned(x, w, t, pair_axis, adjacent, eps=EPS):
    """x [T, H, 128] normed and turned in 64 bits, and the size of each element's terms."""
    y = norm(x.cpu().double(), w, eps)
    if "cos_sin" not in t:
        return y, y.abs()
    table, pos = t["cos_sin"].cpu(), t["positions"].cpu()
    axes = pair_axis if pair_axis is not None else [0] * (table.shape[1] // 2)
    z, size = rotate(y, pos if pos.dim() == 2 else pos[None], table, axes, adjacent)
    return z, torch.maximum(size, y.abs())


def weights(n, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.exp(0.5 * torch.randn(n, generator=gen)).cuda()


def check(c, n, *, rot=128, axes=1, fused=True, adjacent=False, which="qk", seed=0, scale=1.0, eps=EPS, pair_axis=None):
    t = make_inputs(c, n, rot=rot, axes=axes, fused=fused, seed=seed, scale=scale)
    wq = weights(128, seed + 1) if "q" in which else None
    wk = weights(128, seed + 2) if "k" in which else None
    args = {**c.t, **t}
    c.eng.append({**args, "q_weight": wq, "k_weight": wk}, pair_axis=pair_axis, rope_adjacent=adjacent, norm_eps=eps)
    assert c.eng.errors() == 0
    near(t["q_out"], *turned(t["q"], wq, t, pair_axis, adjacent, eps))
    slots = t["slot_map"].cpu()
    if c.kind == "bf16":
        k, size = turned(t["k_new"], wk, t, pair_axis, adjacent, eps)
        near(c.values("k", slots), k, size)
        assert torch.equal(c.values("v", slots), t["v_new"].cpu().double())
    return t


@pytest.mark.parametrize("rot", [0, 16, 64, 96, 128])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("which", ["qk", "q", "k"])
def test_rotations(rot, adjacent, which):
    c = Cache("bf16", 6, 2, page=16, pages=6)
    check(c, 37, rot=rot, adjacent=adjacent, which=which, seed=rot)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (32, 8), (40, 8), (64, 16)])
@pytest.mark.parametrize("n", [1, 2, 33, 700])
def test_heads_and_tokens(hq, hkv, n):
    c = Cache("bf16", hq, hkv, page=64, pages=12)
    check(c, n, axes=3, pair_axis=[i % 3 for i in range(64)], seed=n)


def test_many_tokens():
    c = Cache("bf16", 8, 2, page=64, pages=160)
    check(c, 9999, fused=False, seed=3)


@pytest.mark.parametrize("scale", [1e-20, 1e-4, 1e15])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
def test_sizes_and_eps(scale, eps):
    """Heads far below eps, and large ones (whose squares stay in fp32)."""
    if scale == 1e-20 and eps == 0.0:
        scale = 1e-15  # (squares of 1e-20 are below fp32's range)
    c = Cache("bf16", 4, 2, page=16, pages=4)
    check(c, 20, scale=scale, eps=eps, seed=4)


@pytest.mark.parametrize("kind", ["e4m3", "token", "int4x4", "int4x8", "fp4"])
def test_quantised_kinds_hold_the_normed_key(kind):
    """The same bits as the append of what a bf16 cache holds."""
    c, b = Cache(kind, 4, 2, page=16, pages=6, seed=1), Cache("bf16", 4, 2, page=16, pages=6)
    t = make_inputs(c, 50, rot=64, axes=1, fused=True, seed=5)
    w = dict(q_weight=weights(128, 1), k_weight=weights(128, 2))
    c.eng.append({**c.t, **t, **w})
    q = t["q_out"].clone()
    b.eng.append({**b.t, **t, **w})
    assert torch.equal(q, t["q_out"])
    k = b.values("k", t["slot_map"].cpu()).to(torch.bfloat16).cuda()
    d = Cache(kind, 4, 2, page=16, pages=6, seed=1)
    d.eng.append({**d.t, "k_new": k, "v_new": t["v_new"], "slot_map": t["slot_map"]})
    for name in c.t:
        assert torch.equal(c.t[name], d.t[name])
    assert c.eng.errors() == d.eng.errors() == 0


@pytest.mark.parametrize("n", [1, 65, 3000])
def test_latent_rows(n):
    c = Cache("mla", 128, 1, page=64, pages=50)
    t = make_inputs(c, n, rot=64, axes=1, fused=True, seed=n)
    w = weights(512, 9)
    c.eng.append({**c.t, **t, "k_weight": w})
    assert c.eng.errors() == 0
    slots = t["slot_map"].cpu()
    want = norm(t["k_new"].cpu().double(), w)
    near(c.values("k", slots)[:, 0], want, want.abs())
    plain = Cache("mla", 128, 1, page=64, pages=50)
    q = t["q_out"].clone()
    plain.eng.append({**plain.t, **t})  # queries and rope keys are those of an append without a norm
    assert torch.equal(q, t["q_out"]) and torch.equal(plain.t["v"], c.t["v"])


def test_without_weights_it_is_the_append():
    c, d = Cache("bf16", 8, 2), Cache("bf16", 8, 2)
    t = make_inputs(c, 40, rot=128, axes=1, fused=True, seed=6)
    c.eng.append({**c.t, **t})
    q = t["q_out"].clone()
    args = da.make_append_args({**d.t, **t})
    da.decode_attn_append_normed(d.eng.ctx, args, da.make_norm_args({}), d.eng.workspace)
    assert torch.equal(q, t["q_out"]) and torch.equal(c.t["k"], d.t["k"]) and torch.equal(c.t["v"], d.t["v"])


def test_several_query_tokens_in_place_and_alone():
    c = Cache("bf16", 4, 2, batch=5, q_len=3)
    t = make_inputs(c, 15, rot=128, axes=1, fused=False, seed=7)
    w = weights(128, 8)
    flat = t["q_out"].clone()
    c.eng.append({**c.t, **t, "q_out": flat, "q_weight": w})
    out = torch.zeros(5, 4, 3, 128, dtype=torch.bfloat16, device="cuda")
    c.eng.append({**c.t, **t, "q_out": out, "q_weight": w}, q_len=3)
    assert torch.equal(out.transpose(1, 2).reshape(15, 4, 128), flat)
    q = t["q"].contiguous().clone()  # queries alone, in place
    c.eng.append({"q": q, "q_out": q, "positions": t["positions"], "cos_sin": t["cos_sin"], "q_weight": w})
    assert torch.equal(q, flat)


def test_padding_and_bad_positions_leave_their_rows():
    c = Cache("bf16", 6, 3, page=16, pages=4)
    t = make_inputs(c, 20, rot=128, axes=1, fused=True, seed=9)
    t["slot_map"][3] = -1
    t["slot_map"][7] = c.slots
    t["positions"][0, 11] = 500
    t["positions"][0, 3] = -9  # of padding: not looked at
    before = c.values("k", torch.arange(c.slots))
    t["q"][3] = float("nan")
    c.eng.append({**c.t, **t, "q_weight": weights(128, 1), "k_weight": weights(128, 2)})
    assert c.eng.errors() == da.DA_DEVERR_SLOT | da.DA_DEVERR_POSITION
    for i in (3, 7, 11):
        assert (t["q_out"][i] == 99).all()
    good = [i for i in range(20) if i not in (3, 7, 11)]
    slots = t["slot_map"].cpu()[good]
    after = c.values("k", torch.arange(c.slots))
    rest = torch.ones(c.slots, dtype=torch.bool)
    rest[slots] = False
    assert torch.equal(before[rest], after[rest])
    u = {k: (v[good] if k != "positions" and k != "cos_sin" else v[:, good] if k == "positions" else v) for k, v in t.items()}
    near(u["q_out"], *turned(u["q"], weights(128, 1), u, None, False))


def test_nan_and_infinity_stay_in_their_head():
    c = Cache("bf16", 4, 2, page=16, pages=4)
    t = make_inputs(c, 8, rot=128, axes=1, fused=True, seed=10)
    t["q"][2, 1, 5] = float("nan")
    t["k_new"][4, 1, 100] = float("inf")
    c.eng.append({**c.t, **t, "q_weight": weights(128, 1), "k_weight": weights(128, 2)})
    nan = torch.isnan(t["q_out"]).cpu()
    want = torch.zeros_like(nan)
    want[2, 1] = True
    assert torch.equal(nan, want)
    # x rsqrt(inf): 0 for finite elements, NaN for the infinite one (and what it is turned with)
    k = c.values("k", t["slot_map"].cpu())
    nan = torch.isnan(k)
    want = torch.zeros_like(nan)
    want[4, 1, [36, 100]] = True
    assert torch.equal(nan, want) and (k[4, 1][~want[4, 1]] == 0).all()


def test_captured_and_on_another_stream():
    c = Cache("bf16", 8, 2, page=16, pages=8)
    t = make_inputs(c, 30, rot=128, axes=1, fused=True, seed=11)
    w = dict(q_weight=weights(128, 1), k_weight=weights(128, 2))
    c.eng.append({**c.t, **t, **w})
    want = t["q_out"].clone()
    args, norm_args = da.make_append_args({**c.t, **t}), da.make_norm_args(w, EPS)
    t["q_out"].zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    da.decode_attn_append_normed(c.eng.ctx, args, norm_args, c.eng.workspace, stream=s)
    s.synchronize()
    assert torch.equal(t["q_out"], want)
    t["q_out"].zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        da.decode_attn_append_normed(c.eng.ctx, args, norm_args, c.eng.workspace)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(t["q_out"], want)


def test_refusals():
    c = Cache("bf16", 4, 2)
    t = make_inputs(c, 8, rot=128, axes=1, fused=True, seed=12)
    w = weights(132, 1)
    args = da.make_append_args({**c.t, **t})

    def status(a, n):
        with pytest.raises(da.DecodeAttnError) as e:
            da.decode_attn_append_normed(c.eng.ctx, a, n, c.eng.workspace)
        return e.value.status

    for eps in (-1.0, float("nan"), float("inf")):
        assert status(args, da.make_norm_args(dict(q_weight=w[:128]), eps)) == da.DA_ERR_INVALID_ARG
    bad = da.make_norm_args(dict(q_weight=w[1:129]))  # 4-byte aligned
    assert status(args, bad) == da.DA_ERR_INVALID_ARG
    only_k = da.make_append_args({**c.t, **{k: v for k, v in t.items() if k not in ("q", "q_out")}})
    assert status(only_k, da.make_norm_args(dict(q_weight=w[:128]))) == da.DA_ERR_INVALID_ARG
    only_q = da.make_append_args({k: t[k] for k in ("q", "q_out", "positions", "cos_sin")})
    assert status(only_q, da.make_norm_args(dict(k_weight=w[:128]))) == da.DA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        da.make_norm_args(dict(q_weight=w))
    with pytest.raises(ValueError):
        da.make_norm_args(dict(q_weight=w[:128].half()))
    with pytest.raises(ValueError):
        c.eng.append({**c.t, **t, "k_weight": torch.ones(512, device="cuda")})
    m = Cache("mla", 128, 1, page=64, pages=4)
    u = make_inputs(m, 8, rot=64, axes=1, fused=True, seed=13)
    with pytest.raises(da.DecodeAttnError) as e:
        m.eng.append({**m.t, **u, "q_weight": w[:128].contiguous()})
    assert e.value.status == da.DA_ERR_UNSUPPORTED
    assert c.eng.errors() == 0
