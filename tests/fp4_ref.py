"""Plain 64-bit definitions of the 4-bit float cache and of attention over it,
for the tests. Everything runs on the CPU; nothing here is shared with the
library."""

import math

import torch

D = 128
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantise(x, head_scale):
    """float64 x [..., H, 128] -> codes [..., H, 64] and scales [..., H, 8] (uint8): each block of
    16 gets the e4m3 number nearest to amax / (6 head_scale), each element the grid value nearest
    to x / (block scale * head_scale), ties to even in both."""
    b = x.reshape(*x.shape[:-1], 8, 16)
    hs = head_scale.double()[:, None]
    sb = (b.abs().amax(-1) / 6 / hs).clamp(max=448.0).float().to(torch.float8_e4m3fn)
    eff = (sb.double() * hs)[..., None]
    y = torch.where(eff > 0, b.abs() / torch.where(eff > 0, eff, torch.ones_like(eff)), torch.zeros_like(b))
    y = y.clamp(max=6.0)
    unit = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    mag = torch.round(y / unit) * unit
    code = torch.searchsorted(GRID, mag.contiguous()).to(torch.uint8)
    code |= torch.signbit(b).to(torch.uint8) << 3
    code = code.reshape(*x.shape[:-1], 64, 2)
    return code[..., 0] | (code[..., 1] << 4), sb.view(torch.uint8)


def pack(codes, scales):
    """Codes [X, H, R, 64] and scales [X, H, R, 8] -> granules [X, H, R / 16, 1152]."""
    x, h, r, _ = codes.shape
    return torch.cat([codes.reshape(x, h, r // 16, 1024), scales.reshape(x, h, r // 16, 128)], -1).contiguous()


def unpack(cache):
    x, h, g, _ = cache.shape
    return (cache[..., :1024].reshape(x, h, g * 16, 64), cache[..., 1024:].reshape(x, h, g * 16, 8))


def values(codes, scales, head_scale):
    """float64 values [..., 128] of codes [..., 64] and scales [..., 8]; head_scale broadcasts to [...]."""
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D).long()
    v = GRID[nib & 7] * (1.0 - 2.0 * (nib >> 3).double())
    s = scales.contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return v * s * head_scale.double()[..., None]


def cache_values(cache, head_scale):
    """float64 [X, H, R, 128] of a whole cache."""
    codes, scales = unpack(cache)
    return values(codes, scales, head_scale[None, :, None])


def attend_row(q, k, v, keep, scale, softcap=0.0, bias=None):
    """One query row: q [128], k, v [N, 128] float64, keep [N] bool. Returns out, lse and the
    error bounds of a kernel with f16 weights (rounded by 2^-11 each, 2^-25 below 2^-14), fp32
    scores of 128 products and a bf16 output (2^-8)."""
    k, v = k[keep], v[keep]
    if k.shape[0] == 0:
        return torch.zeros(D, dtype=torch.float64), -math.inf, torch.zeros(D, dtype=torch.float64), 0.0
    s = (k @ q) * scale
    size = (k.abs() @ q.abs()) * abs(scale)
    if softcap > 0:
        s = softcap * torch.tanh(s / softcap)
    if bias is not None:
        s = s + bias[keep]
        size = size + bias[keep].abs()
    lse = torch.logsumexp(s, 0)
    w = torch.exp(s - lse)
    out = w @ v
    # relative error of a weight: 128 fp32 products and sums, three roundings of the
    # score in log2 units, the exponential; the soft cap's error is a few ulp of the cap
    delta = (160 * size.max().item() + 16 * abs(s).max().item() + 16 + 16 * softcap) * 2.0 ** -24
    low = 2.0 ** -25 * v.abs().sum(0) * math.exp(s.max().item() - lse.item())
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2 * delta) * (w @ v.abs()) + low + 2.0 ** -30
    return out, lse.item(), tol, delta + 2.0 ** -21 * (1 + abs(lse.item()))


def reference(t, scale, *, hq, hkv, q_len=1, page=0, softcap=0.0, sparse_block=0, rows=None):
    """Outputs, LSE and their tolerances, [B, HQ, Q, 128] and [B, HQ, Q], from the tensors of a call."""
    b = t["seq_lens"].numel()
    g = hq // hkv
    q = t["q"].double().reshape(b, hq, q_len, D)
    out = torch.zeros(b, hq, q_len, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.zeros(b, hq, q_len, dtype=torch.float64)
    ltol = torch.zeros_like(lse)
    for i in range(b):
        n = int(t["seq_lens"][i])
        for h in range(hkv):
            if page:
                ids = t["block_table"][i, : -(-n // page)].long()
                kc, vc = t["k"][ids, h:h + 1], t["v"][ids, h:h + 1]
            else:
                kc, vc = t["k"][i:i + 1, h:h + 1], t["v"][i:i + 1, h:h + 1]
            k = cache_values(kc, t["k_scale"][h:h + 1]).reshape(-1, D)
            v = cache_values(vc, t["v_scale"][h:h + 1]).reshape(-1, D)
            if sparse_block:
                pos, masked = [], []
                for num, idx, m in (("kv_num_blks", "kv_idx", True), ("kv_full_num_blks", "kv_full_idx", False)):
                    if num in t:
                        for blk in t[idx][i, h, : int(t[num][i, h])].tolist():
                            p = range(blk * sparse_block, min((blk + 1) * sparse_block, n))
                            pos += list(p)
                            masked += [m] * len(p)
                pos = torch.tensor(pos, dtype=torch.long)
                masked = torch.tensor(masked, dtype=torch.bool)
            else:
                pos, masked = torch.arange(n), torch.ones(n, dtype=torch.bool)
            for j in range(g):
                hd = h * g + j
                for tok in range(q_len):
                    qpos = n - q_len + tok
                    if q_len > 1 and "spec_mask" in t:
                        word = int(t["spec_mask"][i, tok])
                        new = pos - (n - q_len)
                        keep = (new < 0) | (((word >> new.clamp(0, 31)) & 1) == 1)
                    else:
                        keep = pos <= qpos
                    if "mask_window" in t:
                        w = int(t["mask_window"][hd])
                        sk = int(t["mask_sink"][hd]) if "mask_sink" in t else 0
                        keep = keep & (~masked | (pos < sk) | torch.tensor(w < 0) | (pos > qpos - w))
                    bias = None
                    if "alibi_slopes" in t:
                        bias = float(t["alibi_slopes"][hd]) * (pos - qpos).double()
                    o, l, e, le = attend_row(q[i, hd, tok], k[pos], v[pos], keep, scale, softcap, bias)
                    out[i, hd, tok], lse[i, hd, tok], tol[i, hd, tok], ltol[i, hd, tok] = o, l, e, le
    return out, lse, tol, ltol


def check(got, got_lse, ref):
    out, lse, tol, ltol = ref
    got, got_lse = got.double().cpu().reshape(out.shape), got_lse.double().cpu().reshape(lse.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(out)), "NaN in other places"
    bad = (got - out).abs() > tol
    assert not bad.any(), f"out: {int(bad.sum())} of {bad.numel()} beyond the bound, worst " \
        f"{((got - out).abs() / tol.clamp(min=1e-30)).max().item():.2f} times it"
    empty = lse == -math.inf
    assert torch.equal(got_lse == -math.inf, empty)
    d = torch.where(empty, torch.zeros_like(lse), (got_lse - lse).abs())
    assert torch.equal(torch.isnan(d), torch.isnan(lse))
    assert not (d > ltol).any(), f"lse off by {d.max().item():.2e}"


def make(*, lens, hq, hkv, page=0, length=0, q_len=1, seed=0, spare=3, extra_len=0):
    """Inputs of one call on the CPU. Cache rows that no row owns (spare pages, slots past a
    row's end) hold 0xFF bytes: every scale there is NaN."""
    gen = torch.Generator().manual_seed(seed)
    b = len(lens)
    t = dict(seq_lens=torch.tensor(lens, dtype=torch.int32))
    t["q"] = torch.randn((b, hq, q_len, D) if q_len > 1 else (b, hq, D), generator=gen).to(torch.bfloat16)
    for s in ("k_scale", "v_scale"):
        t[s] = torch.rand(hkv, generator=gen) * 0.01 + 0.001
    if page:
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        cols = max(max(need), 1) + extra_len
        perm = torch.randperm(pages, generator=gen).int()
        table = torch.full((b, cols), -7, dtype=torch.int32)  # never read
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = perm[at:at + n]
            at += n
        t["block_table"] = table
        shape = (pages, hkv, page)
    else:
        length = length or -(-max(max(lens), 16) // 16) * 16
        shape = (b, hkv, length)
    for s in ("k", "v"):
        x = torch.randn(shape[0] * shape[2], hkv, D, generator=gen, dtype=torch.float64)
        x = x * torch.exp(0.5 * torch.randn(D, generator=gen, dtype=torch.float64))
        codes, scales = quantise(x, t[s + "_scale"])
        codes = codes.reshape(shape[0], shape[2], hkv, 64).transpose(1, 2).contiguous()
        scales = scales.reshape(shape[0], shape[2], hkv, 8).transpose(1, 2).contiguous()
        used = torch.zeros(shape[0], shape[2], dtype=torch.bool)
        for i, n in enumerate(lens):
            if page:
                for j in range(-(-n // page)):
                    used[t["block_table"][i, j], : min(page, n - j * page)] = True
            else:
                used[i, :n] = True
        codes[~used[:, None].expand(-1, hkv, -1)] = 0xFF
        scales[~used[:, None].expand(-1, hkv, -1)] = 0xFF
        t[s] = pack(codes, scales)
    return t
