"""Plain 64-bit definitions of the 8-bit block cache (e4m3 or integer codes, an fp32 scale for
each block of positions and kv head), for the tests. Everything runs on the CPU; nothing here is
shared with the library. Attention over its values and the bounds are those of fp4_ref."""

from unittest import mock

import torch

import decode_attention_flash_gb300 as da
import fp4_ref as R

D = 128
KINDS = {"e4m3": da.DA_DTYPE_FP8_E4M3_BLOCKS, "int8": da.DA_DTYPE_INT8_BLOCKS}
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
MOST = {"e4m3": 448.0, "int8": 127.0}


def codes_of(y, kind):
    """float64 quotients -> codes, to nearest even, saturating."""
    if kind == "int8":
        return y.round().clamp(-127, 127).to(torch.int8)
    y = y.clamp(-448, 448)  # (infinities too; NaN stays)
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    z = torch.where(torch.isnan(y), y, (y / unit).round() * unit)
    return z.float().to(torch.float8_e4m3fn)  # exact


def values(codes, scale, block):
    """Codes [X, H, N, 128] and scales [X, H, N / block] as float64."""
    return codes.double() * scale.double().repeat_interleave(block, -1)[..., None]


def reference(t, scale, *, block, **kw):
    """R.reference over this cache's values."""
    u = dict(t)
    for s in ("k", "v"):
        u[s], u[s + "_scale"] = values(t[s], t[s + "_scale"], block), torch.ones(t[s].shape[1])
    with mock.patch.object(R, "cache_values", lambda cache, _: cache):
        return R.reference(u, scale, **kw)


def make(*, lens, hq, hkv, kind, block, page=0, length=0, q_len=1, seed=0):
    """Inputs of one call on the CPU. Rows past a length hold NaN codes (e4m3) and blocks that no
    row reaches NaN scales."""
    gen = torch.Generator().manual_seed(seed)
    b = len(lens)
    length = length or -(-max(max(lens), block) // block) * block
    t = R.make(lens=lens, hq=hq, hkv=hkv, page=page, length=-(-length // 16) * 16, q_len=q_len, seed=seed)
    if page:
        shape = (t["k"].shape[0], hkv, page)
    else:
        shape = (b, hkv, length)
    x, h, n = shape
    used = torch.zeros(x, n, dtype=torch.bool)
    for i, m in enumerate(lens):
        for j in range(-(-m // page) if page else 1):
            used[t["block_table"][i, j] if page else i, : min(page, m - j * page) if page else m] = True
    for s in ("k", "v"):
        y = torch.randn(x, h, n // block, block, D, generator=gen, dtype=torch.float64)
        y = y * torch.exp(0.5 * torch.randn(D, generator=gen, dtype=torch.float64))
        y = y * torch.exp(0.7 * torch.randn(x, h, n // block, 1, 1, generator=gen, dtype=torch.float64))
        sc = (y.abs().amax((-2, -1)) / MOST[kind]).float()
        codes = codes_of(y / sc.double()[..., None, None], kind).reshape(x, h, n, D)
        raw = codes.view(torch.uint8)
        raw[~used[:, None].expand(-1, h, -1)] = 0x7F
        sc[~used.reshape(x, 1, -1, block).any(-1).expand(-1, h, -1)] = float("nan")
        t[s], t[s + "_scale"] = codes, sc
    return t
