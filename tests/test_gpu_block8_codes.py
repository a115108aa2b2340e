"""Every code of the 8-bit block cache as a key and as a value, for up to eight and up to sixteen query rows a unit,
and scores that are small beside what their queries are made of. Bounds are those of the definition (fp4_ref): a
score's error follows from the sum of |q| |k|."""

import pytest
import torch

import block8_ref as B
from test_gpu_block8 import SCALE, check

pytestmark = pytest.mark.gpu
both = pytest.mark.parametrize("kind", ["e4m3", "int8"])
groups = pytest.mark.parametrize("group", [8, 16])


def all_codes(t, name, kind):
    """Row i's one token: 128 of the codes, turned by i; every code in two rows that follow each other."""
    raw = t[name].view(torch.uint8)
    for i in range(t["seq_lens"].numel()):
        c = (torch.arange(128) + 128 * (i % 2)).roll(i).to(torch.uint8)
        raw[int(t["block_table"][i, 0]), 0, 0] = torch.where((c & 0x7F) == 0x7F, c - 1, c) if kind == "e4m3" else c


@both
@groups
def test_every_value_code(kind, group):
    t = B.make(lens=[1] * 16, hq=group, hkv=1, kind=kind, block=16, page=16, seed=1)
    all_codes(t, "v", kind)
    for i in range(16):
        t["v_scale"][int(t["block_table"][i, 0])] = 2.0 ** (9 * i - 60)
    _, out, _ = check(t, hq=group, hkv=1, kind=kind, block=16, page=16)
    for i, p in enumerate(t["block_table"][:, 0].tolist()):
        want = B.values(t["v"][p][None], t["v_scale"][p][None], 16)[0, 0, 0]
        # the weight is 1, the scale a power of two: one rounding to bf16
        assert ((out.double().cpu()[i] - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -14)).all()


@both
@groups
def test_every_key_code(kind, group):
    """One key a row and a query that is 1 in one element: the LSE is that element's value, times the scale."""
    rows = 256 // group
    t = B.make(lens=[1] * rows, hq=group, hkv=1, kind=kind, block=16, page=16, seed=2)
    all_codes(t, "k", kind)
    t["q"].zero_()
    seen = set()
    for i in range(rows):
        for h in range(group):
            d = (h * (128 // group) + i // 2) % 128
            t["q"][i, h, d] = 1.0
            seen.add(int(t["k"].view(torch.uint8)[int(t["block_table"][i, 0]), 0, 0, d]))
    assert len(seen) == (256 if kind == "int8" else 254)
    _, _, lse = check(t, hq=group, hkv=1, kind=kind, block=16, page=16)
    for i, p in enumerate(t["block_table"][:, 0].tolist()):
        k = B.values(t["k"][p][None], t["k_scale"][p][None], 16)[0, 0, 0]
        want = (t["q"][i].double() @ k) * SCALE
        # products with 1 and 0 are exact; the score's factor, its product and the LSE's are fp32
        assert ((lse[i].double().cpu() - want).abs() <= 8 * 2.0 ** -24 * want.abs() + 2.0 ** -21).all()


@both
@pytest.mark.parametrize("group", [4, 12])
def test_codes_of_every_size(kind, group):
    """Codes at random, the integer -128 among them."""
    t = B.make(lens=[500, 33], hq=group, hkv=1, kind=kind, block=32, page=64, seed=3)
    gen = torch.Generator().manual_seed(4)
    for s in ("k", "v"):
        raw = t[s].view(torch.uint8)
        new = torch.randint(0, 256, raw.shape, generator=gen).to(torch.uint8)
        raw.copy_(torch.where((new & 0x7F) == 0x7F, 0, new) if kind == "e4m3" else new)
        t[s + "_scale"] = torch.rand(t[s + "_scale"].shape, generator=gen) * 0.02
    check(t, hq=group, hkv=1, kind=kind, block=32, page=64)


@both
@groups
@pytest.mark.parametrize("size", [1.0, 40.0, 3000.0])
@pytest.mark.parametrize("spread", [0.1, 1.0])
def test_small_codes_under_queries_that_are_not_centred(kind, group, size, spread):
    """Blocks with one great element, so that all others have the least codes, and queries whose elements do not
    cancel: scores come from differences that are small beside the queries' sum."""
    t = B.make(lens=[700], hq=group, hkv=1, kind=kind, block=16, page=16, seed=5)
    gen = torch.Generator().manual_seed(6)
    raw = t["k"].view(torch.uint8)
    one = {"e4m3": 0x01, "int8": 1}[kind]  # the least code, and its negative
    neg = {"e4m3": 0x81, "int8": 255}[kind]
    c = torch.randint(0, 3, raw.shape, generator=gen)
    new = torch.where(c == 0, 0, torch.where(c == 1, one, neg)).to(torch.uint8)
    new[:, :, 3, 50] = {"e4m3": 0xFE, "int8": 0x81}[kind]  # -448, -127
    used = raw != 0x7F
    raw.copy_(torch.where(used.any(-1, keepdim=True), new, raw))
    least = 2.0 ** -9 if kind == "e4m3" else 1.0
    t["k_scale"] = torch.where(torch.isnan(t["k_scale"]), t["k_scale"], 16.0 / size / least)
    t["q"] = (size * (1 + spread * torch.randn(t["q"].shape, generator=gen)) / (1 + spread)).to(torch.bfloat16)
    check(t, hq=group, hkv=1, kind=kind, block=16, page=16)
