"""Rows appended to the 8-bit block cache and read back, against a model on the host that follows the
definition: scales are powers of two and keys and values are bf16, so quotients, codes and scales are
exact and are compared bit for bit."""

import math

import pytest
import torch

import block8_ref as B
import decode_attention_flash_gb300 as da
from test_gpu_cache_rows import tables

pytestmark = pytest.mark.gpu
both = pytest.mark.parametrize("kind", ["e4m3", "int8"])


def least_scale(amax, kind):
    """float64 amax -> the least power of two that brings it into the codes' range."""
    a = amax.clamp(max=torch.finfo(torch.bfloat16).max)
    s = torch.exp2(torch.ceil(torch.log2(a / B.MOST[kind]))).clamp(min=2.0 ** -126)
    return torch.where(amax > 0, s, torch.where(torch.isnan(amax), amax, torch.zeros_like(amax)))


class Cache:
    """A block cache on the GPU and its model."""

    def __init__(self, kind, hq, hkv, *, block, page=0, pages=12, length=0, batch=2, q_len=1, seed=0):
        self.kind, self.block, self.hkv, self.hq = kind, block, hkv, hq
        kw = dict(batch=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim_qk=128, head_dim_v=128, q_len=q_len,
                  q_dtype=da.DA_DTYPE_BF16, kv_dtype=B.KINDS[kind], kv_groups=block)
        if page:
            kw |= dict(kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=pages, max_pages_per_seq=pages,
                       max_seq_len=pages * page)
        else:
            kw |= dict(kv_layout=da.DA_KV_CONTIGUOUS, max_seq_len=length)
        self.eng = da.DecodeAttention(device=0, **kw)
        self.x, self.rows = (pages, page) if page else (batch, length)
        self.slots = self.x * self.rows
        gen = torch.Generator().manual_seed(seed)
        self.m = {}
        for s in ("k", "v"):  # arbitrary codes; blocks' scales 1, or never written: 0
            self.m[s] = torch.randint(0, 256, (self.x, hkv, self.rows, 128), generator=gen).to(torch.uint8)
            if kind == "e4m3":
                self.m[s] = torch.where((self.m[s] & 0x7F) == 0x7F, 0, self.m[s])
            elif kind == "int8":
                self.m[s] = torch.where(self.m[s] == 0x80, 0, self.m[s])
            self.m[s + "_scale"] = torch.randint(0, 2, (self.x, hkv, self.rows // block), generator=gen).float()
        self.t = {k: (v.view(B.DTYPE[kind]) if v.dtype == torch.uint8 else v).cuda() for k, v in self.m.items()}

    def model(self, name, new, slots):
        """new [T, HKV, 128] bf16 to `slots`, as the definition says."""
        codes, scale = self.m[name], self.m[name + "_scale"]
        runs = {}
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < self.slots:
                runs.setdefault((s // self.rows, s % self.rows // self.block), []).append((s % self.block, i))
        for (x, j), at in runs.items():
            offs, idx = [o for o, _ in at], [i for _, i in at]
            rows = new[idx].double().transpose(0, 1)  # [HKV][n][128]
            mag = rows.abs()
            if self.kind == "e4m3":
                mag = torch.where(torch.isnan(mag), 0.0, mag)
            need = least_scale(mag.amax((1, 2)), self.kind)
            old = torch.zeros(self.hkv, dtype=torch.float64) if 0 in offs else scale[x, :, j].double()
            now = torch.maximum(old, need)
            now = torch.where(torch.isnan(old), old, torch.where(torch.isnan(need), need, now))
            part = codes[x, :, j * self.block:(j + 1) * self.block]
            stay = torch.ones(self.block, dtype=torch.bool)
            stay[offs] = False
            if 0 not in offs:
                grown = now > old
                again = B.codes_of(part.view(B.DTYPE[self.kind]).double() * (old / torch.where(now > 0, now, 1.0))[:, None, None], self.kind)
                m = grown[:, None, None] & stay[None, :, None]
                part.copy_(torch.where(m, again.view(torch.uint8), part))
            y = torch.where(now > 0, 1.0 / torch.where(now > 0, now, 1.0), 0.0)[:, None, None] * rows
            if self.kind == "int8":
                y = torch.where(torch.isnan(now)[:, None, None], 0.0, y)
            part[:, offs] = B.codes_of(y, self.kind).view(torch.uint8)
            scale[x, :, j] = now.float()

    def same(self):
        for name, want in self.m.items():
            got = self.t[name].cpu()
            if want.dtype == torch.uint8:
                got = got.view(torch.uint8)
                if self.kind == "int8":  # (a block whose scale is NaN may hold any codes)
                    dead = torch.isnan(self.m[name + "_scale"]).repeat_interleave(self.block, -1)[..., None]
                    got, want = torch.where(dead, 0, got), torch.where(dead, 0, want)
                else:  # a zero's and a NaN's sign is not the point
                    got, want = (torch.where((x & 0x7F) % 0x7F == 0, x & 0x7F, x) for x in (got, want))
                assert torch.equal(got, want), f"{name}: {int((got != want).sum())} codes differ"
            else:
                assert torch.equal(torch.isnan(got), torch.isnan(want))
                assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want)), name

    def append(self, k, v, slots, **more):
        self.eng.append({**self.t, "k_new": k.cuda(), "v_new": v.cuda(), "slot_map": slots.cuda(), **more})
        assert self.eng.errors() == 0
        self.model("k", k, slots)
        self.model("v", v, slots)


def rows(n, hkv, gen, spread=1.0):
    x = torch.randn(n, hkv, 128, generator=gen)
    return (x * torch.exp(spread * torch.randn(n, hkv, 1, generator=gen))).to(torch.bfloat16)


@both
@pytest.mark.parametrize("page,block", [(16, 16), (64, 16), (64, 32), (64, 64), (128, 128), (256, 256), (192, 64)])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_rows_grow_by_chunks(kind, page, block, hkv):
    """Two rows that share a pool take chunks of many lengths, one token and whole blocks among them."""
    c = Cache(kind, hkv, hkv, block=block, page=page, pages=8, seed=block)
    gen = torch.Generator().manual_seed(page + hkv)
    perm = torch.randperm(8, generator=gen)
    at = [0, 0]
    for step, chunk in enumerate([(1, 1), (3, 0), (block - 3, 5), (1, block), (1, 1), (2 * block + 1, 2), (1, 1), (0, 40), (1, 1)]):
        slots = []
        for b, n in enumerate(chunk):
            n = min(n, 4 * page - at[b])
            pos = torch.arange(at[b], at[b] + n)
            slots.append(perm[b * 4 + pos // page] * page + pos % page)
            at[b] += n
        pad = torch.full((step % 3,), -1)
        slots = torch.cat([slots[0], pad, slots[1], pad])
        n = slots.numel()
        # the scales of different steps differ, so that some grow and some do not
        c.append(rows(n, hkv, gen) * 2.0 ** (step % 4), rows(n, hkv, gen) * 2.0 ** (3 - step % 4), slots)
        c.same()


@both
@pytest.mark.parametrize("block", [16, 64, 256])
def test_contiguous_prefill(kind, block):
    c = Cache(kind, 4, 2, block=block, length=2048, batch=2, seed=1)
    gen = torch.Generator().manual_seed(2)
    slots = torch.cat([torch.arange(1777), 2048 + torch.arange(31, 2048)])
    c.append(rows(slots.numel(), 2, gen), rows(slots.numel(), 2, gen), slots)
    c.same()
    more = torch.cat([torch.arange(1777, 1790), torch.tensor([2048 + 5])])  # a row in the middle, written again
    c.append(rows(14, 2, gen) * 16, rows(14, 2, gen), more)
    c.same()


@both
def test_scales_just_at_the_codes_range(kind):
    """Greatest values beside the border between two scales, and of every size a bf16 has."""
    c = Cache(kind, 1, 1, block=16, page=16, pages=400, seed=3)
    gen = torch.Generator().manual_seed(4)
    most = torch.tensor([B.MOST[kind]]).to(torch.bfloat16).view(torch.int16)
    exps = torch.cat([torch.arange(-126, 118), torch.tensor([0])])
    k = torch.zeros(exps.numel(), 1, 128, dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    for i, e in enumerate(exps.tolist()):
        edge = (most + (i % 3) - 1).view(torch.bfloat16).double() * 2.0 ** (e - (8 if kind == "e4m3" else 6))
        k[i, 0] = (edge * (torch.rand(128, generator=gen, dtype=torch.float64) * 2 - 1)).to(torch.bfloat16)
        k[i, 0, 7] = edge.to(torch.bfloat16)
    v[0, 0, 0] = torch.tensor([1], dtype=torch.int16).view(torch.bfloat16)[0]  # the smallest bf16
    v[1, 0, 0] = torch.finfo(torch.bfloat16).max
    slots = torch.arange(exps.numel()) * 16
    c.append(k, v, slots)
    c.same()
    assert (c.m["v_scale"][2:exps.numel()] == 0).all()  # blocks of zeros


@both
def test_nan_and_infinity(kind):
    c = Cache(kind, 2, 2, block=16, page=16, pages=4, seed=5)
    gen = torch.Generator().manual_seed(6)
    k, v = rows(20, 2, gen), rows(20, 2, gen)
    k[3, 0, 5] = float("nan")
    v[7, 1, 9] = float("inf")
    v[8, 1, 9] = float("-inf")
    slots = torch.arange(16, 36)
    c.append(k, v, slots)
    c.same()
    c.append(rows(1, 2, gen), rows(1, 2, gen), torch.tensor([20]))  # a NaN scale stays
    c.same()
    if kind == "int8":
        assert torch.isnan(c.m["k_scale"][1, 0, 0]) and not torch.isnan(c.m["k_scale"][1, 1, 0])
    c.append(rows(16, 2, gen), rows(16, 2, gen), slots[:16])  # and goes when the block starts anew
    c.same()
    assert torch.isfinite(c.m["k_scale"]).all() and torch.isfinite(c.t["k_scale"]).all()


@both
@pytest.mark.parametrize("block", [16, 64])
def test_a_token_at_a_time_stays_near(kind, block):
    """A block filled by single tokens of growing size: integers within one step of the last scale (the
    halves of all roundings), e4m3 within half a step of its format, 2^-4 of the value, and of its least one."""
    c = Cache(kind, 1, 1, block=block, page=block, pages=2, seed=7)
    gen = torch.Generator().manual_seed(8)
    k = rows(block, 1, gen, 0.5) * torch.exp2(torch.arange(block) / 6)[:, None, None].to(torch.bfloat16)
    k = k.to(torch.bfloat16)
    for i in range(block):
        c.append(k[i:i + 1], k[i:i + 1], torch.tensor([i]))
    c.same()
    s = float(c.t["k_scale"][0, 0, 0])
    got = c.t["k"].cpu()[0, 0].double() * s
    want = k[:, 0].double()
    tol = s if kind == "int8" else 2.0 ** -4 * want.abs() + 2.0 ** -9 * s
    assert ((got - want).abs() <= tol).all()


@both
@pytest.mark.parametrize("rot,adjacent", [(128, False), (64, False), (96, True), (0, False)])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("block,n", [(16, 5), (32, 200), (64, 700)])
def test_turned_and_normed_keys_are_those_of_a_bf16_cache(kind, rot, adjacent, normed, block, n):
    c = Cache(kind, 6, 2, block=block, page=64, pages=20, seed=9)
    gen = torch.Generator().manual_seed(n)
    wide = torch.randn(n, 10, 128, generator=gen).to(torch.bfloat16).cuda()
    slots = torch.randperm(20, generator=gen)[torch.arange(n) // 64] * 64 + torch.arange(n) % 64
    t = dict(q=wide[:, :6], k_new=wide[:, 6:8], v_new=wide[:, 8:], slot_map=slots.cuda(),
             q_out=torch.zeros(n, 6, 128, dtype=torch.bfloat16, device="cuda"))
    if rot:
        t["cos_sin"] = tables(rot, 900).cuda()
        t["positions"] = torch.randint(0, 900, (2, n), generator=gen).int().cuda()
    axis = [i % 2 for i in range(rot // 2)] if rot else None
    w = dict(q_weight=torch.rand(128, generator=gen).cuda() + 0.5, k_weight=torch.rand(128, generator=gen).cuda() + 0.5) if normed else {}
    plain = da.DecodeAttention(device=0, batch=2, num_q_heads=6, num_kv_heads=2, head_dim_qk=128, head_dim_v=128,
                               kv_layout=da.DA_KV_PAGED, page_size=64, num_pages=20, max_pages_per_seq=20, max_seq_len=1280)
    pool = {s: torch.zeros(20, 2, 64, 128, dtype=torch.bfloat16, device="cuda") for s in ("k", "v")}
    plain.append({**pool, **t, **w}, pair_axis=axis, rope_adjacent=adjacent)
    q = t["q_out"].clone()
    t["q_out"].zero_()
    c.eng.append({**c.t, **t, **w}, pair_axis=axis, rope_adjacent=adjacent)
    assert c.eng.errors() == 0 and torch.equal(q, t["q_out"])
    k = pool["k"].cpu()[slots // 64, :, slots % 64]
    c.model("k", k, slots)
    c.model("v", wide[:, 8:].cpu(), slots)
    c.same()


@both
def test_bad_tokens_are_left_out(kind):
    c = Cache(kind, 2, 1, block=16, page=16, pages=4, seed=10)
    gen = torch.Generator().manual_seed(11)
    k, v = rows(30, 1, gen), rows(30, 1, gen)
    slots = torch.arange(5, 35)
    slots[11] = 64  # these three where a block begins: its other tokens stay neighbours
    slots[27] = -1
    pos = torch.arange(30).int()
    pos[8] = 100
    pos[27] = -1  # of padding
    t = dict(cos_sin=torch.cat([torch.ones(50, 64), torch.zeros(50, 64)], -1).cuda(), positions=pos.cuda())
    c.eng.append({**c.t, "k_new": k.cuda(), "v_new": v.cuda(), "slot_map": slots.cuda(), **t})
    assert c.eng.errors() == da.DA_DEVERR_SLOT | da.DA_DEVERR_POSITION
    slots[8] = -1
    c.model("k", k, slots)
    c.model("v", v, slots)
    c.same()
    slots[0] = -8
    c.eng.append({**c.t, "k_new": k[:0].cuda(), "v_new": v[:0].cuda(), "slot_map": slots[:0].cuda()})
    c.eng.append({**c.t, "k_new": k[:1].cuda(), "v_new": v[:1].cuda(), "slot_map": slots[:1].cuda()})
    assert c.eng.errors() == da.DA_DEVERR_SLOT
    c.same()


@both
@pytest.mark.parametrize("hkv,n", [(1, 1), (3, 77), (8, 1000)])
def test_read_back(kind, hkv, n):
    c = Cache(kind, hkv, hkv, block=32, page=64, pages=20, seed=12)
    gen = torch.Generator().manual_seed(13)
    for s in ("k", "v"):
        c.m[s + "_scale"] = torch.rand(c.m[s + "_scale"].shape, generator=gen) * 0.01
        c.t[s + "_scale"].copy_(c.m[s + "_scale"])
    slots = torch.randperm(c.slots, generator=gen)[:n]
    slots[0] = -1 if n > 1 else slots[0]
    out = {s + "_out": torch.full((n, hkv, 128), 5.0, dtype=torch.bfloat16, device="cuda") for s in ("k", "v")}
    c.eng.gather({**c.t, "slot_map": slots.cuda(), **out})
    assert c.eng.errors() == 0
    for s in ("k", "v"):
        raw = c.m[s].view(B.DTYPE[kind]).float() * c.m[s + "_scale"].repeat_interleave(32, -1)[..., None]
        want = raw.to(torch.bfloat16)[slots // 64, :, slots % 64]  # one fp32 product, rounded once
        if n > 1:
            want[0] = 5.0
        assert torch.equal(out[s + "_out"].cpu(), want)


def test_refusals():
    c = Cache("e4m3", 2, 2, block=16, page=16)
    gen = torch.Generator().manual_seed(14)
    t = dict(k_new=rows(3, 2, gen).cuda(), v_new=rows(3, 2, gen).cuda(), slot_map=torch.arange(3).cuda())
    with pytest.raises(ValueError):
        c.eng.append({**c.t, **t, "k_scale": torch.zeros(2, device="cuda")})
    with pytest.raises(ValueError):
        c.eng.append({**c.t, **t, "k_scale": None})
    a = da.make_append_args({**c.t, **t})
    a.k_scale = None
    with pytest.raises(da.DecodeAttnError) as e:
        da.decode_attn_append(c.eng.ctx, a, c.eng.workspace)
    assert e.value.status == da.DA_ERR_INVALID_ARG
    a = da.make_append_args({**c.t, **t})
    a.v_scale += 2
    with pytest.raises(da.DecodeAttnError) as e:
        da.decode_attn_append(c.eng.ctx, a, c.eng.workspace)
    assert e.value.status == da.DA_ERR_INVALID_ARG
    c.same()
    assert math.isfinite(float(c.t["k_scale"].sum()))
