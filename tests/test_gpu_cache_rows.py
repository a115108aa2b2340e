"""Rows appended to the cache (rotary positions, quantisation) and read back, on
the GPU, against plain definitions in 64 bits.

Tolerances: a rotated element is two fp32 products and a sum (2^-24 of the products
each) rounded to bf16 (2^-8); a quantised element is at most half a step of its
format from the bf16 key it came from; a read-back value is one fp32 rounding or
two and one to bf16. Each is derived beside its use."""

import pytest
import torch

import decode_attention_flash_gb300 as da
import fp4_ref as R

pytestmark = pytest.mark.gpu
KINDS = {"bf16": da.DA_DTYPE_BF16, "e4m3": da.DA_DTYPE_FP8_E4M3, "token": da.DA_DTYPE_FP8_E4M3_TOKEN_SCALE,
         "int4x4": da.DA_DTYPE_INT4_GROUPS, "int4x8": da.DA_DTYPE_INT4_GROUPS, "fp4": da.DA_DTYPE_FP4_E2M1_BLOCKS}
FILL = 0x5A


class Cache:
    """One cache of `kind`: its engine and its tensors, filled with a byte pattern."""

    def __init__(self, kind, hq, hkv, *, page=16, pages=40, batch=4, length=0, q_len=1, seed=0):
        self.kind, self.hq, self.hkv, self.page = kind, hq, hkv, page
        mla = kind == "mla"
        self.groups = {"int4x4": 4, "int4x8": 8}.get(kind, 0)
        kw = dict(batch=batch, num_q_heads=128 if mla else hq, num_kv_heads=hkv, head_dim_qk=576 if mla else 128,
                  head_dim_v=512 if mla else 128, is_mla=int(mla), ckv_dim=512 * mla, kpe_dim=64 * mla,
                  q_dtype=da.DA_DTYPE_BF16, kv_dtype=KINDS.get(kind, 0), kv_groups=self.groups, q_len=q_len)
        if page:
            kw |= dict(kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=pages, max_pages_per_seq=pages,
                       max_seq_len=pages * page)
        else:
            kw |= dict(kv_layout=da.DA_KV_CONTIGUOUS, max_seq_len=length)
        self.eng = da.DecodeAttention(device=0, **kw)
        self.blocks, self.rows = (pages, page) if page else (batch, length)
        self.slots = self.blocks * self.rows
        kb, vb, _ = self.eng._cache_sizes()
        self.t = dict(k=torch.full((kb,), FILL, dtype=torch.uint8, device="cuda"),
                      v=torch.full((vb,), FILL, dtype=torch.uint8, device="cuda"))
        gen = torch.Generator().manual_seed(seed)
        if kind in ("e4m3", "fp4"):
            for s in ("k_scale", "v_scale"):
                self.t[s] = (torch.rand(hkv, generator=gen) * 0.01 + 0.002).cuda()
        if kind == "token":
            for s in ("k_scale_shift", "v_scale_shift"):
                self.t[s] = torch.full((self.slots * hkv,), FILL, dtype=torch.int32, device="cuda")

    def rows_of(self, name):
        """The cache as [slot, kv head, bytes of a row] (4-bit float: codes then scales)."""
        x = self.t[name].cpu()
        if self.kind == "mla":
            return x.view(self.slots, 1, -1)
        x = x.view(self.blocks, self.hkv, -1)
        if self.kind == "fp4":
            codes, scales = R.unpack(x.view(self.blocks, self.hkv, -1, 1152))
            x = torch.cat([codes, scales], -1)
        else:
            x = x.view(self.blocks, self.hkv, self.rows, -1)
        return x.transpose(1, 2).reshape(self.slots, self.hkv, -1)

    def words_of(self, name):
        return self.t[name].cpu().view(self.blocks, self.hkv, self.rows).transpose(1, 2).reshape(self.slots, self.hkv)

    def values(self, name, slots):
        """float64 [T, HKV, D] that the rows `slots` stand for, from the formats' definitions."""
        raw = self.rows_of(name)[slots]
        hs = self.t.get(name + "_scale")
        if self.kind in ("bf16", "mla"):
            return raw.contiguous().view(torch.bfloat16).double()
        if self.kind == "fp4":
            return R.values(raw[..., :64], raw[..., 64:], hs.cpu()[None])
        if self.kind == "e4m3":
            return raw.contiguous().view(torch.float8_e4m3fn).double() * hs.cpu().double()[None, :, None]
        if self.kind == "token":
            pair = self.words_of(name + "_scale_shift")[slots].contiguous().view(torch.float16).double()
            pair = pair.view(*raw.shape[:2], 2)
            return raw.contiguous().view(torch.float8_e4m3fn).double() * pair[..., :1] + pair[..., 1:]
        g = self.groups
        pair = raw[..., : 4 * g].contiguous().view(torch.float16).double().view(*raw.shape[:2], g, 2)
        w = raw[..., 4 * g:].long()
        codes = torch.stack([w & 15, w >> 4], -1).view(*raw.shape[:2], g, 128 // g).double()
        return (codes * pair[..., :1] + pair[..., 1:]).flatten(-2)


def tables(rot, positions, seed=0):
    """A cosine table with values of every sign (angles of 1e4^(-2i/rot) per position)."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], -1).float()


def rotate(x, pos, table, pair_axis, adjacent):
    """x [T, H, D] float64, turned; and the size of the fp32 terms of each element."""
    n = table.shape[1] // 2
    y, size = x.clone(), torch.zeros_like(x)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
        row = table[pos[pair_axis[i]].long()].double()
        c, s = row[:, i, None], row[:, n + i, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        size[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, size


def near_bf16(got, want, size):
    # two products and a sum in fp32 (at most 3 half steps of 2^-24 of the terms), then bf16
    tol = 2.0 ** -8 * (want.abs() + 3 * 2.0 ** -24 * size) + 3 * 2.0 ** -24 * size + 2.0 ** -133
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {((got.double() - want).abs() / tol).max():.2f}"


def make_inputs(c, n, *, rot, axes, fused, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    d = 64 if c.kind == "mla" else 128
    hq = 128 if c.kind == "mla" else c.hq
    kd, vd = (512, 64) if c.kind == "mla" else (c.hkv * 128, c.hkv * 128)
    wide = torch.randn(n, hq * d + kd + vd + (24 if fused else 0), generator=gen) * scale
    wide = (wide * torch.exp(0.5 * torch.randn(wide.shape[1], generator=gen))).to(torch.bfloat16).cuda()
    parts = [wide[:, : hq * d], wide[:, hq * d: hq * d + kd], wide[:, hq * d + kd: hq * d + kd + vd]]
    if not fused:
        parts = [x.contiguous() for x in parts]
    t = dict(q=parts[0].unflatten(1, (hq, d)), k_new=parts[1], v_new=parts[2])
    if c.kind != "mla":
        t["k_new"], t["v_new"] = (t[k].unflatten(1, (c.hkv, 128)) for k in ("k_new", "v_new"))
    t["slot_map"] = torch.randperm(c.slots, generator=gen)[:n].cuda()
    t["q_out"] = torch.full((n, hq, d), 99.0, dtype=torch.bfloat16, device="cuda")
    if rot:
        t["cos_sin"] = tables(rot, 500).cuda()
        t["positions"] = torch.randint(0, 500, (axes, n), generator=gen).int().cuda()
    return t


def axis_of(rot, axes, mixed):
    n = rot // 2
    if axes == 1:
        return None
    if mixed:
        return [i % axes for i in range(n)]
    return [min(i * axes // n, axes - 1) for i in range(n)]


def check_append(c, t, *, rot, pair_axis, adjacent, pad=()):
    """Appends and checks queries, the bf16 rows and every byte of the cache that is no row of the call."""
    before = {k: c.rows_of(k) for k in ("k", "v")}
    c.eng.append(t | c.t, pair_axis=pair_axis, rope_adjacent=adjacent)
    torch.cuda.synchronize()
    assert c.eng.errors() == 0
    slots = t["slot_map"].cpu()
    live = slots >= 0
    pos = torch.where(live, t["positions"].cpu(), 0) if rot else None  # (padding's are never used)
    table = t["cos_sin"].cpu() if rot else None
    ax = pair_axis or [0] * (rot // 2)

    def turned(x):
        x = x.cpu().double()
        return rotate(x, pos, table, ax, adjacent) if rot else (x, torch.zeros_like(x))
    want, size = turned(t["q"])
    got = t["q_out"].cpu()
    near_bf16(got[live], want[live], size[live])
    assert (got[~live] == 99.0).all()
    for name in ("k", "v"):
        after = c.rows_of(name)
        other = torch.ones(c.slots, dtype=torch.bool)
        other[slots[live]] = False
        assert torch.equal(after[other], before[name][other]), "a row of no token changed"
    return slots[live], live, turned


@pytest.mark.parametrize("rot,axes,mixed,adjacent", [(0, 1, False, False), (128, 1, False, False), (128, 3, False, False),
                                                     (128, 3, True, False), (96, 3, True, False), (64, 1, False, False),
                                                     (16, 2, True, False), (128, 1, False, True), (32, 3, True, True),
                                                     (128, 4, False, True)])
@pytest.mark.parametrize("n,hq,hkv,fused", [(1, 4, 1, False), (7, 6, 2, True), (300, 9, 3, True)])
def test_rotated_rows(rot, axes, mixed, adjacent, n, hq, hkv, fused):
    c = Cache("bf16", hq, hkv)
    t = make_inputs(c, n, rot=rot, axes=axes, fused=fused, seed=rot + n)
    ax = axis_of(rot, axes, mixed) if rot else None
    slots, live, turned = check_append(c, t, rot=rot, pair_axis=ax, adjacent=adjacent)
    want, size = turned(t["k_new"])
    near_bf16(c.values("k", slots), want[live], size[live])
    assert torch.equal(c.values("v", slots), t["v_new"].cpu().double())


@pytest.mark.parametrize("n,fused", [(1, False), (33, True), (700, True)])
@pytest.mark.parametrize("adjacent", [False, True])
def test_latent_rows(n, fused, adjacent):
    c = Cache("mla", 128, 1, page=64)
    t = make_inputs(c, n, rot=64, axes=1, fused=fused, seed=n)
    slots, live, turned = check_append(c, t, rot=64, pair_axis=None, adjacent=adjacent)
    want, size = turned(t["v_new"][:, None])
    near_bf16(c.values("v", slots), want, size)
    assert torch.equal(c.values("k", slots)[:, 0], t["k_new"].cpu().double())


def step_of_e4m3(x):
    """Half a step of e4m3 at |x| (normal: 2^-4 of the value's power of two; below 2^-6: 2^-10)."""
    p = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))))
    return p * 2.0 ** -4


def check_quantised(c, name, x, slots):
    """x float64 [T, HKV, 128], the bf16 values that went in."""
    got = c.values(name, slots)
    hs = c.t[name + "_scale"].cpu().double()[None, :, None] if c.kind in ("e4m3", "fp4") else None
    fine = 1 + 2.0 ** -20  # the fp32 quotients
    if c.kind == "e4m3":
        y = x / hs
        tol = step_of_e4m3(y) * fine * hs
        inside = y.abs() <= 448
        assert ((got - x).abs() <= tol)[inside].all()
        assert ((got / hs).abs() > 447)[~inside].all()
    elif c.kind == "fp4":
        raw = c.rows_of(name)[slots]
        b = x.unflatten(-1, (8, 16))
        want = b.abs().amax(-1) / 6 / hs
        sb = raw[..., 64:].contiguous().view(torch.float8_e4m3fn).double()
        assert ((sb - want.clamp(max=448.0)).abs() <= step_of_e4m3(want) * fine).all()  # (saturating)
        assert (sb == 448)[want > 448].all()
        eff = (sb * hs)[..., None].clamp(min=1e-300)
        y = (b / eff).abs()
        unit = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
        g = got.unflatten(-1, (8, 16))
        inside = y <= 6
        assert ((g - b).abs() <= unit / 2 * eff * fine + 2.0 ** -20 * b.abs())[inside].all()
        assert torch.allclose(g.abs()[~inside], (6 * eff).expand_as(g)[~inside], rtol=1e-12)
        assert (y < 6 * (1 + 2.0 ** -4) * fine).all() or (want > 448).any()
        assert ((g * b) >= 0).all()
    else:
        g = {"token": 1, "int4x4": 4, "int4x8": 8}[c.kind]
        b = x.unflatten(-1, (g, 128 // g))
        hi, lo = b.amax(-1, keepdim=True), b.amin(-1, keepdim=True)
        if c.kind == "token":
            shift, scale = (hi + lo) / 2, (hi - lo) / 896
            scale = torch.where(scale > 0, scale, torch.ones_like(scale))  # as defined for a constant row
            y = (b - shift) / scale
            # half a step of the code, the f16 roundings of scale (2^-11 each side of the quotient)
            # and of shift, and what saturates when the rounded range falls short
            tol = step_of_e4m3(y) * scale + (2.0 ** -10 * y.abs() + 2.0 ** -11) * scale + 2.0 ** -10 * shift.abs() + 2.0 ** -24
            tol = torch.maximum(tol, step_of_e4m3(y * 1.001) * scale * 1.001)
        else:
            scale = (hi - lo) / 15
            tol = scale * (0.5 + 15 * 2.0 ** -11) + 2.0 ** -11 * lo.abs() + 2.0 ** -22
        assert ((got.unflatten(-1, (g, 128 // g)) - b).abs() <= tol * fine).all()


@pytest.mark.parametrize("kind", ["e4m3", "token", "int4x4", "int4x8", "fp4"])
@pytest.mark.parametrize("n,page,length", [(1, 16, 0), (45, 64, 0), (200, 192, 0), (60, 0, 208)])
def test_quantised_rows(kind, n, page, length):
    hq, hkv = 6, 3
    kw = dict(page=page, length=length, pages=20)
    plain, c = Cache("bf16", hq, hkv, **kw), Cache(kind, hq, hkv, **kw)
    t = make_inputs(c, n, rot=128, axes=3, fused=True, seed=n)
    ax = axis_of(128, 3, False)
    plain.eng.append(t | plain.t, pair_axis=ax)
    slots, live, _ = check_append(c, t, rot=128, pair_axis=ax, adjacent=False)
    for name in ("k", "v"):
        check_quantised(c, name, plain.values(name, slots), slots)
    # and what is read back is what the bytes stand for, rounded once or twice
    out = {k: torch.full((n, hkv, 128), 99.0, dtype=torch.bfloat16, device="cuda") for k in ("k_out", "v_out")}
    c.eng.gather(c.t | out | dict(slot_map=t["slot_map"]))
    torch.cuda.synchronize()
    assert c.eng.errors() == 0
    for name in ("k", "v"):
        want = c.values(name, slots)
        assert ((out[name + "_out"].cpu().double() - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -14) * want.abs() + 2.0 ** -120).all()


@pytest.mark.parametrize("kind", ["bf16", "mla"])
def test_gather_copies_bf16_rows(kind):
    c = Cache(kind, 6, 1 if kind == "mla" else 3, page=64)
    t = make_inputs(c, 100, rot=64, axes=1, fused=False, seed=3)
    c.eng.append(t | c.t)
    kv = (512, 64) if kind == "mla" else (3 * 128, 3 * 128)
    slots = t["slot_map"].clone()
    slots[5], slots[77] = -1, slots[6]  # a padded row, and a row read twice
    out = dict(k_out=torch.full((100, kv[0]), 99.0, dtype=torch.bfloat16, device="cuda"),
               v_out=torch.full((100, kv[1]), 99.0, dtype=torch.bfloat16, device="cuda"))
    c.eng.gather(c.t | out | dict(slot_map=slots))
    torch.cuda.synchronize()
    assert c.eng.errors() == 0
    for name in ("k", "v"):
        got = out[name + "_out"].cpu().double()
        want = c.values(name, slots.cpu().clamp(min=0)).reshape(100, -1)
        assert (got[5] == 99.0).all()
        keep = torch.arange(100) != 5
        assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("kind", ["e4m3", "token", "int4x4", "fp4"])
def test_special_rows(kind):
    """Zero rows, constant rows, values below and above the formats' ranges."""
    c = Cache(kind, 1, 1)
    rows = torch.zeros(6, 1, 128)
    rows[1] = 3.0
    rows[2, 0, ::2] = 1e-30
    rows[3, 0, 7] = -200.0
    rows[4] = torch.randn(128, generator=torch.Generator().manual_seed(1)) * 1e-6
    rows[5] = 1.0
    rows[5, 0, 64:] = -1.0
    x = rows.to(torch.bfloat16).cuda()
    t = dict(k_new=x, v_new=x, slot_map=torch.tensor([5, 0, 17, 33, 2, 9]).cuda())
    c.eng.append(t | c.t)
    torch.cuda.synchronize()
    assert c.eng.errors() == 0
    got = c.values("k", t["slot_map"].cpu())
    assert torch.isfinite(got).all()
    want = rows.to(torch.bfloat16).double()
    if kind in ("token", "int4x4"):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (got[0] == 0).all()
    check_quantised(c, "k", want[[1, 3, 5]], t["slot_map"].cpu()[[1, 3, 5]])


def test_a_nan_makes_its_block_nan_and_an_infinity_saturates():
    c = Cache("fp4", 1, 1)
    x = torch.ones(1, 1, 128)
    x[0, 0, 20] = float("nan")
    x[0, 0, 100] = float("-inf")
    x = x.to(torch.bfloat16).cuda()
    t = dict(k_new=x, v_new=x, slot_map=torch.tensor([3]).cuda())
    c.eng.append(t | c.t)
    torch.cuda.synchronize()
    got = c.values("k", torch.tensor([3]))[0, 0]
    nan = torch.isnan(got)
    assert nan[16:32].all() and not nan[:16].any() and not nan[32:].any()
    assert got[100] == -6 * 448 * c.t["k_scale"].cpu().double()[0]


def test_padding_and_bad_tokens_leave_everything_as_it_was():
    c = Cache("bf16", 4, 2)
    t = make_inputs(c, 40, rot=128, axes=2, fused=True, seed=9)
    t["slot_map"][30:] = -1
    t["positions"][:, 30:] = -12345  # never used
    check_append(c, t, rot=128, pair_axis=axis_of(128, 2, False), adjacent=False)
    before = c.rows_of("k")
    t["q_out"].fill_(99.0)
    t["slot_map"][:] = -1
    t["slot_map"][3] = c.slots
    t["slot_map"][4] = -2
    t["slot_map"][5] = 7
    t["positions"][1, 5] = 500
    t["slot_map"][6] = 8
    t["positions"][0, 6] = -1
    c.eng.append(t | c.t, pair_axis=axis_of(128, 2, False))
    torch.cuda.synchronize()
    assert c.eng.errors() == da.DA_DEVERR_SLOT | da.DA_DEVERR_POSITION
    assert torch.equal(c.rows_of("k"), before) and (t["q_out"] == 99.0).all()
    assert c.eng.errors() == 0
    out = dict(k_out=torch.full((40, 256), 99.0, dtype=torch.bfloat16, device="cuda"),
               v_out=torch.full((40, 256), 99.0, dtype=torch.bfloat16, device="cuda"))
    t["slot_map"][5:] = -1
    c.eng.gather(c.t | out | dict(slot_map=t["slot_map"]))
    assert c.eng.errors() == da.DA_DEVERR_SLOT and (out["k_out"] == 99.0).all()


def test_queries_alone_in_place_and_in_the_layout_of_several_tokens():
    c = Cache("bf16", 6, 2, batch=5, q_len=2)
    t = make_inputs(c, 10, rot=128, axes=1, fused=False, seed=11)
    want, size = rotate(t["q"].cpu().double(), t["positions"].cpu(), t["cos_sin"].cpu(), [0] * 64, False)
    base = dict(q=t["q"], cos_sin=t["cos_sin"], positions=t["positions"][0])
    out = torch.zeros(5, 6, 2, 128, dtype=torch.bfloat16, device="cuda")
    c.eng.append(base | dict(q_out=out), q_len=2)
    near_bf16(out.cpu().transpose(1, 2).reshape(10, 6, 128), want, size)
    q = t["q"].clone()
    c.eng.append(base | dict(q=q, q_out=q))
    near_bf16(q.cpu(), want, size)
    assert c.eng.errors() == 0


def test_no_tokens():
    c = Cache("fp4", 4, 2)
    e = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(0, dtype=torch.int64, device="cuda")
    before = c.rows_of("k")
    c.eng.append(dict(k_new=e, v_new=e, slot_map=z) | c.t)
    c.eng.gather(dict(k_out=e, v_out=e, slot_map=z) | c.t)
    assert c.eng.errors() == 0 and torch.equal(c.rows_of("k"), before)


def test_two_streams_at_once():
    c = Cache("fp4", 8, 2, pages=200)
    t = make_inputs(c, 2000, rot=128, axes=1, fused=True, seed=12)
    c.eng.append(t | c.t)
    torch.cuda.synchronize()
    want, q = c.rows_of("k"), t["q_out"].clone()
    for k in ("k", "v"):
        c.t[k].fill_(FILL)
    t["q_out"].fill_(0)
    halves = []
    for i, s in enumerate((torch.cuda.Stream(), torch.cuda.Stream())):
        h = {k: (v[i * 1000:(i + 1) * 1000] if k in ("q", "k_new", "v_new", "q_out", "slot_map") else v) for k, v in t.items()}
        h["positions"] = t["positions"][0, i * 1000:(i + 1) * 1000].contiguous()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.eng.append(h | c.t)
        halves.append((h, s))
    torch.cuda.synchronize()
    assert c.eng.errors() == 0 and torch.equal(c.rows_of("k"), want) and torch.equal(t["q_out"], q)


def test_refusals():
    c = Cache("fp4", 4, 2)
    t = make_inputs(c, 8, rot=128, axes=1, fused=False, seed=13)
    t |= c.t
    lib = da.load()

    def status(change, call="append"):
        a = da.make_append_args(t) if call == "append" else da.make_gather_args(
            t | dict(k_out=t["k_new"], v_out=t["v_new"]))
        change(a)
        ws = c.eng.workspace
        import ctypes
        return getattr(lib, "decode_attn_" + call)(c.eng.ctx, ctypes.byref(a), ctypes.c_void_p(ws.data_ptr()),
                                                   ws.numel(), da._stream(None))
    bad = da.DA_ERR_INVALID_ARG
    for field, value, want in [("num_tokens", -1, bad), ("slot_map", None, bad), ("k", None, bad), ("v_new", None, bad),
                               ("q_out", None, bad), ("k_scale", None, bad), ("q_stride", 511, bad), ("k_stride", 128, bad),
                               ("rope_dim", 144, bad), ("rope_dim", 24, da.DA_ERR_UNSUPPORTED), ("rope_dim", -16, bad),
                               ("positions", None, bad), ("cos_sin", None, bad), ("max_position", 0, bad),
                               ("rope_axes", 0, bad), ("rope_adjacent", 2, bad), ("q_len", 2, bad), ("q_len", -1, bad),
                               ("k_new", t["k_new"].data_ptr() + 2, bad), ("q_out", t["q_out"].data_ptr() + 8, bad)]:
        assert status(lambda a: setattr(a, field, value)) == want, field
    import ctypes
    pairs = (ctypes.c_uint8 * 64)(*([0] * 63 + [1]))
    assert status(lambda a: setattr(a, "pair_axis", ctypes.cast(pairs, ctypes.c_void_p))) == bad
    for field in ("k", "slot_map", "k_out", "v_out", "v_scale"):
        assert status(lambda a: setattr(a, field, None), "gather") == bad, field
    with pytest.raises(da.DecodeAttnError):
        da.decode_attn_append(c.eng.ctx, da.make_append_args(t), c.eng.workspace[1:])
    with pytest.raises(ValueError):
        c.eng.append(t | dict(k=t["k"][:-1]))
    with pytest.raises(ValueError):
        c.eng.append(t | dict(q=t["q"][:, :3]))
    with pytest.raises(ValueError):
        c.eng.gather(t | dict(k_out=t["k_new"][:4], v_out=t["v_new"]))
    assert c.eng.errors() == 0


@pytest.mark.parametrize("n,hq,hkv", [(60, 32, 8), (1201, 15, 5), (3001, 32, 8), (3001, 6, 3), (10001, 8, 1)])
def test_many_tokens_in_one_part_and_in_several(n, hq, hkv):
    # a token's heads in as many parts as a wave of warps holds, in two, and whole
    c = Cache("bf16", hq, hkv, page=64, pages=160)
    t = make_inputs(c, n, rot=128, axes=3, fused=True, seed=n)
    slots, live, turned = check_append(c, t, rot=128, pair_axis=axis_of(128, 3, False), adjacent=False)
    want, size = turned(t["k_new"])
    near_bf16(c.values("k", slots), want[live], size[live])


@pytest.mark.parametrize("kind", ["fp4", "int4x4", "token", "bf16"])
@pytest.mark.parametrize("n,hkv", [(1, 1), (3, 5), (1000, 3), (15001, 1), (30001, 2)])
def test_read_back_of_few_and_of_many_rows(kind, n, hkv):
    # two tokens a warp: odd numbers of them, one of the two a padded one
    c = Cache(kind, hkv, hkv, page=32, pages=20)
    t = make_inputs(c, 500, rot=64, axes=1, fused=False, seed=hkv)
    c.eng.append(t | c.t)
    gen = torch.Generator().manual_seed(n)
    pick = t["slot_map"].cpu()
    slots = pick[torch.randint(0, len(pick), (n,), generator=gen)]
    slots[torch.rand(n, generator=gen) < 0.1] = -1
    out = {k: torch.full((n, hkv, 128), 99.0, dtype=torch.bfloat16, device="cuda") for k in ("k_out", "v_out")}
    c.eng.gather(c.t | out | dict(slot_map=slots.cuda()))
    torch.cuda.synchronize()
    assert c.eng.errors() == 0
    live = slots >= 0
    for name in ("k", "v"):
        got = out[name + "_out"].cpu().double()
        want = c.values(name, slots[live])
        assert (got[~live] == 99.0).all()
        assert ((got[live] - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -14) * want.abs() + 2.0 ** -120).all()
