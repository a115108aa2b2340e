"""Measured cases of the cache operators around decode attention.

Four operators that one serving step uses in turn: block tables and slot maps
built from the requests' lengths, rotary positions (one or several axes) with
the append of the new keys and values to the cache, the cache read back as
bf16 rows, and decode attention over a cache held in 4-bit floating point
(e2m1 codes, an e4m3 scale per 16 elements, an fp32 scale per kv head).

``run`` computes each in its plain form (elementary torch operations in 32
bits), or, where ``own`` is set, by the library's calls.
"""

import math
import random

import torch

own = False

D = 128
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of a busy server: every row gets one token, a few get a page
        dict(name="tables_decode", op="tables", rows=256, page=16, old_lo=0, old_hi=8192,
             new_lo=1, new_hi=1, lens=1),
        # a chunked-prefill step: ragged chunks, rows without new tokens among them
        dict(name="tables_prefill", op="tables", rows=61, page=64, old_lo=0, old_hi=32768,
             new_lo=0, new_hi=4099, lens=2),
        # one decode step's keys into a bf16 cache: latency counts
        dict(name="append_decode", op="append", kind="bf16", tokens=32, hq=32, hkv=8, page=16,
             axes=1, rot=128, pad=0),
        # an image and text prefill with time / height / width positions, odd length
        dict(name="append_axes3", op="append", kind="bf16", tokens=16381, hq=32, hkv=8, page=16,
             axes=3, rot=128, pad=0),
        # a prefill into e4m3 with per-token scales, half of each head rotated, a padded batch
        dict(name="append_e4m3_token", op="append", kind="e4m3_token", tokens=4099, hq=64, hkv=8,
             page=64, axes=1, rot=64, pad=37),
        # latent rows of a 128-head model: ckv copied, the 64 rope columns rotated
        dict(name="append_latent", op="append", kind="mla", tokens=2048, hq=128, hkv=1, page=64,
             axes=1, rot=64, pad=0),
        # chunked prefill over a 4-bit cache: the chunk appended, then its whole context read back
        dict(name="chunk_fp4", op="chunk", kind="fp4", tokens=4096, context=24581, hq=32, hkv=8,
             page=16, axes=3, rot=128),
        # a 4-bit context read back as bf16 for a dense prefill
        dict(name="gather_fp4", op="gather", kind="fp4", context=65537, hkv=8, page=64),
        # a handful of short rows: latency
        dict(name="fp4_short", op="attend", rows=4, hq=32, hkv=8, page=16, lo=1, hi=700, qlen=1,
             lens=3),
        # an ordinary decode batch, small pages
        dict(name="fp4_paged", op="attend", rows=32, hq=32, hkv=8, page=16, lo=1024, hi=8192,
             qlen=1, lens=4),
        # one long context, contiguous cache
        dict(name="fp4_long", op="attend", rows=1, hq=64, hkv=8, page=0, lo=131072, hi=131072,
             qlen=1, lens=5),
        # speculative decoding: four query tokens a row, ragged rows, larger pages
        dict(name="fp4_spec", op="attend", rows=16, hq=32, hkv=8, page=64, lo=1000, hi=20000,
             qlen=4, lens=6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "chunk", "gather", "attend", "attend"])
    if op == "tables":
        decode = rng.random() < 0.5
        return dict(op=op, rows=_log_int(rng, 1, 1024) if decode else _log_int(rng, 1, 61),
                    page=rng.choice([16, 32, 64, 128]), old_lo=0, old_hi=_log_int(rng, 1, 32768),
                    new_lo=0 if not decode else 1, new_hi=1 if decode else _log_int(rng, 2, 4099),
                    lens=rng.randrange(1 << 20))
    if op == "append":
        kind = rng.choice(["bf16", "e4m3_token", "mla"])
        g, hkv = (rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 4, 8]))
        most = {"bf16": 16381, "e4m3_token": 8192, "mla": 2048}[kind]
        tokens = _log_int(rng, 1, most if g * hkv <= 32 or kind == "mla" else most // 2)
        return dict(op=op, kind=kind, tokens=tokens, hq=128 if kind == "mla" else g * hkv,
                    hkv=1 if kind == "mla" else hkv,
                    page=64 if kind == "mla" else rng.choice([16, 32, 64, 128]),
                    axes=rng.choice([1, 3]), rot=64 if kind == "mla" else rng.choice([64, 96, 128]),
                    pad=rng.randrange(0, tokens // 4 + 1))
    if op == "chunk":
        tokens = _log_int(rng, 1, 4096)
        return dict(op=op, kind="fp4", tokens=tokens, context=tokens + _log_int(rng, 1, 20480),
                    hq=rng.choice([8, 16, 32]), hkv=rng.choice([1, 2, 4, 8]), page=rng.choice([16, 32, 64]),
                    axes=rng.choice([1, 3]), rot=rng.choice([64, 128]))
    if op == "gather":
        return dict(op=op, kind="fp4", context=_log_int(rng, 1, 65537), hkv=rng.choice([1, 2, 4, 8]),
                    page=rng.choice([16, 32, 64, 128]))
    g = rng.choice([1, 2, 4, 6, 8, 16])
    hkv = rng.choice([1, 2, 4, 8])
    q = rng.choice([1, 1, 2, 3, 4])
    q = q if g * q <= 16 else 1
    rows = _log_int(rng, 1, 64)
    most = max(2, min(131072, 140000 * 8 // (rows * hkv)))  # the longest row of all: fp4_paged's work
    hi = _log_int(rng, 2, most)
    return dict(op="attend", rows=rows, hq=g * hkv, hkv=hkv, page=rng.choice([0, 16, 16, 32, 64, 128]),
                lo=hi // rng.choice([1, 2, 8, 1 << 20]), hi=hi, qlen=q, lens=rng.randrange(1 << 20))


def _lens(seed, n, lo, hi):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def _row_lens(c):
    if c["op"] == "tables":
        return (_lens(c["lens"], c["rows"], c["old_lo"], c["old_hi"]),
                _lens(c["lens"] + 7, c["rows"], c["new_lo"], c["new_hi"]))
    return _lens(c["lens"], c["rows"], c["lo"], c["hi"])


def _up(a, b):
    return -(-a // b)


def work(c):
    if c["op"] == "tables":
        old, new = _row_lens(c)
        t = sum(new)
        pages = sum(_up(o + n, c["page"]) - _up(o, c["page"]) for o, n in zip(old, new))
        # lengths in and out, prefix sums, slots (8) and positions (4) of each token, the pages
        # taken from the free list into the table, and each row's page that is part full
        return dict(bytes=float(16 * c["rows"] + 12 * t + 8 * pages + 8), flops=0.0)
    row = 144  # a 4-bit key and value: 64 bytes of codes and 8 of scales each
    if c["op"] == "gather":
        return dict(bytes=float(c["context"] * (8 + c["hkv"] * (row + 4 * D))), flops=0.0)
    if c["op"] in ("append", "chunk"):
        t = c["tokens"] - c.get("pad", 0)
        rope = 4 * c["rot"] + 4 * c["axes"] + 8
        if c["kind"] == "mla":
            per = 2 * (2 * 64 * c["hq"]) + 2 * (2 * 576) + rope
        else:
            per = 2 * (2 * D * c["hq"]) + 4 * D * c["hkv"] + rope
            per += c["hkv"] * {"bf16": 4 * D, "e4m3_token": 2 * D + 8, "fp4": row}[c["kind"]]
        more = 0
        if c["op"] == "chunk":  # rows that the call itself wrote count once
            more = c["context"] * (8 + c["hkv"] * (row + 4 * D)) - t * c["hkv"] * row
        return dict(bytes=float(t * per + more), flops=float(6 * t * c["rot"] * (c["hq"] + c["hkv"])))
    lens = _row_lens(c)
    tokens = sum(lens)
    rows = c["rows"] * c["hq"] * c["qlen"]
    table = sum(_up(n, c["page"]) * 4 for n in lens) if c["page"] else 0
    return dict(bytes=float(tokens * c["hkv"] * row + rows * (4 * D + 4) + table + 4 * c["rows"]),
                flops=float(4 * D * c["hq"] * c["qlen"] * tokens))


# ------------------------------------------------------------------ 4-bit values (plain form)

def _e2m1(a):
    """Codes 0..7 of magnitudes a: to the nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))


def _quantise(x, scale):
    """x fp32 [..., 128] (heads on axis -2) -> codes [..., 64] and scales [..., 8], both bytes."""
    x = x.reshape(*x.shape[:-1], 8, 16)
    s = scale[:, None, None]  # heads on the axis before the blocks
    amax = x.abs().amax(-1, keepdim=True)
    sb = (amax / (6.0 * s)).clamp(max=448.0).to(torch.float8_e4m3fn)
    eff = sb.float() * s
    inv = torch.where(eff > 0, 1.0 / eff, torch.zeros_like(eff))
    y = x * inv
    code = _e2m1(y.abs()) | (torch.signbit(y).to(torch.uint8) << 3)
    code = code.reshape(*code.shape[:-2], 64, 2)
    return code[..., 0] | (code[..., 1] << 4), sb.view(torch.uint8).squeeze(-1)


def _values(codes, scales, scale):
    """Codes [..., 64] and block scales [..., 8] (bytes), heads on axis -2 -> fp32 [..., 128]."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                       device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 8, 16)
    v = lut[c.int()] * scales.view(torch.float8_e4m3fn).float()[..., None]
    return (v * scale[:, None, None]).reshape(*codes.shape[:-1], D)


def _parts(cache):
    """The codes [..., P, 64] and scales [..., P, 8] inside a 4-bit cache [..., P / 16, 1152]."""
    codes = cache[..., :1024].unflatten(-1, (16, 64)).flatten(-3, -2)
    scales = cache[..., 1024:].unflatten(-1, (16, 8)).flatten(-3, -2)
    return codes, scales


def _rows_of(cache, slots, page):
    """Codes [T][HKV][64] and scales [T][HKV][8] of the cache rows `slots` of a paged 4-bit cache."""
    p, o = slots // page, slots % page
    g, r = o // 16, o % 16
    codes = cache[..., :1024].unflatten(-1, (16, 64))
    scales = cache[..., 1024:].unflatten(-1, (16, 8))
    return codes[p, :, g, r], scales[p, :, g, r]


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _kv(g, *shape):
    """Keys or values as a model has them: channels of different sizes, a few large ones."""
    x = torch.randn(shape, generator=g, device=DEV)
    w = torch.exp(0.6 * torch.randn(shape[-1], generator=g, device=DEV))
    return x * w


def _cos_sin(rot, positions):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], -1).float()


def _pair_axis(rot, axes):
    """Which position axis turns each pair: a quarter time, the rest height and width."""
    n = rot // 2
    if axes == 1:
        return [0] * n
    t, h = n // 4, (n - n // 4) // 2
    return [0] * t + [1] * h + [2] * (n - t - h)


def _positions(c, g, first):
    """[axes][tokens]: one running position, or image patches of 24 x 32 frame after frame."""
    i = torch.arange(c["tokens"], device=DEV)
    base = first + int(torch.randint(0, 64, (1,), generator=g, device=DEV))
    if c["axes"] == 1:
        return (base + i)[None].int().contiguous()
    return torch.stack([base + i // 768, base + i // 32 % 24, base + i % 32]).int().contiguous()


def _append_inputs(c, g, s):
    t, hq, hkv = c["tokens"], c["hq"], c["hkv"]
    if c["kind"] == "mla":
        s["q"] = _randn(g, t, hq, 64)
        latent = _randn(g, t, 576)  # the down-projection's output: ckv and kpe side by side
        s["k"], s["v"] = latent[:, :512], latent[:, 512:]
        s["q_out"] = torch.zeros(t, hq, 64, device=DEV, dtype=torch.bfloat16)
    else:
        qkv = _kv(g, t, hq + 2 * hkv, D).to(torch.bfloat16)  # one fused projection's output
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.zeros(t, hq, D, device=DEV, dtype=torch.bfloat16)
    first = c.get("context", t) - t
    s["positions"] = _positions(c, g, first)
    s["cos_sin"] = _cos_sin(c["rot"], first + t + 1024)
    s["pair_axis"] = _pair_axis(c["rot"], c["axes"])


def _slots(c, g, n, pages):
    perm = torch.randperm(pages, generator=g, device=DEV)
    i = torch.arange(n, device=DEV)
    return perm[i // c["page"]] * c["page"] + i % c["page"]


def _engine(c, pages, **more):
    import decode_attention_flash_gb300 as da
    mla = c.get("kind") == "mla"
    kind = {"bf16": da.DA_DTYPE_BF16, "mla": da.DA_DTYPE_BF16,
            "e4m3_token": da.DA_DTYPE_FP8_E4M3_TOKEN_SCALE,
            "fp4": da.DA_DTYPE_FP4_E2M1_BLOCKS}[c.get("kind", "fp4")]
    page = c["page"]
    kw = dict(batch=c.get("rows", 1), num_q_heads=c.get("hq", c.get("hkv", 1)),
              num_kv_heads=c.get("hkv", 1), head_dim_qk=576 if mla else D,
              head_dim_v=512 if mla else D, is_mla=int(mla), ckv_dim=512 if mla else 0,
              kpe_dim=64 if mla else 0, q_dtype=da.DA_DTYPE_BF16, kv_dtype=kind)
    if page:
        kw |= dict(kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=pages,
                   max_pages_per_seq=pages, max_seq_len=pages * page)
    kw.update(more)
    return da, da.DecodeAttention(device=0, **kw)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "tables":
        return _prepare_tables(c, g, s)
    if c["op"] == "attend":
        return _prepare_attend(c, g, s)
    n = c.get("context", c.get("tokens"))
    pages = _up(n, c["page"]) + 64
    if c["op"] in ("append", "chunk"):
        _append_inputs(c, g, s)
    s["slots"] = _slots(c, g, n, pages)
    if c.get("pad"):
        s["slots"][c["tokens"] - c["pad"]:] = -1
    hkv, page = c["hkv"], c["page"]
    if c["kind"] == "bf16":
        for k in ("k_cache", "v_cache"):
            s[k] = torch.zeros(pages, hkv, page, D, device=DEV, dtype=torch.bfloat16)
    elif c["kind"] == "mla":
        s["k_cache"] = torch.zeros(pages, page, 512, device=DEV, dtype=torch.bfloat16)
        s["v_cache"] = torch.zeros(pages, page, 64, device=DEV, dtype=torch.bfloat16)
    elif c["kind"] == "e4m3_token":
        for k in ("k", "v"):
            s[k + "_cache"] = torch.zeros(pages, hkv, page, D, device=DEV, dtype=torch.float8_e4m3fn)
            s[k + "_scale_shift"] = torch.zeros(pages, hkv, page, device=DEV, dtype=torch.int32)
    else:
        for k in ("k", "v"):
            s[k + "_scale"] = torch.rand(hkv, generator=g, device=DEV) * 0.002 + 0.001
            x = _kv(g, pages * (page // 16) * 16, hkv, D)
            codes, scales = _quantise(x, s[k + "_scale"])
            s[k + "_cache"] = _laid_out(codes, scales, pages, hkv, page)
            s[k + "_out"] = torch.zeros(n, hkv, D, device=DEV, dtype=torch.bfloat16)
    if own:
        da, eng = _engine(c, pages)
        s["da"], s["eng"] = da, eng
        kv = {k: s[k + "_cache"] for k in ("k", "v")}
        extra = {k: s[k] for k in ("k_scale", "v_scale", "k_scale_shift", "v_scale_shift") if k in s}
        if c["op"] in ("append", "chunk"):
            t = c["tokens"]
            new = s["slots"][n - t:].contiguous()
            s["new_slots"] = new
            s["append"] = da.make_append_args(
                dict(q=s["q"], k_new=s["k"], v_new=s["v"], q_out=s["q_out"], slot_map=new,
                     positions=s["positions"], cos_sin=s["cos_sin"], **kv, **extra),
                pair_axis=s["pair_axis"])
        if c["op"] in ("gather", "chunk"):
            s["gather"] = da.make_gather_args(dict(slot_map=s["slots"], k_out=s["k_out"],
                                                   v_out=s["v_out"], **kv, **extra))
    return s


def _laid_out(codes, scales, pages, hkv, page):
    """Codes [rows][HKV][64] and scales [rows][HKV][8] of all cache rows as [pages][HKV][P/16][1152]."""
    def order(x):
        return x.reshape(pages, page // 16, 16, hkv, -1).permute(0, 3, 1, 2, 4).flatten(-2)
    return torch.cat([order(codes), order(scales)], -1).contiguous()


def _prepare_tables(c, g, s):
    old, new = _row_lens(c)
    p, b = c["page"], c["rows"]
    have = [_up(o, p) for o in old]
    need = sum(_up(o + n, p) - h for o, n, h in zip(old, new, have))
    cols = max(1, max(_up(o + n, p) for o, n in zip(old, new)))
    pages = sum(have) + need + 64
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    h = torch.tensor(have, device=DEV)
    col = torch.arange(cols, device=DEV)[None]
    at = (h.cumsum(0) - h)[:, None] + col
    s["table"] = torch.where(col < h[:, None], perm[at.clamp(max=pages - 1)], torch.zeros_like(perm[:1]))
    s["free"] = perm[sum(have):].contiguous()
    s["num_free"] = torch.tensor([s["free"].numel()], device=DEV, dtype=torch.int32)
    s["old"] = torch.tensor(old, device=DEV, dtype=torch.int32)
    s["new"] = torch.tensor(new, device=DEV, dtype=torch.int32)
    t = sum(new)
    s["slot_map"] = torch.zeros(t, device=DEV, dtype=torch.int64)
    s["positions"] = torch.zeros(t, device=DEV, dtype=torch.int32)
    s["cu_new"] = torch.zeros(b + 1, device=DEV, dtype=torch.int32)
    s["old_out"] = torch.zeros_like(s["old"])
    s["num_free_out"] = torch.zeros_like(s["num_free"])
    if own:
        da, eng = _engine(dict(c, hkv=1, hq=1), pages, max_pages_per_seq=cols, max_seq_len=cols * p)
        s["da"], s["eng"] = da, eng
        s["tables"] = da.make_table_args(dict(
            seq_lens=s["old"], new_lens=s["new"], block_table=s["table"], free_pages=s["free"],
            num_free=s["num_free"], seq_lens_out=s["old_out"], num_free_out=s["num_free_out"],
            slot_map=s["slot_map"], positions=s["positions"], cu_new=s["cu_new"]))
    return s


def _prepare_attend(c, g, s):
    lens = _row_lens(c)
    b, hq, hkv, q = c["rows"], c["hq"], c["hkv"], c["qlen"]
    s["scale"] = D ** -0.5
    shape = (b, hq, q, D) if q > 1 else (b, hq, D)
    s["q"] = _randn(g, *shape)
    s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    s["out"] = torch.zeros(shape, device=DEV, dtype=torch.bfloat16)
    s["lse"] = torch.zeros(shape[:-1], device=DEV)
    for k in ("k", "v"):
        s[k + "_scale"] = torch.rand(hkv, generator=g, device=DEV) * 0.002 + 0.001
    page = c["page"]
    if page:
        need = [_up(n, page) for n in lens]
        pages, cols = sum(need) + 64, max(need)
        perm = torch.randperm(pages, generator=g, device=DEV).int()
        h = torch.tensor(need, device=DEV)
        col = torch.arange(cols, device=DEV)[None]
        at = (h.cumsum(0) - h)[:, None] + col
        s["table"] = torch.where(col < h[:, None], perm[at.clamp(max=pages - 1)], torch.zeros_like(perm[:1]))
        rows, shape = pages * page, (pages, hkv, page // 16, 1152)
    else:
        length = _up(max(lens), 16) * 16
        pages, rows, shape = 0, b * length, (b, hkv, length // 16, 1152)
    for k in ("k", "v"):
        cache = torch.empty(shape, device=DEV, dtype=torch.uint8)
        step = max(1, (1 << 26) // (hkv * D * shape[2] * 16))
        for i in range(0, shape[0], step):  # a slice of the cache at a time
            n = min(step, shape[0] - i)
            codes, scales = _quantise(_kv(g, n * shape[2] * 16, hkv, D), s[k + "_scale"])
            cache[i:i + n] = _laid_out(codes, scales, n, hkv, shape[2] * 16)
        s[k] = cache
    if own:
        more = dict(q_len=q)
        if page:
            more |= dict(max_pages_per_seq=s["table"].shape[1], max_seq_len=s["table"].shape[1] * page)
        else:
            import decode_attention_flash_gb300 as da
            more |= dict(kv_layout=da.DA_KV_CONTIGUOUS, max_seq_len=length)
        da, eng = _engine(c, pages, seq_lens_host=lens, **more)
        s["da"], s["eng"] = da, eng
        t = dict(q=s["q"], k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                 seq_lens=s["lens"], block_table=s.get("table"))
        s["args"] = da.make_args(t, s["scale"], s["out"], s["lse"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        da, eng = s["da"], s["eng"]
        if op == "tables":
            da.decode_attn_build_tables(eng.ctx, s["tables"], eng.workspace)
            return _tables_out(s, s["table"], s["old_out"], s["num_free_out"], s["slot_map"],
                               s["positions"], s["cu_new"])
        if op == "attend":
            da.decode_attn_run(eng.ctx, s["args"], eng.workspace)
            return dict(out=s["out"], lse=s["lse"])
        if op in ("append", "chunk"):
            da.decode_attn_append(eng.ctx, s["append"], eng.workspace)
        if op in ("gather", "chunk"):
            da.decode_attn_gather(eng.ctx, s["gather"], eng.workspace)
    else:
        if op == "tables":
            return _plain_tables(s)
        if op == "attend":
            return _plain_attend(s)
        if op in ("append", "chunk"):
            _plain_append(s)
        if op in ("gather", "chunk"):
            _plain_gather(s)
    return _cache_out(s)


def _tables_out(s, table, old, free, slots, positions, cu):
    return dict(block_table=table, seq_lens=old, num_free=free, slot_map=slots, positions=positions,
                cu_new=cu)


def _cache_out(s):
    """The rotated queries, and the cache as it was left (4 bits: the rows read back)."""
    op, kind = s["case"]["op"], s["case"]["kind"]
    r = {}
    if op != "gather":
        r["q"] = s["q_out"]
    if kind == "fp4":
        r |= dict(k=s["k_out"], v=s["v_out"])
    else:
        r |= dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if kind == "e4m3_token":  # fp16 scale and shift of each row
        r |= {k: s[k].view(torch.float16) for k in ("k_scale_shift", "v_scale_shift")}
    return r


def _plain_tables(s):
    p, table = s["case"]["page"], s["table"]
    old, new = s["old"].long(), s["new"].long()
    first, last = (old + p - 1) // p, (old + new + p - 1) // p
    need = last - first
    ahead = need.cumsum(0) - need  # pages that earlier rows take
    total = s["num_free"].long()
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    col = torch.arange(table.shape[1], device=DEV)[None]
    taken = (total - 1 - (ahead[:, None] + col - first[:, None])).clamp(0, s["free"].numel() - 1)
    fresh = (col >= first[:, None]) & (col < last[:, None])
    table = torch.where(fresh, s["free"][taken], table)
    n = s["slot_map"].numel()
    row = torch.repeat_interleave(torch.arange(old.numel(), device=DEV), new, output_size=n)
    pos = old[row] + torch.arange(n, device=DEV) - cu[row]
    slots = table[row, pos // p].long() * p + pos % p
    return _tables_out(s, table, (old + new).int(), (total - need.sum()).int(), slots, pos.int(), cu.int())


def _rotate(x, s):
    """x fp32 [T][H][dims]: its first `rot` dims turned by the tokens' angles, rounded to bf16."""
    n = len(s["pair_axis"])
    axis = torch.tensor(s["pair_axis"], device=DEV)
    pair = torch.arange(n, device=DEV)
    pos = s["positions"].long()[axis].T  # [T][pairs]
    c, w = s["cos_sin"][pos, pair][:, None], s["cos_sin"][pos, n + pair][:, None]
    a, b = x[..., :n], x[..., n:2 * n]
    return torch.cat([a * c - b * w, b * c + a * w, x[..., 2 * n:]], -1).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    t, page = c["tokens"], c["page"]
    slots = s["slots"][-t:]
    keep = t - c.get("pad", 0)  # the padding is at the end
    slots = slots[:keep]
    s["q_out"][:keep] = _rotate(s["q"].float(), s)[:keep]
    p, o = slots // page, slots % page
    if c["kind"] == "mla":
        s["k_cache"][p, o] = s["k"][:keep]
        s["v_cache"][p, o] = _rotate(s["v"].float()[:, None], s)[:keep, 0]
        return
    k, v = _rotate(s["k"].float(), s)[:keep], s["v"][:keep]
    if c["kind"] == "bf16":
        s["k_cache"][p, :, o], s["v_cache"][p, :, o] = k, v
    elif c["kind"] == "e4m3_token":
        _put_e4m3_token(s, "k", k.float(), p, o)
        _put_e4m3_token(s, "v", v.float(), p, o)
    else:
        _put_fp4(s, "k", k.float(), p, o)
        _put_fp4(s, "v", v.float(), p, o)


def _put_e4m3_token(s, name, x, p, o):
    hi, lo = x.amax(-1), x.amin(-1)
    shift = ((hi + lo) * 0.5).half()
    scale = ((hi - lo) * 0.5 / 448.0).half()
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    y = ((x - shift.float()[..., None]) / scale.float()[..., None]).clamp(-448, 448)
    s[name + "_cache"].view(torch.uint8)[p, :, o] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    word = scale.view(torch.int16).int() & 0xFFFF | shift.view(torch.int16).int() << 16
    s[name + "_scale_shift"][p, :, o] = word


def _put_fp4(s, name, x, p, o):
    codes, scales = _quantise(x, s[name + "_scale"])
    cache = s[name + "_cache"]
    cache[..., :1024].unflatten(-1, (16, 64))[p, :, o // 16, o % 16] = codes
    cache[..., 1024:].unflatten(-1, (16, 8))[p, :, o // 16, o % 16] = scales


def _plain_gather(s):
    for k in ("k", "v"):
        codes, scales = _rows_of(s[k + "_cache"], s["slots"], s["case"]["page"])
        s[k + "_out"].copy_(_values(codes, scales, s[k + "_scale"]))


def _dense(s, name):
    """The rows' keys or values as fp32 [B][HKV][N][128], N the longest row."""
    c, cache = s["case"], s[name]
    codes, scales = _parts(cache)  # [pages or B][HKV][P or L][..]
    if c["page"]:
        pick = s["table"].long()
        codes = codes[pick].transpose(1, 2).flatten(2, 3)
        scales = scales[pick].transpose(1, 2).flatten(2, 3)
    x = _values(codes.transpose(1, 2), scales.transpose(1, 2), s[name + "_scale"])  # [B][N][HKV][128]
    return x.transpose(1, 2)


def _plain_attend(s):
    c = s["case"]
    b, hq, hkv, q = c["rows"], c["hq"], c["hkv"], c["qlen"]
    k = _dense(s, "k")
    n = k.shape[2]
    x = s["q"].float().reshape(b, hkv, hq // hkv * q, D)
    score = torch.matmul(x, k.transpose(-1, -2)) * s["scale"]
    del k
    score = score.view(b, hkv, hq // hkv, q, n)
    last = s["lens"].long()[:, None] - q + torch.arange(q, device=DEV)  # [B][q]
    seen = torch.arange(n, device=DEV) <= last[..., None]
    score = torch.where(seen[:, None, None], score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, hkv, -1, n), _dense(s, "v")).view(b, hkv, hq // hkv, q, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = top + torch.log(total)
    return dict(out=out.to(torch.bfloat16).view(s["out"].shape), lse=lse.view(s["lse"].shape))


# ------------------------------------------------------------------ 64 bits

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_values(cache, scale):
    """A 4-bit cache [X][HKV][G][1152] as float64 [X][HKV][16 G][128], from the format's definition:
    byte 64 r + j of a granule holds elements 2 j and 2 j + 1 of row r, byte 1024 + 8 r + i the scale of
    elements 16 i .. 16 i + 15."""
    x, h, g, _ = cache.shape
    raw = cache[..., :1024].reshape(x, h, g * 16, 64).long()
    nib = torch.empty(x, h, g * 16, D, device=cache.device, dtype=torch.long)
    nib[..., 0::2] = raw % 16
    nib[..., 1::2] = raw // 16
    grid = torch.tensor(_GRID, device=cache.device, dtype=torch.float64)
    v = grid[nib % 8] * (1 - 2 * (nib // 8)).double()
    e = cache[..., 1024:].reshape(x, h, g * 16, 8).long()
    exp, man = e // 8 % 16, e % 8
    sb = torch.where(exp == 0, man.double() / 8 * 2.0 ** -6, (1 + man.double() / 8) * torch.exp2(exp.double() - 7))
    return v * sb.repeat_interleave(16, -1) * scale.double()[None, :, None, None]


def _exact_fp4(x, scale):
    """What 4 bits keep of float64 x [T][HKV][128]: the block's scale to the nearest e4m3, then each element
    to the nearest of the grid, both ties to even."""
    t, h, _ = x.shape
    b = x.view(t, h, 8, 16)
    want = b.abs().amax(-1) / 6 / scale.double()[None, :, None]
    unit = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
    sb = ((want / unit).round() * unit).clamp(max=448.0)
    eff = (sb * scale.double()[None, :, None])[..., None]
    y = torch.where(eff > 0, b.abs() / torch.where(eff > 0, eff, 1.0), 0.0).clamp(max=6.0)
    unit = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (y / unit).round() * unit
    return (torch.sign(b) * y * eff).view(t, h, D)


def _exact_rotate(x, s):
    n = len(s["pair_axis"])
    y = x.clone()
    for i, a in enumerate(s["pair_axis"]):
        row = s["cos_sin"][s["positions"][a].long()].double()
        c, w = row[:, i, None], row[:, n + i, None]
        y[..., i] = x[..., i] * c - x[..., n + i] * w
        y[..., n + i] = x[..., n + i] * c + x[..., i] * w
    return y


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "tables":
        return None  # whole numbers only
    if c["op"] == "attend":
        return _exact_attend(s)
    r = {}
    if c["op"] in ("append", "chunk"):
        t = c["tokens"]
        keep = t - c.get("pad", 0)
        slots = s["slots"][-t:][:keep]
        p, o = slots // c["page"], slots % c["page"]
        q = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
        q[:keep] = _exact_rotate(s["q"].double(), s)[:keep]
        r["q"] = q
        if c["kind"] == "mla":
            r["k_cache"], r["v_cache"] = s["k_cache"].double(), s["v_cache"].double()
            r["k_cache"][p, o] = s["k"][:keep].double()
            r["v_cache"][p, o] = _exact_rotate(s["v"].double()[:, None], s)[:keep, 0]
            return r
        k, v = _exact_rotate(s["k"].double(), s)[:keep], s["v"].double()[:keep]
        if c["kind"] == "bf16":
            r["k_cache"], r["v_cache"] = s["k_cache"].double(), s["v_cache"].double()
            r["k_cache"][p, :, o], r["v_cache"][p, :, o] = k, v
            return r
        k = k.to(torch.bfloat16).double()  # a quantised cache holds what a bf16 one would, quantised
        if c["kind"] == "e4m3_token":
            for name, x in (("k", k), ("v", v)):
                hi, lo = x.amax(-1), x.amin(-1)
                pair = torch.zeros(s[name + "_scale_shift"].shape + (2,), device=DEV, dtype=torch.float64)
                pair[p, :, o] = torch.stack([(hi - lo) / 896, (hi + lo) / 2], -1)
                r[name + "_scale_shift"] = pair.flatten(-2)
                r[name + "_cache"] = None  # codes follow the rounded scale and shift
            return r
    for name in ("k", "v"):
        x = _exact_values(s[name + "_cache"], s[name + "_scale"])
        x = x.transpose(1, 2).flatten(0, 1)  # [cache rows][HKV][128]
        if c["op"] == "chunk":
            x[slots] = _exact_fp4(k if name == "k" else v, s[name + "_scale"])
        r[name] = x[s["slots"]]
    return r


def _exact_attend(s):
    c = s["case"]
    b, hq, hkv, q, page = c["rows"], c["hq"], c["hkv"], c["qlen"], c["page"]
    out = torch.zeros(b, hq, q, D, device=DEV, dtype=torch.float64)
    lse = torch.full((b, hq, q), -math.inf, device=DEV, dtype=torch.float64)
    x = s["q"].double().view(b, hkv, hq // hkv, q, D)
    for i, n in enumerate(s["lens"].tolist()):
        kv = []
        for name in ("k", "v"):
            if page:
                part = s[name][s["table"][i, :_up(n, page)].long()]
            else:
                part = s[name][i:i + 1]
            rows = _exact_values(part, s[name + "_scale"])
            kv.append(rows.transpose(0, 1).flatten(1, 2)[:, :n])  # [HKV][n][128]
        for t in range(q):
            m = n - q + 1 + t  # positions that query token t sees
            if m <= 0:
                continue
            w = torch.einsum("hgd,hnd->hgn", x[i, :, :, t], kv[0][:, :m]) * s["scale"]
            total = torch.logsumexp(w, -1)
            lse[i, :, t] = total.reshape(-1)
            out[i, :, t] = torch.einsum("hgn,hnd->hgd", torch.exp(w - total[..., None]), kv[1][:, :m]).reshape(hq, D)
    return dict(out=out.view(s["out"].shape), lse=lse.view(s["lse"].shape))
