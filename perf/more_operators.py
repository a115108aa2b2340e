"""Measured cases of the 8-bit block cache, the normed append and the verification of drafts.

What a serving step that drafts tokens adds to the cache calls: queries and keys normed head by
head and turned by their positions on the way into the cache, a cache held in 8 bits (e4m3 or
integers) with one scale for each block of positions and kv head, decode attention over it, its
rows read back as bf16, and drafted tokens verified against the target's probabilities with given
random numbers, the rejected ones taken back from the lengths and their pages from the table.

``run`` computes each in its plain form (elementary torch operations in 32 bits, 64 where sums over
a vocabulary meet a border), or, where ``own`` is set, by the library's calls.
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
        # a handful of short rows over e4m3 blocks of a 16-token page: latency
        dict(name="blocks_short", op="attend", kind="e4m3", rows=4, hq=32, hkv=8, page=16, block=16,
             lo=1, hi=700, qlen=1, lens=3),
        # an ordinary decode batch, small pages, a scale a page
        dict(name="blocks_paged", op="attend", kind="e4m3", rows=32, hq=32, hkv=8, page=16, block=16,
             lo=1024, hi=8192, qlen=1, lens=4),
        # one long context in 8-bit integers, contiguous, wide blocks
        dict(name="blocks_long", op="attend", kind="int8", rows=1, hq=64, hkv=8, page=0, block=128,
             lo=131072, hi=131072, qlen=1, lens=5),
        # speculative decoding: four query tokens a row, ragged rows, larger pages
        dict(name="blocks_spec", op="attend", kind="int8", rows=16, hq=32, hkv=8, page=64, block=64,
             lo=1000, hi=20000, qlen=4, lens=6),
        # one decode step's queries and keys normed, turned and written in bf16: latency counts
        dict(name="norm_decode", op="append", kind="bf16", tokens=32, hq=32, hkv=8, page=16, axes=1,
             rot=128, norm=1),
        # an image and text prefill, three position axes, odd length
        dict(name="norm_prefill", op="append", kind="bf16", tokens=16381, hq=32, hkv=8, page=16, axes=3,
             rot=128, norm=1),
        # latent rows normed as they are cached, the 64 rope columns turned
        dict(name="norm_latent", op="append", kind="mla", tokens=2048, hq=128, hkv=1, page=64, axes=1,
             rot=64, norm=1),
        # one decode step into e4m3 blocks that earlier tokens have part filled
        dict(name="blocks_append", op="append", kind="e4m3", tokens=64, hq=32, hkv=8, page=64, block=64,
             axes=1, rot=128, norm=1, lo=0, hi=2048, lens=8),
        # chunked prefill into integers: the chunk normed and written, its whole context read back
        dict(name="blocks_chunk", op="chunk", kind="int8", tokens=4096, context=24581, hq=32, hkv=8,
             page=64, block=32, axes=1, rot=128, norm=1),
        # a few rows with three drafted tokens each, small vocabulary: latency
        dict(name="verify_short", op="verify", rows=4, q=4, vocab=32000, drafts="probs", ragged=0, page=16,
             near=1.0, lens=9),
        # drafts that a table proposed (no probabilities of their own), an odd vocabulary, ragged
        dict(name="verify_fixed", op="verify", rows=64, q=8, vocab=151937, drafts="fixed", ragged=1, page=16,
             near=0.0, lens=10),
        # a large batch, four drafted tokens a row
        dict(name="verify_batch", op="verify", rows=256, q=5, vocab=128000, drafts="probs", ragged=1, page=64,
             near=0.5, lens=11),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _block(rng, page):
    """A scale's positions: 16, 32, .., 256 that divide the page (0: a contiguous cache)."""
    return rng.choice([b for b in (16, 32, 64, 128, 256) if page == 0 or page % b == 0])


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "chunk", "verify", "verify"])
    seed = rng.randrange(1 << 20)
    if op == "append":
        kind = rng.choice(["bf16", "mla", "e4m3", "e4m3"])
        g, hkv = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 4, 8])
        c = dict(op=op, kind=kind, hq=128 if kind == "mla" else g * hkv, hkv=1 if kind == "mla" else hkv,
                 page=64 if kind == "mla" else rng.choice([16, 32, 64, 128]), axes=rng.choice([1, 3]),
                 rot=64 if kind == "mla" else rng.choice([0, 64, 96, 128]), norm=1)
        if kind == "e4m3":  # a decode step: a token each of some rows
            return c | dict(tokens=_log_int(rng, 1, 256), block=_block(rng, c["page"]), lo=0,
                            hi=_log_int(rng, 1, 2048), lens=seed)
        most = 2048 if kind == "mla" else 16381 if g * hkv <= 32 else 8192
        return c | dict(tokens=_log_int(rng, 1, most))
    if op == "chunk":
        tokens, page = _log_int(rng, 1, 4096), rng.choice([16, 32, 64, 128])
        return dict(op=op, kind=rng.choice(["int8", "e4m3"]), tokens=tokens,
                    context=tokens + _log_int(rng, 1, 20480), hq=rng.choice([8, 16, 32]),
                    hkv=rng.choice([1, 2, 4, 8]), page=page, block=_block(rng, page), axes=rng.choice([1, 3]),
                    rot=rng.choice([64, 128]), norm=1)
    if op == "verify":
        q, vocab = rng.randint(1, 8), _log_int(rng, 1000, 160000)
        rows = _log_int(rng, 1, max(1, min(256, 256 * 5 * 128000 // (q * vocab))))
        return dict(op=op, rows=rows, q=q, vocab=vocab, drafts=rng.choice(["probs", "probs", "fixed"]),
                    ragged=rng.randrange(2), page=rng.choice([16, 64]), near=rng.choice([0.0, 0.3, 1.0, 3.0]),
                    lens=seed)
    g = rng.choice([1, 2, 4, 6, 8, 16])
    hkv = rng.choice([1, 2, 4, 8])
    q = rng.choice([1, 1, 2, 3, 4])
    q = q if g * q <= 16 else 1
    rows = _log_int(rng, 1, 64)
    most = max(2, min(131072, 140000 * 8 // (rows * hkv)))
    hi = _log_int(rng, 2, most)
    page = rng.choice([0, 16, 16, 32, 64, 128])
    return dict(op="attend", kind=rng.choice(["e4m3", "int8"]), rows=rows, hq=g * hkv, hkv=hkv, page=page,
                block=_block(rng, page), lo=hi // rng.choice([1, 2, 8, 1 << 20]), hi=hi, qlen=q, lens=seed)


def _lens(seed, n, lo, hi):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def _row_lens(c):
    return _lens(c["lens"], c["rows"] if c["op"] == "attend" else c["tokens"], c["lo"], c["hi"])


def _drafts(c):
    """How many drafted tokens each row has."""
    n = c["q"] - 1
    return _lens(c["lens"], c["rows"], 0, n) if c["ragged"] else [n] * c["rows"]


def _up(a, b):
    return -(-a // b)


def work(c):
    if c["op"] == "verify":
        # a probability of target and draft for each drafted token, and one distribution of each a row
        # (a row may accept every token and then needs no draft's: that follows from the inputs)
        n = sum(_drafts(c))
        per = 2 if c["drafts"] == "probs" else 1
        return dict(bytes=float(per * 4 * c["rows"] * c["vocab"] + 4 * n * (2 + per) + 8 * c["rows"] * (4 + c["q"])),
                    flops=float(per * c["rows"] * c["vocab"]))
    if c["op"] == "attend":
        lens = _row_lens(c)
        tokens, rows = sum(lens), c["rows"] * c["hq"] * c["qlen"]
        table = sum(_up(n, c["page"]) * 4 for n in lens) if c["page"] else 0
        scales = sum(_up(n, c["block"]) for n in lens) * c["hkv"] * 8
        return dict(bytes=float(tokens * c["hkv"] * 2 * D + scales + rows * (4 * D + 4) + table + 4 * c["rows"]),
                    flops=float(4 * D * c["hq"] * c["qlen"] * tokens))
    t = c["tokens"]
    rope = 4 * c["rot"] + 4 * c["axes"] + 8
    if c["kind"] == "mla":
        per = 2 * (2 * 64 * c["hq"]) + 2 * (2 * 576) + rope
    else:
        per = 2 * (2 * D * c["hq"]) + 4 * D * c["hkv"] + rope
        per += c["hkv"] * (4 * D if c["kind"] == "bf16" else 2 * D)
    more = 0
    if "block" in c:  # the scales of the blocks that get tokens
        blocks = t if c["op"] == "append" else _up(t, c["block"])
        more += blocks * c["hkv"] * 16
    if c["op"] == "chunk":  # rows that the call itself wrote count once
        more += c["context"] * (8 + c["hkv"] * 2 * (D + 2 * D)) - t * c["hkv"] * 2 * D
    heads = c["hq"] + c["hkv"] if c["kind"] != "mla" else 8
    return dict(bytes=float(t * per + more), flops=float(t * (6 * c["rot"] * (c["hq"] + c["hkv"]) + 4 * D * heads)))


# ------------------------------------------------------------------ 8-bit blocks (plain form)

DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def _to_codes(y, kind):
    """Quotients of fp32 as codes, to nearest even."""
    if kind == "int8":
        return y.round().clamp(-127, 127).to(torch.int8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn)


def _least_scale(amax, kind):
    """The least power of two that brings amax into the codes' range (0 for 0)."""
    frac, exp = torch.frexp(amax)  # amax = frac 2^exp, frac in [0.5, 1)
    most, at = (0.9921875, 7) if kind == "int8" else (0.875, 9)  # 127 and 448
    exp = (exp - at + (frac > most).int()).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), exp), torch.zeros_like(amax))


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _kv(g, *shape):
    """Keys or values as a model has them: channels of different sizes, a few large ones."""
    x = torch.randn(shape, generator=g, device=DEV)
    return x * torch.exp(0.6 * torch.randn(shape[-1], generator=g, device=DEV))


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
    """[axes][tokens]: running positions, or image patches of 24 x 32 frame after frame."""
    i = torch.arange(c["tokens"], device=DEV)
    base = first + int(torch.randint(0, 64, (1,), generator=g, device=DEV))
    if c["axes"] == 1:
        return (base + i)[None].int().contiguous()
    return torch.stack([base + i // 768, base + i // 32 % 24, base + i % 32]).int().contiguous()


def _weights(g, n):
    """Norm weights as trained ones are: around one, a few small."""
    return torch.exp(0.3 * torch.randn(n, generator=g, device=DEV))


def _append_inputs(c, g, s):
    t, hq, hkv = c["tokens"], c["hq"], c["hkv"]
    if c["kind"] == "mla":
        s["q"] = _randn(g, t, hq, 64)
        latent = _randn(g, t, 576)  # the down-projection's output: ckv and kpe side by side
        s["k"], s["v"] = latent[:, :512], latent[:, 512:]
        s["k_weight"] = _weights(g, 512)
    else:
        qkv = _kv(g, t, hq + 2 * hkv, D).to(torch.bfloat16)  # one fused projection's output
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_weight"], s["k_weight"] = _weights(g, D), _weights(g, D)
    s["q_out"] = torch.zeros(s["q"].shape, device=DEV, dtype=torch.bfloat16)
    s["eps"] = 1e-6
    first = c.get("context", t) - t
    s["positions"] = _positions(c, g, first)
    if c["rot"]:
        s["cos_sin"] = _cos_sin(c["rot"], first + t + 1024)
    s["pair_axis"] = _pair_axis(c["rot"], c["axes"])


def _fill_blocks(c, g, s, name, pages, powers):
    """A paged cache whose blocks hold quantised rows. `powers`: scales as the append makes them."""
    hkv, page, block, kind = c["hkv"], c["page"], c["block"], c["kind"]
    cache = torch.empty(pages, hkv, page, D, device=DEV, dtype=DTYPE[kind])
    scale = torch.empty(pages, hkv, page // block, device=DEV)
    step = max(1, (1 << 26) // (hkv * D * page))
    for i in range(0, pages, step):  # a slice of the cache at a time
        n = min(step, pages - i)
        x = _kv(g, n, hkv, page // block, block, D)
        if powers:
            x = x.bfloat16().float()
        amax = x.abs().amax((-2, -1))
        sc = _least_scale(amax, kind) if powers else amax / (127.0 if kind == "int8" else 448.0)
        cache[i:i + n] = _to_codes(x / sc[..., None, None], kind).reshape(n, hkv, page, D)
        scale[i:i + n] = sc
    s[name], s[name + "_scale"] = cache, scale


def _engine(c, pages, **more):
    import decode_attention_flash_gb300 as da
    mla = c.get("kind") == "mla"
    kind = {"bf16": da.DA_DTYPE_BF16, "mla": da.DA_DTYPE_BF16, "e4m3": da.DA_DTYPE_FP8_E4M3_BLOCKS,
            "int8": da.DA_DTYPE_INT8_BLOCKS}[c.get("kind", "bf16")]
    page = c["page"]
    kw = dict(batch=c.get("rows", 1), num_q_heads=c.get("hq", 1), num_kv_heads=c.get("hkv", 1),
              head_dim_qk=576 if mla else D, head_dim_v=512 if mla else D, is_mla=int(mla),
              ckv_dim=512 if mla else 0, kpe_dim=64 if mla else 0, q_dtype=da.DA_DTYPE_BF16, kv_dtype=kind,
              kv_groups=c.get("block", 0))
    if page:
        kw |= dict(kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=pages, max_pages_per_seq=pages,
                   max_seq_len=pages * page)
    kw.update(more)
    return da, da.DecodeAttention(device=0, **kw)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "verify":
        return _prepare_verify(c, g, s)
    if c["op"] == "attend":
        return _prepare_attend(c, g, s)
    page, t = c["page"], c["tokens"]
    _append_inputs(c, g, s)
    if "lo" in c:  # a token each of rows of different lengths, at their ends
        old = _row_lens(c)
        need = [o // page + 1 for o in old]
        pages = sum(need) + 16
        perm = torch.randperm(pages, generator=g, device=DEV)
        last = torch.tensor(need, device=DEV).cumsum(0) - 1
        o = torch.tensor(old, device=DEV)
        s["slots"] = perm[last] * page + o % page
        s["positions"] = o[None].int().repeat(c["axes"], 1).contiguous()
        if c["rot"]:
            s["cos_sin"] = _cos_sin(c["rot"], c["hi"] + 1)
    else:
        n = c.get("context", t)
        pages = _up(n, page) + 16
        perm = torch.randperm(pages, generator=g, device=DEV)
        i = torch.arange(n, device=DEV)
        s["slots"] = perm[i // page] * page + i % page
    hkv = c["hkv"]
    if c["kind"] == "bf16":
        for k in ("k_cache", "v_cache"):
            s[k] = torch.zeros(pages, hkv, page, D, device=DEV, dtype=torch.bfloat16)
    elif c["kind"] == "mla":
        s["k_cache"] = torch.zeros(pages, page, 512, device=DEV, dtype=torch.bfloat16)
        s["v_cache"] = torch.zeros(pages, page, 64, device=DEV, dtype=torch.bfloat16)
    else:
        for k in ("k_cache", "v_cache"):
            _fill_blocks(c, g, s, k, pages, True)
    if c["op"] == "chunk":
        for k in ("k_out", "v_out"):
            s[k] = torch.zeros(c["context"], hkv, D, device=DEV, dtype=torch.bfloat16)
    s["new_slots"] = s["slots"][-t:].contiguous()
    if own:
        da, eng = _engine(c, pages)
        s["da"], s["eng"] = da, eng
        cache = dict(k=s["k_cache"], v=s["v_cache"])
        if "block" in c:
            cache |= dict(k_scale=s["k_cache_scale"], v_scale=s["v_cache_scale"])
        s["append"] = da.make_append_args(
            dict(q=s["q"], k_new=s["k"], v_new=s["v"], q_out=s["q_out"], slot_map=s["new_slots"],
                 positions=s["positions"], cos_sin=s.get("cos_sin"), **cache),
            pair_axis=s["pair_axis"] if c["rot"] else None)
        s["norm"] = da.make_norm_args(dict(q_weight=s.get("q_weight"), k_weight=s["k_weight"]), eps=s["eps"])
        if c["op"] == "chunk":
            s["gather"] = da.make_gather_args(dict(slot_map=s["slots"], k_out=s["k_out"], v_out=s["v_out"], **cache))
    return s


def _table(c, g, lens):
    """A block table [rows][columns] of rows of `lens` positions, in pages from all over the pool."""
    need = [_up(n, c["page"]) for n in lens]
    pages, cols = sum(need) + 64, max(1, max(need))
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    h = torch.tensor(need, device=DEV)
    col = torch.arange(cols, device=DEV)[None]
    at = (h.cumsum(0) - h)[:, None] + col
    return torch.where(col < h[:, None], perm[at.clamp(max=pages - 1)], torch.zeros_like(perm[:1])), perm, sum(need)


def _prepare_attend(c, g, s):
    lens = _row_lens(c)
    b, hq, hkv, q, page = c["rows"], c["hq"], c["hkv"], c["qlen"], c["page"]
    s["scale"] = D ** -0.5
    shape = (b, hq, q, D) if q > 1 else (b, hq, D)
    s["q"] = _randn(g, *shape)
    s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    s["out"] = torch.zeros(shape, device=DEV, dtype=torch.bfloat16)
    s["lse"] = torch.zeros(shape[:-1], device=DEV)
    if page:
        s["table"], perm, _ = _table(c, g, lens)
        pages = perm.numel()
        for k in ("k", "v"):
            _fill_blocks(c, g, s, k, pages, False)
    else:
        length = _up(max(lens), 256) * 256
        for k in ("k", "v"):
            _fill_blocks(dict(c, page=length), g, s, k, b, False)
        pages = 0
    if own:
        import decode_attention_flash_gb300 as da
        more = dict(q_len=q, seq_lens_host=lens)
        if page:
            more |= dict(max_pages_per_seq=s["table"].shape[1], max_seq_len=s["table"].shape[1] * page)
        else:
            more |= dict(kv_layout=da.DA_KV_CONTIGUOUS, max_seq_len=length)
        da, eng = _engine(c, pages, **more)
        s["da"], s["eng"] = da, eng
        t = {k: s.get(k) for k in ("q", "k", "v", "k_scale", "v_scale")}
        s["args"] = da.make_args(t | dict(seq_lens=s["lens"], block_table=s.get("table")), s["scale"], s["out"],
                                 s["lse"])
    return s


def _prepare_verify(c, g, s):
    b, q, v, page = c["rows"], c["q"], c["vocab"], c["page"]
    n = q - 1
    num = _drafts(c)
    s["num_draft"] = torch.tensor(num, device=DEV, dtype=torch.int32)
    s["target"] = torch.empty(b, q, v, device=DEV)
    fixed = c["drafts"] == "fixed"
    s["draft"] = None if fixed else torch.empty(b, n, v, device=DEV)
    s["tokens"] = torch.zeros(b, n, device=DEV, dtype=torch.int32)
    for i in range(q):
        for at in range(0, b, 32):  # logits with a heavy head, some tokens cut off
            m = min(32, b - at)
            x = 3.0 * torch.randn(m, v, generator=g, device=DEV)
            p = torch.softmax(torch.where(x > -4.0, x, -math.inf), -1)
            s["target"][at:at + m, i] = p
            if i == n:
                continue
            # the draft's distribution: the target's logits, further off the larger `near` is
            y = x + c["near"] * torch.randn(m, v, generator=g, device=DEV)
            d = torch.softmax(y, -1)
            if not fixed:
                s["draft"][at:at + m, i] = d
            noise = torch.rand(m, v, generator=g, device=DEV).clamp(min=1e-30)
            s["tokens"][at:at + m, i] = (noise.log() / d.clamp(min=1e-38)).argmax(-1).int()
    s["uniforms"] = torch.rand(b, q, generator=g, device=DEV)
    # the rows' lengths with the query tokens in, and the pages they hold
    lens = _lens(c["lens"] + 1, b, q, 2000)
    s["table"], perm, used = _table(c, g, lens)
    s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    s["free"] = torch.cat([perm[used:], torch.zeros(used, device=DEV, dtype=torch.int32)])
    s["num_free"] = torch.tensor([perm.numel() - used], device=DEV, dtype=torch.int32)
    s["tokens_out"] = torch.zeros(b, q, device=DEV, dtype=torch.int32)
    s["num_accepted"] = torch.zeros(b, device=DEV, dtype=torch.int32)
    s["lens_out"] = torch.zeros_like(s["lens"])
    s["num_free_out"] = torch.zeros_like(s["num_free"])
    if own:
        cols = s["table"].shape[1]
        da, eng = _engine(c, perm.numel(), max_pages_per_seq=cols, max_seq_len=cols * page)
        s["da"], s["eng"] = da, eng
        s["verify"] = da.make_verify_args(dict(
            target_probs=s["target"], draft_probs=s["draft"], draft_tokens=s["tokens"], num_draft=s["num_draft"],
            uniforms=s["uniforms"], tokens_out=s["tokens_out"], num_accepted=s["num_accepted"],
            seq_lens=s["lens"], seq_lens_out=s["lens_out"], block_table=s["table"], free_pages=s["free"],
            num_free=s["num_free"], num_free_out=s["num_free_out"]))
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        da, eng = s["da"], s["eng"]
        if op == "verify":
            da.decode_attn_verify(eng.ctx, s["verify"], eng.workspace)
            return _verify_out(s)
        if op == "attend":
            da.decode_attn_run(eng.ctx, s["args"], eng.workspace)
            return dict(out=s["out"], lse=s["lse"])
        da.decode_attn_append_normed(eng.ctx, s["append"], s["norm"], eng.workspace)
        if op == "chunk":
            da.decode_attn_gather(eng.ctx, s["gather"], eng.workspace)
    else:
        if op == "verify":
            _plain_verify(s)
            return _verify_out(s)
        if op == "attend":
            return _plain_attend(s)
        _plain_append(s)
        if op == "chunk":
            _plain_gather(s)
    return _cache_out(s)


def _verify_out(s):
    return dict(tokens=s["tokens_out"], num_accepted=s["num_accepted"], seq_lens=s["lens_out"],
                free_pages=s["free"], num_free=s["num_free_out"])


def _cache_out(s):
    """The queries, and the cache as it was left (after a chunk: the context's rows read back)."""
    r = dict(q=s["q_out"])
    if s["case"]["op"] == "chunk":
        return r | dict(k=s["k_out"], v=s["v_out"])
    r |= dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if "block" in s["case"]:
        r |= dict(k_scale=s["k_cache_scale"], v_scale=s["v_cache_scale"])
    return r


def _normed(x, w, eps):
    """x fp32 [..., n] over its root mean square, times w."""
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def _rotate(x, s):
    """x fp32 [T][H][dims]: its first `rot` dims turned by the tokens' angles, rounded to bf16."""
    n = len(s["pair_axis"])
    if n == 0:
        return x.to(torch.bfloat16)
    axis = torch.tensor(s["pair_axis"], device=DEV)
    pair = torch.arange(n, device=DEV)
    pos = s["positions"].long()[axis].T  # [T][pairs]
    c, w = s["cos_sin"][pos, pair][:, None], s["cos_sin"][pos, n + pair][:, None]
    a, b = x[..., :n], x[..., n:2 * n]
    return torch.cat([a * c - b * w, b * c + a * w, x[..., 2 * n:]], -1).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    page, slots = c["page"], s["new_slots"]
    p, o = slots // page, slots % page
    s["q_out"].copy_(_rotate(_normed(s["q"].float(), s.get("q_weight"), s["eps"]), s))
    if c["kind"] == "mla":
        s["k_cache"][p, o] = _normed(s["k"].float(), s["k_weight"], s["eps"]).to(torch.bfloat16)
        s["v_cache"][p, o] = _rotate(s["v"].float()[:, None], s)[:, 0]
        return
    k = _rotate(_normed(s["k"].float(), s["k_weight"], s["eps"]), s)
    if c["kind"] == "bf16":
        s["k_cache"][p, :, o], s["v_cache"][p, :, o] = k, s["v"]
    else:
        _put_blocks(s, "k_cache", k.float(), p, o)
        _put_blocks(s, "v_cache", s["v"].float(), p, o)


def _put_blocks(s, name, x, p, o):
    """x [T][HKV][128] at (page, offset): a block's scale is the least power of two that holds its tokens,
    or the one it has where that is more (a token in a block's first row starts it anew); rows that
    stay are rounded again where it grew."""
    c = s["case"]
    kind, page, block, hkv = c["kind"], c["page"], c["block"], c["hkv"]
    cache, scale = s[name], s[name + "_scale"]
    pages, per = cache.shape[0], page // block
    at = (p * per + o // block)[:, None].expand(-1, hkv)  # the token's block
    amax = torch.zeros(pages * per, hkv, device=DEV).scatter_reduce(0, at, x.abs().amax(-1), "amax")
    fresh = torch.zeros(pages * per, device=DEV).scatter_reduce(0, at[:, 0], (o % block == 0).float(), "amax") > 0
    new = _least_scale(amax, kind).view(pages, per, hkv).transpose(1, 2)
    fresh = fresh.view(pages, 1, per)
    was = torch.where(fresh, torch.zeros_like(scale), scale)
    grown = torch.maximum(was, new)
    keep = ~fresh & (grown > scale)
    ratio = torch.where(keep, scale * (1.0 / grown), torch.ones_like(scale))
    rows = cache.view(pages, hkv, per, block, D)
    rows.copy_(_to_codes(rows.float() * ratio[..., None, None], kind))
    touched = torch.zeros(pages * per, device=DEV, dtype=torch.bool)
    touched[at[:, 0]] = True
    scale.copy_(torch.where(touched.view(pages, 1, per), grown, scale))
    mine = scale[p, :, o // block]  # [T][HKV]
    inv = torch.where(mine > 0, 1.0 / mine, torch.zeros_like(mine))
    raw = _to_codes(x * inv[..., None], kind)
    cache.view(torch.uint8)[p, :, o] = raw.view(torch.uint8)


def _plain_gather(s):
    c = s["case"]
    p, o = s["slots"] // c["page"], s["slots"] % c["page"]
    for k in ("k", "v"):
        rows = s[k + "_cache"].view(torch.uint8)[p, :, o].view(DTYPE[c["kind"]]).float()
        s[k + "_out"].copy_(rows * s[k + "_cache_scale"][p, :, o // c["block"]][..., None])


def _dense(s, name):
    """The rows' keys or values as fp32 [B][HKV][N][128], N the longest row."""
    c, cache, scale = s["case"], s[name], s[name + "_scale"]
    if c["page"]:
        pick = s["table"].long()
        cache = cache.view(torch.uint8)[pick].view(DTYPE[c["kind"]]).transpose(1, 2).flatten(2, 3)
        scale = scale[pick].transpose(1, 2).flatten(2, 3)
    b, h, n, _ = cache.shape
    x = cache.float().view(b, h, n // c["block"], c["block"], D) * scale[..., None, None]
    return x.view(b, h, n, D)


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


def _plain_verify(s):
    c, target, draft = s["case"], s["target"], s["draft"]
    b, q, page = c["rows"], c["q"], c["page"]
    n, num = q - 1, s["num_draft"].long()
    row = torch.arange(b, device=DEV)
    tok, u = s["tokens"].long(), s["uniforms"]
    if n:
        i = torch.arange(n, device=DEV)
        pt = target[row[:, None], i, tok].double()
        pd = draft[row[:, None], i, tok].double() if draft is not None else torch.ones_like(pt)
        ok = (u[:, :n].double() * pd < pt) & (i < num[:, None])
        kept = ok.int().cumprod(-1).sum(-1)  # drafted tokens up to the first rejected one
    else:
        kept = torch.zeros_like(num)
    # the next token: of max(target - draft, 0) where one was rejected, else of the target
    w = target[row, kept].double()
    if n:
        rejected = (kept < num)[:, None]
        at = kept.clamp(max=n - 1)
        if draft is not None:
            less = draft[row, at].double()
        else:
            less = (torch.arange(c["vocab"], device=DEV) == tok[row, at][:, None]).double()
        rest = (w - less).clamp(min=0)
        rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w)
        w = torch.where(rejected, rest, w)
    cum = w.cumsum(-1)
    pick = (cum <= u[:, n:].double() * cum[:, -1:]).sum(-1)  # the first whose sum passes the number
    j = torch.arange(q, device=DEV)
    out = torch.cat([tok, pick[:, None]], -1)
    out = torch.where(j < kept[:, None], out, torch.where(j == kept[:, None], pick[:, None], -1))
    s["tokens_out"].copy_(out)
    s["num_accepted"].copy_(kept)
    lens = s["lens"].long()
    short = lens - (num - kept)
    s["lens_out"].copy_(short)
    # pages that only rejected tokens had go back: the last row's first, each row's from its end
    old, new = (lens + page - 1) // page, (short + page - 1) // page
    give = (old - new).flip(0)
    ahead = (give.cumsum(0) - give).flip(0)
    most = _up(n, page) + 1
    k = torch.arange(most, device=DEV)
    col = (old[:, None] - 1 - k).clamp(min=0)
    on = k < (old - new)[:, None]
    pos = torch.where(on, s["num_free"].long() + ahead[:, None] + k, s["free"].numel())
    spare = torch.cat([s["free"], s["free"][:1]])
    spare[pos] = s["table"][row[:, None], col]
    s["free"].copy_(spare[:-1])
    s["num_free_out"].copy_(s["num_free"] + (old - new).sum())


# ------------------------------------------------------------------ 64 bits

def _exact_rows(cache, scale, block):
    """A block cache [X][HKV][N][128] as float64, a position times its block's scale."""
    return cache.double() * scale.double().repeat_interleave(block, -1)[..., None]


def _exact_turn(x, w, s):
    """x [T][H][n]: normed by w where it is given, then its pairs turned."""
    if w is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w.double()
    n = len(s["pair_axis"])
    y = x.clone()
    for i, a in enumerate(s["pair_axis"]):
        row = s["cos_sin"][s["positions"][a].long()].double()
        c, t = row[:, i, None], row[:, n + i, None]
        y[..., i] = x[..., i] * c - x[..., n + i] * t
        y[..., n + i] = x[..., n + i] * c + x[..., i] * t
    return y


def _exact_blocks(c, cache, scale, x, slots):
    """Scales and values of a block cache after x [T][HKV][128] float64 went to `slots`, block by block."""
    page, block, kind = c["page"], c["block"], c["kind"]
    values = _exact_rows(cache, scale, block)
    scale = scale.double().clone()
    most = 127.0 if kind == "int8" else 448.0

    def rounded(v, sc):
        y = v / sc
        if kind == "int8":
            return y.round().clamp(-127, 127) * sc
        unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return (y / unit).round().mul(unit).clamp(-most, most) * sc

    spots = {}
    for i, slot in enumerate(slots.tolist()):
        spots.setdefault((slot // page, slot % page // block), []).append((slot % block, i))
    for (p, j), at in spots.items():
        offs = torch.tensor([o for o, _ in at], device=DEV)
        new = x[torch.tensor([i for _, i in at], device=DEV)]  # [n][HKV][128]
        amax = new.abs().amax((0, -1))
        need = torch.exp2(torch.ceil(torch.log2(amax / most)))
        old = scale[p, :, j]
        part = values[p, :, j * block:(j + 1) * block]
        if any(o == 0 for o, _ in at):  # its other rows keep their codes, whatever those now stand for
            sc = need
            part = part / old[:, None, None] * sc[:, None, None]
        else:
            sc = torch.maximum(old, need)
            part = torch.where((sc > old)[:, None, None], rounded(part, sc[:, None, None]), part)
        part[:, offs] = rounded(new.transpose(0, 1), sc[:, None, None])
        values[p, :, j * block:(j + 1) * block] = part
        scale[p, :, j] = sc
    return values, scale


def exact(case, seed):
    c = case
    if c["op"] == "verify":
        return None  # whole numbers only
    s = prepare(case, seed)
    if c["op"] == "attend":
        return _exact_attend(s)
    page, slots = c["page"], s["new_slots"]
    p, o = slots // page, slots % page
    r = dict(q=_exact_turn(s["q"].double(), s.get("q_weight"), s))
    k_cache, v_cache = s["k_cache"], s["v_cache"]
    if c["kind"] == "mla":
        k, v = k_cache.double(), v_cache.double()
        x = s["k"].double()
        k[p, o] = x / (x.square().mean(-1, keepdim=True) + s["eps"]).sqrt() * s["k_weight"].double()
        v[p, o] = _exact_turn(s["v"].double()[:, None], None, s)[:, 0]
        return r | dict(k_cache=k, v_cache=v)
    new = dict(k=_exact_turn(s["k"].double(), s["k_weight"], s), v=s["v"].double())
    if c["kind"] == "bf16":
        k, v = k_cache.double(), v_cache.double()
        k[p, :, o], v[p, :, o] = new["k"], new["v"]
        return r | dict(k_cache=k, v_cache=v)
    new["k"] = new["k"].to(torch.bfloat16).double()  # a quantised cache holds what a bf16 one would, quantised
    for name in ("k", "v"):
        values, scale = _exact_blocks(c, s[name + "_cache"], s[name + "_cache_scale"], new[name], slots)
        if c["op"] == "chunk":
            at, off = s["slots"] // page, s["slots"] % page
            r[name] = values[at, :, off]
        else:  # codes: the values over their blocks' scales
            r[name + "_cache"] = values / scale.repeat_interleave(c["block"], -1)[..., None]
            r[name + "_scale"] = scale
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
            at = s["table"][i, :_up(n, page)].long() if page else slice(i, i + 1)
            raw = s[name].view(torch.uint8)[at].view(DTYPE[c["kind"]])
            rows = _exact_rows(raw, s[name + "_scale"][at], c["block"])
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
