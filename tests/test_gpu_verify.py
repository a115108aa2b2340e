"""Drafted tokens verified on the GPU (decode_attn_verify), against the definition in 64 bits on the
host. Outputs are whole numbers and are compared as such: the kernel's sums are good to 2^-40, and the
random inputs here leave no border nearer than that; exact ties are cases of their own, in numbers whose
sums are exact."""

import pytest
import torch

import decode_attention_flash_gb300 as da

pytestmark = pytest.mark.gpu


def engine(batch, *, page=16, cols=64, pages=4096, length=0):
    kw = dict(batch=batch, num_q_heads=1, num_kv_heads=1, head_dim_qk=128, head_dim_v=128)
    if page:
        kw |= dict(kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=pages, max_pages_per_seq=cols, max_seq_len=cols * page)
    else:
        kw |= dict(kv_layout=da.DA_KV_CONTIGUOUS, max_seq_len=length)
    return da.DecodeAttention(device=0, **kw)


def draw(w, r):
    """The first token whose running sum passes r times the sum; None: no weight at all."""
    w = torch.where(w > 0, w, 0.0)
    cum = w.cumsum(0)
    if not cum[-1] > 0:
        return None
    return int((cum <= float(r) * cum[-1]).sum())


def reference(t):
    """Tokens and accepted counts from the tensors of a call, in 64 bits."""
    greedy = t.get("target_tokens")
    first = t["target_probs"] if greedy is None else greedy
    b, q = first.shape[:2]
    out, kept = torch.full((b, q), -1), torch.zeros(b, dtype=torch.long)
    vocab = first.shape[2] if greedy is None else 1 << 21
    for i in range(b):
        n = q - 1 if t.get("num_draft") is None else min(int(t["num_draft"][i]), q - 1)
        if n < 0:
            continue
        a, rejected = 0, False
        while a < n:
            x = int(t["draft_tokens"][i, a])
            if not 0 <= x < vocab:
                break
            if greedy is not None:
                ok = int(greedy[i, a]) == x
            else:
                d = float(t["draft_probs"][i, a, x]) if t.get("draft_probs") is not None else 1.0
                ok = float(t["uniforms"][i, a]) * d < float(t["target_probs"][i, a, x])
            if not ok:
                rejected = True
                break
            a += 1
        kept[i] = a
        out[i, :a] = t["draft_tokens"][i, :a]
        if greedy is not None:
            out[i, a] = greedy[i, a]
            continue
        p, r = t["target_probs"][i, a].double(), t["uniforms"][i, q - 1]
        got = None
        if rejected:
            less = t["draft_probs"][i, a].double() if t.get("draft_probs") is not None else torch.zeros(vocab, dtype=torch.float64)
            if t.get("draft_probs") is None:
                less[int(t["draft_tokens"][i, a])] = 1.0
            got = draw(p - less, r)
        if got is None:
            got = draw(p, r)
        out[i, a] = -1 if got is None else got
    return out, kept


def run(eng, t, **more):
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) and not v.is_cuda else v) for k, v in (t | more).items()}
    first = dev["target_probs"] if dev.get("target_probs") is not None else dev["target_tokens"]
    b, q = first.shape[:2]
    dev.setdefault("tokens_out", torch.full((b, q), 99, dtype=torch.int32, device="cuda"))
    dev.setdefault("num_accepted", torch.full((b,), 99, dtype=torch.int32, device="cuda"))
    eng.verify(dev)
    torch.cuda.synchronize()
    return dev


def check(t, flags=0, eng=None, **more):
    b = (t.get("target_probs") if t.get("target_probs") is not None else t["target_tokens"]).shape[0]
    eng = eng or engine(b)
    dev = run(eng, t, **more)
    assert eng.errors() == flags
    out, kept = reference(t)
    assert torch.equal(dev["num_accepted"].cpu().long(), kept)
    assert torch.equal(dev["tokens_out"].cpu().long(), out), (dev["tokens_out"].cpu().long() != out).nonzero()[:5]
    return dev, kept


def make(b, q, vocab, drafts="probs", near=1.0, ragged=False, seed=0, sharp=3.0):
    gen = torch.Generator().manual_seed(seed)
    x = sharp * torch.randn(b, q, vocab, generator=gen)
    p = torch.softmax(torch.where(x > -sharp, x, -float("inf")), -1)
    p = torch.where(torch.isnan(p), 1.0 / vocab, p)
    y = x[:, :-1] + near * torch.randn(b, q - 1, vocab, generator=gen)
    d = torch.softmax(y, -1)
    noise = torch.rand(d.shape, generator=gen).clamp(min=1e-30)
    t = dict(target_probs=p, draft_tokens=(noise.log() / d.clamp(min=1e-38)).argmax(-1).int() if q > 1 else
             torch.zeros(b, 0, dtype=torch.int32), uniforms=torch.rand(b, q, generator=gen))
    if drafts == "probs":
        t["draft_probs"] = d
    if ragged:
        t["num_draft"] = torch.randint(-1, q, (b,), generator=gen).int()
    return t


@pytest.mark.parametrize("drafts", ["probs", "fixed"])
@pytest.mark.parametrize("vocab", [1, 2, 31, 512, 513, 5000, 32771])
@pytest.mark.parametrize("q", [1, 2, 5])
def test_vocabularies_and_drafts(drafts, vocab, q):
    for near in (0.0, 0.3, 2.0):
        check(make(7, q, vocab, drafts, near, ragged=near > 0, seed=vocab + q))


@pytest.mark.parametrize("vocab", [128000, 151937, 300001])
def test_large_vocabularies(vocab):
    check(make(5, 3, vocab, seed=1))
    check(make(3, 3, vocab, "fixed", near=0.0, seed=2))


def test_the_largest_vocabulary():
    v = 1 << 21
    check(make(2, 2, v, seed=1))
    t = make(1, 1, 8, seed=2)
    t["target_probs"], t["draft_probs"] = torch.zeros(1, 1, v + 1, device="cuda"), None
    with pytest.raises(da.DecodeAttnError) as e:
        run(engine(1), t)
    assert e.value.status == da.DA_ERR_UNSUPPORTED


def test_many_rows_of_the_largest_vocabulary():
    """More rows than clusters of several CTAs are made for: a share's sums still fit."""
    b, v = 700, 1 << 21
    gen = torch.Generator(device="cuda").manual_seed(17)
    p = torch.rand(b, 1, v, generator=gen, device="cuda")
    t = dict(target_probs=p, draft_tokens=torch.zeros(b, 0, dtype=torch.int32), uniforms=torch.rand(b, 1, generator=gen, device="cuda"))
    dev = run(eng := engine(b, pages=16, cols=1), t)
    assert eng.errors() == 0
    for i in range(0, b, 70):
        cum = p[i, 0].double().cumsum(0)
        assert int(dev["tokens_out"][i, 0]) == int((cum <= t["uniforms"][i, 0].double() * cum[-1]).sum())


@pytest.mark.parametrize("b", [1, 3, 300, 700])
def test_batches(b):
    check(make(b, 4, 1000, ragged=True, near=0.5, seed=b))


@pytest.mark.parametrize("q", [17, 33, 34, 65, 100])
def test_many_drafts(q):
    # drafts near the target's own: long accepted runs
    check(make(6, q, 300, near=0.02, seed=q))
    check(make(6, q, 300, near=0.02, ragged=True, seed=q + 1))


def test_greedy():
    gen = torch.Generator().manual_seed(3)
    for b, q in ((1, 1), (5, 4), (200, 40)):
        target = torch.randint(0, 50000, (b, q), generator=gen).int()
        draft = target[:, :-1].clone()
        for i in range(b):
            if q > 1 and i % 4:
                draft[i, i % (q - 1)] = 7
        t = dict(target_tokens=target, draft_tokens=draft)
        check(t)
        check(t | dict(num_draft=torch.randint(-1, q, (b,), generator=gen).int()))


def test_rows_of_a_wider_tensor():
    t = make(4, 3, 1000, seed=5)
    wide = torch.full((4, 3, 1037), 9.0)
    wide[..., 5:1005] = t["target_probs"]
    dwide = torch.full((4, 2, 1003), 9.0)
    dwide[..., :1000] = t["draft_probs"]
    dev, _ = check(t)
    got = run(engine(4), t, target_probs=wide.cuda()[..., 5:1005], draft_probs=dwide.cuda()[..., :1000])
    assert torch.equal(got["tokens_out"], dev["tokens_out"])


def test_exact_borders():
    """u q < p and running sums at their borders, in numbers whose products and sums are exact."""
    p = torch.tensor([0.25, 0.0, 0.25, 0.5, 0.0])
    d = torch.tensor([0.5, 0.25, 0.0, 0.25, 0.0])
    us = [0.0, 0.25, 0.5 - 2.0 ** -25, 0.5, 0.5 + 2.0 ** -24, 1.0 - 2.0 ** -24]
    rows = [(x, u, r) for x in range(5) for u in us for r in us]
    t = dict(target_probs=p.expand(len(rows), 2, 5).contiguous(), draft_probs=d.expand(len(rows), 1, 5).contiguous(),
             draft_tokens=torch.tensor([[x] for x, _, _ in rows], dtype=torch.int32),
             uniforms=torch.tensor([[u, r] for _, u, r in rows]))
    dev, kept = check(t)
    at = {row: (int(kept[i]), dev["tokens_out"][i].tolist()) for i, row in enumerate(rows)}
    assert at[(0, 0.5, 0.0)] == (0, [2, -1])            # 0.5 * 0.5 is not below 0.25; the rest is tokens 2 and 3
    assert at[(0, 0.5 - 2.0 ** -25, 0.25)] == (1, [0, 2])  # accepted; 0.25 of the target ends with token 0
    assert at[(1, 0.0, 0.0)][0] == 0                     # the target never has token 1
    assert at[(2, 1.0 - 2.0 ** -24, 0.5)] == (1, [2, 3])    # the draft never had token 2
    assert at[(3, 1.0 - 2.0 ** -24, 0.0)] == (1, [3, 0])


@pytest.mark.parametrize("vocab", [100003, 262144])
def test_running_sums_keep_small_probabilities(vocab):
    """Equal probabilities: a number in the middle of a token's range finds it. A running sum in fp32 would
    be off by many of them."""
    p = torch.full((vocab,), 1.0 / vocab)
    want = torch.arange(37, vocab, vocab // 50)
    r = ((want.double() + 0.5) / vocab).float()
    # (fp32 numbers are at most 2^-25 off: less than the half range 2^-19 of a token)
    t = dict(target_probs=p.expand(want.numel(), 1, vocab).contiguous(), draft_tokens=torch.zeros(want.numel(), 0, dtype=torch.int32),
             uniforms=r[:, None].contiguous())
    dev, _ = check(t)
    assert torch.equal(dev["tokens_out"][:, 0].cpu().long(), want)


def test_a_great_probability_before_small_ones():
    v = 50000
    p = torch.full((v,), 2.0 ** -40)
    p[3] = 1.0
    n = 40
    border = 1.0 - 2.0 ** -24  # the largest number below 1
    p2 = p.clone()
    p2[v // 2:] = 2.0 ** -38
    t = dict(target_probs=torch.stack([p, p2] * n)[:, None].contiguous(), draft_tokens=torch.zeros(2 * n, 0, dtype=torch.int32),
             uniforms=torch.tensor([[border - i * 2.0 ** -24] for i in range(2 * n)]))
    check(t)


def test_rest_that_is_zero_and_weights_that_are_odd():
    t = make(6, 2, 40, seed=6)
    t["draft_probs"][0, 0] = t["target_probs"][0, 0]      # alike, and yet rejected: u is past 1
    t["uniforms"][0, 0] = 1.5
    t["target_probs"][1, :] = 0.0                         # no token at all
    t["target_probs"][2, 0, 5] = float("nan")
    t["draft_tokens"][2, 0] = 5                           # NaN is never accepted
    t["draft_probs"][3, 0, :] = float("nan")              # nor weighs a rest: the target's own
    t["target_probs"][4, :, 7] = -1.0
    t["uniforms"][5, 1] = float("nan")                    # as 0
    u = {k: v.clone() for k, v in t.items()}
    u["uniforms"][5, 1] = 0.0
    dev = run(eng := engine(6), t)
    assert eng.errors() == da.DA_DEVERR_PROBS
    out, kept = reference(u)
    assert torch.equal(dev["tokens_out"].cpu().long(), out) and torch.equal(dev["num_accepted"].cpu().long(), kept)
    assert out[1].tolist() == [-1, -1] and int(kept[2]) == 0 and int(kept[0]) == 0
    v = make(2, 1, 40, seed=7)
    v["target_probs"][0, 0, 3] = float("inf")
    dev = run(eng, {k: x.repeat(3, *[1] * (x.dim() - 1)) for k, x in v.items()})
    assert eng.errors() == da.DA_DEVERR_PROBS and dev["tokens_out"][0, 0] == -1 and dev["tokens_out"][1, 0] >= 0


def test_numbers_past_their_range_pick_a_token_all_the_same():
    t = make(4, 1, 777, seed=8)
    t["uniforms"][:, 0] = torch.tensor([1.0, 5.0, -2.0, float("inf")])
    dev = run(eng := engine(4), t)
    assert eng.errors() == 0
    some = [(t["target_probs"][i, 0] > 0).nonzero()[:, 0] for i in range(4)]
    got = dev["tokens_out"][:, 0].tolist()
    assert got[:3] == [int(some[0][-1]), int(some[1][-1]), int(some[2][0])] and 0 <= got[3] < 777


def test_padding_and_tokens_past_the_vocabulary_end_the_drafts():
    t = make(4, 5, 64, near=0.0, seed=9)
    t["draft_tokens"][0, 2] = -1
    t["draft_tokens"][1, 0] = -5
    check(t)
    t["draft_tokens"][2, 1] = 64
    check(t, da.DA_DEVERR_TOKEN)
    # one behind the first rejection does not matter
    u = make(1, 3, 64, seed=10)
    u["uniforms"][0, 0] = 2.0
    u["draft_tokens"][0, 1] = 1 << 30
    check(u)


def test_tokens_are_distributed_as_the_target():
    """Of 60000 rows with one drafted token each: the first token out follows the target, whatever the draft.
    Five standard deviations, sqrt(p (1 - p) / n)."""
    n, v = 60000, 6
    gen = torch.Generator().manual_seed(11)
    p = torch.tensor([0.05, 0.3, 0.0, 0.25, 0.3, 0.1])
    d = torch.tensor([0.3, 0.1, 0.2, 0.2, 0.15, 0.05])
    x = torch.multinomial(d, n, replacement=True, generator=gen).int()
    t = dict(target_probs=p.expand(n, 2, v).contiguous(), draft_probs=d.expand(n, 1, v).contiguous(),
             draft_tokens=x[:, None].contiguous(), uniforms=torch.rand(n, 2, generator=gen))
    dev = run(engine(n, pages=16, cols=1), t)
    share = torch.bincount(dev["tokens_out"][:, 0].cpu().long(), minlength=v) / n
    assert ((share - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all()
    assert abs(float(dev["num_accepted"].float().mean()) - float(torch.minimum(p, d).sum())) < 5 * 0.5 / n ** 0.5


class Pages:
    """Rows with pages from a pool, and what is left of it on a stack."""

    def __init__(self, lens, page, cols, spare, room, seed):
        gen = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        perm = torch.randperm(self.pages, generator=gen).int()
        self.table = torch.full((len(lens), cols), -3, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = perm[at:at + n]
            at += n
        self.free = torch.cat([perm[at:], torch.full((room,), -9, dtype=torch.int32)])
        self.num = torch.tensor([spare], dtype=torch.int32)

    def tensors(self, lens):
        return dict(seq_lens=torch.tensor(lens, dtype=torch.int32), seq_lens_out=torch.zeros(len(lens), dtype=torch.int32),
                    block_table=self.table, free_pages=self.free.clone(), num_free=self.num, num_free_out=torch.zeros(1, dtype=torch.int32))


def give_back(t, kept, page, cols, pages):
    b, q = t["draft_tokens"].shape[0], t["draft_tokens"].shape[1] + 1
    lens, free, top = t["seq_lens"].clone(), t["free_pages"].clone(), int(t["num_free"])
    for i in reversed(range(b)):
        n = q - 1 if t.get("num_draft") is None else min(int(t["num_draft"][i]), q - 1)
        old = int(lens[i])
        new = old if n < 0 else old - (n - int(kept[i]))
        if new < 0 or old > cols * page:
            continue
        lens[i] = new
        for c in reversed(range(-(-new // page), -(-old // page))):
            if 0 <= int(t["block_table"][i, c]) < pages:
                if top < free.numel():
                    free[top] = t["block_table"][i, c]
                top += 1
    return lens, free, min(top, free.numel())


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("b,q", [(1, 2), (9, 40), (300, 5), (600, 20)])
@pytest.mark.parametrize("in_place", [False, True])
def test_lengths_and_pages_go_back(page, b, q, in_place):
    gen = torch.Generator().manual_seed(b)
    lens = torch.randint(q, 8 * page, (b,), generator=gen).tolist()
    pool = Pages(lens, page, 8, 5, 3000, seed=b)
    t = make(b, q, 60, near=0.5, ragged=True, seed=q) | pool.tensors(lens)
    eng = engine(b, page=page, cols=8, pages=pool.pages)
    more = {}
    if in_place:
        sl, nf = t["seq_lens"].cuda(), t["num_free"].cuda()
        more = dict(seq_lens=sl, seq_lens_out=sl, num_free=nf, num_free_out=nf)
    dev, kept = check(t, eng=eng, **more)
    lens, free, top = give_back(t, kept, page, 8, pool.pages)
    assert torch.equal(dev["seq_lens_out"].cpu(), lens) and int(dev["num_free_out"]) == top
    assert torch.equal(dev["free_pages"].cpu(), free) and torch.equal(dev["block_table"].cpu(), pool.table)


def test_lengths_alone_and_a_contiguous_cache():
    t = make(5, 4, 60, seed=12) | dict(seq_lens=torch.tensor([100, 4, 50, 7, 9], dtype=torch.int32),
                                       seq_lens_out=torch.zeros(5, dtype=torch.int32))
    for eng in (engine(5), engine(5, page=0, length=128)):
        dev, kept = check(t, eng=eng)
        assert torch.equal(dev["seq_lens_out"].cpu(), (t["seq_lens"] - (3 - kept)).int())


def test_bad_lengths_pages_and_stacks():
    lens = [40, 40, 40, 40]
    pool = Pages(lens, 16, 3, 2, 1, seed=13)
    t = make(4, 16, 60, seed=14) | pool.tensors(lens)
    t["uniforms"][:, 0] = 2.0  # the first draft rejected: 15 of 40 tokens go, and with them one page
    eng = engine(4, cols=3, pages=pool.pages)
    u = {k: v.clone() for k, v in t.items()}
    u["block_table"][3, 2] = pool.pages  # last in its row, outside the pool
    u["seq_lens"][1] = 14                # fewer than were drafted
    u["seq_lens"][0] = 49                # past the table
    dev, kept = check(u, da.DA_DEVERR_PAGE_INDEX | da.DA_DEVERR_SEQ_LEN, eng=eng)
    assert dev["seq_lens_out"].tolist() == [49, 14, 25, 25] and int(dev["num_free_out"]) == 3
    assert dev["free_pages"].tolist() == pool.free[:2].tolist() + [int(pool.table[2, 2])]
    dev, kept = check(t, da.DA_DEVERR_NO_PAGES, eng=eng)  # four pages, room for one
    assert int(dev["num_free_out"]) == 3 and int(dev["free_pages"][2]) == int(pool.table[3, 2])
    v = t | dict(num_free=torch.tensor([-4], dtype=torch.int32))
    dev, _ = check(v, da.DA_DEVERR_NO_PAGES, eng=eng)
    assert int(dev["num_free_out"]) == 3


def test_captured_and_on_two_streams():
    t = make(20, 4, 5000, seed=15)
    engines = [engine(20), engine(20)]
    out, kept = reference(t)
    devs = [run(e, t) for e in engines]
    args = [da.make_verify_args(d) for d in devs]
    for d in devs:
        d["tokens_out"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for e, a, s in zip(engines, args, streams):
            da.decode_attn_verify(e.ctx, a, e.workspace, stream=s)
    torch.cuda.synchronize()
    for d in devs:
        assert torch.equal(d["tokens_out"].cpu().long(), out)
    devs[0]["tokens_out"].zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            da.decode_attn_verify(engines[0].ctx, args[0], engines[0].workspace)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(devs[0]["tokens_out"].cpu().long(), out) and torch.equal(devs[0]["num_accepted"].cpu().long(), kept)


def test_refusals():
    t = {k: v.cuda() for k, v in make(3, 3, 50, seed=16).items()}
    t |= dict(tokens_out=torch.zeros(3, 3, dtype=torch.int32, device="cuda"), num_accepted=torch.zeros(3, dtype=torch.int32, device="cuda"))
    eng = engine(3)
    lens = torch.full((3,), 20, dtype=torch.int32, device="cuda")

    def status(**change):
        a = da.make_verify_args(t)
        for k, v in change.items():
            setattr(a, k, v.data_ptr() if isinstance(v, torch.Tensor) else v)
        with pytest.raises(da.DecodeAttnError) as e:
            da.decode_attn_verify(eng.ctx, a, eng.workspace)
        return e.value.status

    for change in (dict(tokens_out=None), dict(num_accepted=None), dict(target_probs=None), dict(uniforms=None),
                   dict(draft_tokens=None), dict(vocab=0), dict(q_len=0), dict(target_stride=49), dict(draft_stride=49),
                   dict(target_tokens=lens), dict(seq_lens=lens), dict(seq_lens_out=lens), dict(block_table=lens),
                   dict(free_pages=lens), dict(num_free=lens),
                   dict(seq_lens=lens, seq_lens_out=lens, free_pages=lens, num_free=lens, num_free_out=lens)):
        assert status(**change) == da.DA_ERR_INVALID_ARG, change
    assert status(vocab=(1 << 21) + 1, target_stride=1 << 22, draft_stride=1 << 22) == da.DA_ERR_UNSUPPORTED
    flat = engine(3, page=0, length=64)
    a = da.make_verify_args(t | dict(seq_lens=lens, seq_lens_out=lens, block_table=lens, free_pages=lens, num_free=lens[:1], num_free_out=lens[:1]))
    with pytest.raises(da.DecodeAttnError):
        da.decode_attn_verify(flat.ctx, a, flat.workspace)
    for change, match in ((dict(uniforms=t["uniforms"][:2]), "elements"), (dict(target_probs=t["target_probs"].double()), "float32"),
                          (dict(draft_probs=t["draft_probs"][:, :1]), "rows"), (dict(target_probs=t["target_probs"].cpu()), "device"),
                          (dict(target_probs=t["target_probs"].transpose(1, 2).contiguous().transpose(1, 2)), "contiguous"),
                          (dict(draft_tokens=t["draft_tokens"].long()), "int32"), (dict(tokens_out=None), "tokens_out")):
        with pytest.raises(ValueError, match=match):
            eng.verify(t | change)
    with pytest.raises(ValueError, match="rows"):
        engine(4).verify(t)
    assert eng.errors() == 0
