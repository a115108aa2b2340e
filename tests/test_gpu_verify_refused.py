"""Steps with drafts in which a row did not get all of its tokens: the pool was dry, its table was full, or the slot
map was. With the lengths from before the step (`seq_lens_before`) such a row takes no part in the verification and
goes back to what it had; nothing is taken off a length that did not grow."""

import pytest
import torch

import block8_ref as B
import decode_attention_flash_gb300 as da
from test_gpu_speculative_step import HKV, HQ, PAGE, Q, ROWS, SCALE, Server
from test_gpu_verify import Pages, engine, make, reference, run

pytestmark = pytest.mark.gpu


def expected(t, page=1, capacity=None, pages=0):
    """Tokens, accepted counts, lengths, the stack and its top, row by row."""
    b, q = t["uniforms"].shape if t.get("uniforms") is not None else t["target_tokens"].shape
    n = t.get("num_draft")
    n = torch.full((b,), q - 1) if n is None else n.clamp(max=q - 1).clone()
    refused, odd = [], []
    for i in range(b):
        old, now = int(t["seq_lens_before"][i]), int(t["seq_lens"][i])
        odd.append(not 0 <= old <= now)
        refused.append(int(n[i]) >= 0 and (odd[i] or now - old <= int(n[i])))
    out, kept = reference({**t, "num_draft": torch.where(torch.tensor(refused), -1, n).int()})
    lens, free, top = t["seq_lens"].clone(), None, 0
    if t.get("free_pages") is not None:
        free, top = t["free_pages"].clone(), int(t["num_free"])
    for i in reversed(range(b)):
        now = int(lens[i])
        if now < 0 or (capacity and now > capacity) or odd[i] or int(n[i]) < 0:
            continue
        new = int(t["seq_lens_before"][i]) if refused[i] else now - (int(n[i]) - int(kept[i]))
        lens[i] = new
        for c in reversed(range(-(-new // page), -(-now // page))):
            if free is not None:
                free[top] = t["block_table"][i, c]
                top += 1
    return out, kept, lens, free, top


def same(dev, want):
    out, kept, lens, free, top = want
    assert torch.equal(dev["tokens_out"].cpu().long(), out)
    assert torch.equal(dev["num_accepted"].cpu().long(), kept)
    assert torch.equal(dev["seq_lens_out"].cpu(), lens)
    if free is not None:
        assert int(dev["num_free_out"]) == top and torch.equal(dev["free_pages"].cpu(), free)


@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("alias", [None, "seq_lens", "seq_lens_before"])
@pytest.mark.parametrize("b,vocab", [(12, 60), (300, 60), (12, 9000)])
def test_rows_that_got_fewer_tokens_take_no_part(b, vocab, alias, greedy):
    q, page = 5, 16
    gen = torch.Generator().manual_seed(b + vocab)
    before = torch.randint(0, 7 * page - q, (b,), generator=gen).int()
    got = torch.randint(0, q + 1, (b,), generator=gen).int()  # of q tokens, none and all among them
    got[:q + 1] = torch.arange(q + 1)
    lens = (before + got).tolist()
    pool = Pages(lens, page, 8, 5, 2000, seed=b)
    t = make(b, q, vocab, near=0.3, seed=b) | pool.tensors(lens) | dict(seq_lens_before=before)
    if greedy:
        t["target_tokens"] = torch.cat([t["draft_tokens"], t["draft_tokens"][:, :1]], 1)
        t["target_tokens"][::3, 2] += 1
        for name in ("target_probs", "uniforms"):
            del t[name]
        t.pop("draft_probs", None)
    eng = engine(b, page=page, cols=8, pages=pool.pages)
    for ragged in (False, True):
        if ragged:
            t["num_draft"] = torch.randint(-1, q, (b,), generator=gen).int()
        more = {}
        if alias:
            more[alias] = more["seq_lens_out"] = t[alias].cuda()
        want = expected(t, page, 8 * page)
        same(run(eng, t, **more), want)
        plain = {k: v for k, v in t.items() if k not in ("block_table", "free_pages", "num_free", "num_free_out")}
        if alias:
            more[alias] = more["seq_lens_out"] = t[alias].cuda()
        same(run(eng, plain, **more), expected(plain, page, 8 * page))
        assert eng.errors() == 0


def test_lengths_from_before_that_cannot_be():
    t = make(4, 3, 50, seed=2) | dict(seq_lens=torch.tensor([20, 20, 20, 2000], dtype=torch.int32),
                                      seq_lens_out=torch.zeros(4, dtype=torch.int32),
                                      seq_lens_before=torch.tensor([21, -1, 17, 1990], dtype=torch.int32))
    eng = engine(4, cols=4)
    dev = run(eng, t)
    assert eng.errors() == da.DA_DEVERR_SEQ_LEN
    same(dev, expected(t, 1, 64))
    assert dev["seq_lens_out"].tolist()[:2] == [20, 20] and dev["num_accepted"].tolist()[:2] == [0, 0]


def test_lengths_from_before_need_lengths():
    t = make(3, 3, 50, seed=3) | dict(seq_lens_before=torch.full((3,), 5, dtype=torch.int32))
    with pytest.raises(da.DecodeAttnError) as e:
        run(engine(3), t)
    assert e.value.status == da.DA_ERR_INVALID_ARG
    t["seq_lens_before"] = t["seq_lens_before"][:2]
    with pytest.raises(ValueError, match="seq_lens_before"):
        run(engine(3), t)


class Tight(Server):
    """A server that keeps the committed lengths apart from the step's, on a pool that runs dry."""

    def __init__(self, kind, block, spare, seed=0):
        super().__init__(kind, block, seed)
        self.now = torch.zeros_like(self.lens)
        self.num_free.fill_(spare)

    def step(self, checks=False):
        free = dict(free_pages=self.free, num_free=self.num_free, num_free_out=self.num_free)
        self.eng.build_tables(dict(seq_lens=self.lens, new_lens=self.new, seq_lens_out=self.now, block_table=self.table,
                                   slot_map=self.slots, positions=self.pos, **free))
        new = dict(q=self.qkv[:, :HQ], k_new=self.qkv[:, HQ:HQ + HKV], v_new=self.qkv[:, HQ + HKV:], q_out=self.q_out,
                   slot_map=self.slots, positions=self.pos, cos_sin=self.cos_sin, **self.w)
        self.eng.append({**self.cache, **new}, q_len=Q)
        if checks:
            self.plain.append({**self.rows, **new}, q_len=Q)
        self.eng.run({**self.cache, "q": self.q_out, "block_table": self.table, "seq_lens": self.now}, SCALE,
                     out=self.out, lse=self.lse)
        logits = self.out.transpose(1, 2).reshape(ROWS, Q, HQ * 128).float() @ self.head
        self.probs = torch.softmax(logits, -1)
        self.eng.verify(dict(target_probs=self.probs, draft_tokens=self.draft, uniforms=self.uniforms, tokens_out=self.tokens,
                             num_accepted=self.kept, seq_lens=self.now, seq_lens_before=self.lens, seq_lens_out=self.lens,
                             block_table=self.table, **free))

    def check(self, lens, pool):
        """Lengths, and every page once: with a row, or on the stack."""
        assert self.lens.tolist() == lens
        n = int(self.num_free)
        used = [p for b in range(ROWS) for p in self.table[b, : -(-lens[b] // PAGE)].tolist()]
        assert sorted(used + self.free[:n].tolist()) == sorted(pool)
        for s in ("k", "v"):
            got = B.values(self.cache[s].cpu(), self.cache[s + "_scale"].cpu(), self.block)
            step = self.cache[s + "_scale"].cpu().double().repeat_interleave(self.block, -1)[..., None]
            want = self.rows[s].cpu().double()
            tol = 2.0 ** -4 * want.abs() + 2.0 ** -9 * step if self.kind == "e4m3" else step
            for b in range(ROWS):
                for j in range(-(-lens[b] // PAGE)):
                    p, m = int(self.table[b, j]), min(PAGE, lens[b] - j * PAGE)
                    assert not ((got[p, :, :m] - want[p, :, :m]).abs() > tol[p].expand_as(want[p])[:, :m]).any()



@pytest.mark.parametrize("kind,block", [("e4m3", 16), ("int8", 32)])
def test_a_dry_pool_leaves_the_rows_that_got_nothing(kind, block):
    s = Tight(kind, block, spare=8, seed=2)
    pool = s.free[:8].tolist()
    gen = torch.Generator().manual_seed(6)
    lens, dry, back = [0] * ROWS, 0, 0
    for _ in range(60):
        s.inputs(gen)
        s.step(checks=True)
        now, kept = s.now.tolist(), s.kept.tolist()
        flags = s.eng.errors()
        s.plain.errors()
        for b in range(ROWS):
            if now[b] == lens[b]:  # the pool was dry for it
                dry += 1
                assert flags & da.DA_DEVERR_NO_PAGES and kept[b] == 0 and (s.tokens[b] == -1).all()
            else:
                assert now[b] == lens[b] + Q
                assert s.tokens[b, :kept[b]].tolist() == s.draft[b, :kept[b]].tolist() and int(s.tokens[b, kept[b]]) >= 0
                back += Q - 1 - kept[b]
                lens[b] += 1 + kept[b]
        assert flags & ~(da.DA_DEVERR_NO_PAGES | da.DA_DEVERR_PROBS) == 0
        s.check(lens, pool)
    assert dry > ROWS and back > 0


def test_a_row_at_its_capacity_stays_there_and_captured_steps_are_the_same():
    a, b = (Tight("e4m3", 16, spare=ROWS * 12, seed=3) for _ in range(2))
    cap = 12 * PAGE
    start = [cap - Q - 1, cap - 2, cap - 70, 5, 0]
    for s in (a, b):  # rows that hold zeros so far
        at = 0
        for i, n in enumerate(start):
            m = -(-n // PAGE)
            s.table[i, :m] = s.free[ROWS * 12 - at - m:ROWS * 12 - at].flip(0)
            at += m
        s.num_free.fill_(ROWS * 12 - at)
        s.lens.copy_(torch.tensor(start))
    pool = a.free.tolist()
    warm = Tight("e4m3", 16, spare=0, seed=3)
    warm.inputs(torch.Generator().manual_seed(4))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        warm.step()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step()
    gens = [torch.Generator().manual_seed(5) for _ in range(2)]
    lens, cut = list(start), 0
    for _ in range(25):
        a.inputs(gens[0])
        a.step(checks=True)
        b.inputs(gens[1])
        g.replay()
        now, kept = a.now.tolist(), a.kept.tolist()
        assert a.eng.errors() & ~(da.DA_DEVERR_SEQ_LEN | da.DA_DEVERR_PROBS) == 0
        a.plain.errors()
        for i in range(ROWS):
            assert now[i] == min(lens[i] + Q, cap)
            if now[i] < lens[i] + Q:
                cut += 1
                assert kept[i] == 0 and (a.tokens[i] == -1).all()
            else:
                lens[i] += 1 + kept[i]
        a.check(lens, pool)
    assert cut >= 25 and lens[3] > start[3]
    torch.cuda.synchronize()
    for name in ("lens", "num_free", "table", "tokens", "kept"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    for name in a.cache:
        assert torch.equal(a.cache[name].view(torch.uint8), b.cache[name].view(torch.uint8)), name
