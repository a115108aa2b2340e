"""Serving steps that draft tokens, as a program runs them: tables for the query tokens, queries and keys
normed, turned and written into 8-bit blocks, attention of several query tokens, the drafts verified against
probabilities made of its output, lengths and pages taken back. Nothing of the library is waited for between the
calls; the last test captures the whole step."""

import pytest
import torch

import block8_ref as B
import decode_attention_flash_gb300 as da
import fp4_ref as R
from test_gpu_cache_rows import tables

pytestmark = pytest.mark.gpu
ROWS, HQ, HKV, Q, PAGE, COLS, VOCAB = 5, 8, 2, 4, 32, 12, 301
SCALE = 128 ** -0.5


class Server:
    def __init__(self, kind, block, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.kind, self.block, self.pages = kind, block, ROWS * COLS
        kw = dict(device=0, batch=ROWS, num_q_heads=HQ, num_kv_heads=HKV, head_dim_qk=128, head_dim_v=128,
                  kv_layout=da.DA_KV_PAGED, page_size=PAGE, num_pages=self.pages, max_pages_per_seq=COLS,
                  max_seq_len=COLS * PAGE, q_len=Q)
        self.eng = da.DecodeAttention(kv_dtype=B.KINDS[kind], kv_groups=block, **kw)
        self.plain = da.DecodeAttention(**kw)  # the same rows in bf16, to compare with
        z = dict(device="cuda")
        self.cache = {s: torch.zeros(self.pages, HKV, PAGE, 128, dtype=B.DTYPE[kind], **z) for s in ("k", "v")}
        self.cache |= {s + "_scale": torch.zeros(self.pages, HKV, PAGE // block, **z) for s in ("k", "v")}
        self.rows = {s: torch.zeros(self.pages, HKV, PAGE, 128, dtype=torch.bfloat16, **z) for s in ("k", "v")}
        i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, **z)  # noqa: E731
        self.lens, self.new, self.num_free = i32(ROWS), torch.full((ROWS,), Q, dtype=torch.int32, **z), torch.tensor([self.pages], dtype=torch.int32, **z)
        self.free, self.table = torch.randperm(self.pages, generator=gen).int().cuda(), i32(ROWS, COLS)
        self.slots, self.pos = torch.zeros(ROWS * Q, dtype=torch.int64, **z), i32(ROWS * Q)
        self.q_out = torch.zeros(ROWS, HQ, Q, 128, dtype=torch.bfloat16, **z)
        self.out, self.lse = torch.zeros_like(self.q_out), torch.zeros(ROWS, HQ, Q, **z)
        self.tokens, self.kept = i32(ROWS, Q), i32(ROWS)
        self.qkv = torch.zeros(ROWS * Q, HQ + 2 * HKV, 128, dtype=torch.bfloat16, **z)
        self.draft, self.uniforms = i32(ROWS, Q - 1), torch.zeros(ROWS, Q, **z)
        self.w = dict(q_weight=torch.rand(128, generator=gen).cuda() + 0.5, k_weight=torch.rand(128, generator=gen).cuda() + 0.5)
        self.cos_sin = tables(128, COLS * PAGE).cuda()
        self.head = torch.randn(HQ * 128, VOCAB, generator=gen).cuda() * 0.02

    def inputs(self, gen):
        self.qkv.copy_(torch.randn(ROWS * Q, HQ + 2 * HKV, 128, generator=gen))
        self.draft.copy_(torch.randint(0, VOCAB, (ROWS, Q - 1), generator=gen))
        u = torch.rand(ROWS, Q, generator=gen)
        u[:, :-1] *= 0.004  # (a random draft's probability is about 1 / 301: many are accepted)
        self.uniforms.copy_(u)

    def step(self, checks=False):
        free = dict(free_pages=self.free, num_free=self.num_free, num_free_out=self.num_free)
        self.eng.build_tables(dict(seq_lens=self.lens, new_lens=self.new, seq_lens_out=self.lens, block_table=self.table,
                                   slot_map=self.slots, positions=self.pos, **free))
        new = dict(q=self.qkv[:, :HQ], k_new=self.qkv[:, HQ:HQ + HKV], v_new=self.qkv[:, HQ + HKV:], q_out=self.q_out,
                   slot_map=self.slots, positions=self.pos, cos_sin=self.cos_sin, **self.w)
        self.eng.append({**self.cache, **new}, q_len=Q)
        if checks:
            self.plain.append({**self.rows, **new}, q_len=Q)
        self.eng.run({**self.cache, "q": self.q_out, "block_table": self.table, "seq_lens": self.lens}, SCALE,
                     out=self.out, lse=self.lse)
        if checks:
            self.check_attention()
        logits = self.out.transpose(1, 2).reshape(ROWS, Q, HQ * 128).float() @ self.head
        self.probs = torch.softmax(logits, -1)
        self.eng.verify(dict(target_probs=self.probs, draft_tokens=self.draft, uniforms=self.uniforms, tokens_out=self.tokens,
                             num_accepted=self.kept, seq_lens=self.lens, seq_lens_out=self.lens, block_table=self.table, **free))

    def check_attention(self):
        t = {k: v.cpu() for k, v in self.cache.items()} | dict(q=self.q_out.cpu(), block_table=self.table.cpu(), seq_lens=self.lens.cpu())
        R.check(self.out, self.lse, B.reference(t, SCALE, block=self.block, hq=HQ, hkv=HKV, q_len=Q, page=PAGE))

    def check_state(self, lens):
        """Lengths, pages and what the rows' positions hold, after a step."""
        assert self.eng.errors() == self.plain.errors() == 0
        assert self.lens.tolist() == lens
        n = int(self.num_free)
        used = [p for b in range(ROWS) for p in self.table[b, : -(-lens[b] // PAGE)].tolist()]
        assert sorted(used + self.free[:n].tolist()) == list(range(self.pages))
        for s in ("k", "v"):
            got = B.values(self.cache[s].cpu(), self.cache[s + "_scale"].cpu(), self.block)
            step = self.cache[s + "_scale"].cpu().double().repeat_interleave(self.block, -1)[..., None]
            want = self.rows[s].cpu().double()
            # half a step of e4m3 (2^-4 of the value, or the halves of its least ones); one step of an integer
            tol = 2.0 ** -4 * want.abs() + 2.0 ** -9 * step if self.kind == "e4m3" else step
            for b in range(ROWS):
                for j in range(-(-lens[b] // PAGE)):
                    p, m = int(self.table[b, j]), min(PAGE, lens[b] - j * PAGE)
                    bad = (got[p, :, :m] - want[p, :, :m]).abs() > tol[p].expand_as(want[p])[:, :m]
                    assert not bad.any()


@pytest.mark.parametrize("kind,block", [("e4m3", 16), ("int8", 32)])
def test_steps_with_drafts(kind, block):
    s = Server(kind, block)
    gen = torch.Generator().manual_seed(3)
    lens, most = [0] * ROWS, 0
    for _ in range(40):
        s.inputs(gen)
        s.step(checks=True)
        kept = s.kept.tolist()
        lens = [n + 1 + k for n, k in zip(lens, kept)]
        most = max(most, *kept)
        for b in range(ROWS):
            assert s.tokens[b, :kept[b]].tolist() == s.draft[b, :kept[b]].tolist()
            assert 0 <= int(s.tokens[b, kept[b]]) < VOCAB and (s.tokens[b, kept[b] + 1:] == -1).all()
        s.check_state(lens)
    assert most > 0 and max(lens) > 2 * PAGE


def test_a_captured_step_is_the_same():
    a, b = Server("e4m3", 16, seed=1), Server("e4m3", 16, seed=1)
    gen = torch.Generator().manual_seed(4)
    a.inputs(gen)
    warm = Server("e4m3", 16, seed=1)
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
    for _ in range(12):
        a.inputs(gens[0])
        a.step()
        b.inputs(gens[1])
        g.replay()
    torch.cuda.synchronize()
    assert a.eng.errors() == b.eng.errors() == 0
    for name in ("lens", "num_free", "table", "out", "tokens", "kept"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    for name in a.cache:
        assert torch.equal(a.cache[name].view(torch.uint8), b.cache[name].view(torch.uint8)), name
