"""The operators of a serving step together: tables from lengths, rows appended,
decode attention over the cache (and the rows read back), for every element
kind, against 64 bits; then a decode loop as one captured graph."""

import math

import pytest
import torch

import decode_attention_flash_gb300 as da

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
KINDS = {"bf16": (da.DA_DTYPE_BF16, 0), "e4m3": (da.DA_DTYPE_FP8_E4M3, 0),
         "token": (da.DA_DTYPE_FP8_E4M3_TOKEN_SCALE, 0), "int4": (da.DA_DTYPE_INT4_GROUPS, 4),
         "fp4": (da.DA_DTYPE_FP4_E2M1_BLOCKS, 0)}


class Server:
    def __init__(self, kind, batch=5, hq=8, hkv=2, page=16, pages=120, cols=20):
        self.batch, self.hq, self.hkv, self.page = batch, hq, hkv, page
        dtype, groups = KINDS[kind]
        self.eng = da.DecodeAttention(
            device=0, batch=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim_qk=128, head_dim_v=128,
            kv_layout=da.DA_KV_PAGED, page_size=page, max_seq_len=cols * page, max_pages_per_seq=cols, num_pages=pages,
            q_dtype=da.DA_DTYPE_BF16, kv_dtype=dtype, kv_groups=groups)
        kb, vb, slots = self.eng._cache_sizes()
        gen = torch.Generator().manual_seed(7)
        self.cache = dict(k=torch.zeros(kb, dtype=torch.uint8, device="cuda"), v=torch.zeros(vb, dtype=torch.uint8, device="cuda"))
        if kind in ("e4m3", "fp4"):
            s = 0.02 if kind == "e4m3" else 0.003
            self.cache |= dict(k_scale=torch.full((hkv,), s, device="cuda"), v_scale=torch.full((hkv,), s * 1.3, device="cuda"))
        if kind == "token":
            self.cache |= {k: torch.zeros(slots * hkv, dtype=torch.int32, device="cuda") for k in ("k_scale_shift", "v_scale_shift")}
        z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.tab = dict(seq_lens=z(batch), block_table=z(batch, cols), num_free=torch.tensor([pages], dtype=torch.int32, device="cuda"),
                        free_pages=torch.randperm(pages, generator=gen).int().cuda())
        self.tab |= dict(seq_lens_out=self.tab["seq_lens"], num_free_out=self.tab["num_free"])
        inv = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
        a = torch.arange(cols * page, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([a.cos(), a.sin()], -1).float().cuda()
        self.gen = gen

    def feed(self, new, capacity):
        """New tokens for the rows (a list of counts), appended; the rotated queries."""
        hq, hkv = self.hq, self.hkv
        qkv = torch.randn(capacity, hq + 2 * hkv, 128, generator=self.gen).to(torch.bfloat16).cuda()
        t = dict(new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"),
                 slot_map=torch.zeros(capacity, dtype=torch.int64, device="cuda"),
                 positions=torch.zeros(capacity, dtype=torch.int32, device="cuda"))
        self.eng.build_tables(self.tab | t)
        q_out = torch.zeros(capacity, hq, 128, dtype=torch.bfloat16, device="cuda")
        self.eng.append(self.cache | dict(q=qkv[:, :hq], k_new=qkv[:, hq:hq + hkv], v_new=qkv[:, hq + hkv:], q_out=q_out,
                                          slot_map=t["slot_map"], positions=t["positions"], cos_sin=self.cos_sin))
        return q_out

    def read(self):
        """Every cached row in order, bf16 [tokens, HKV, 128] twice."""
        n = int(self.tab["seq_lens"].sum())
        t = dict(seq_lens=torch.zeros_like(self.tab["seq_lens"]), new_lens=self.tab["seq_lens"], block_table=self.tab["block_table"],
                 seq_lens_out=torch.zeros_like(self.tab["seq_lens"]), slot_map=torch.zeros(n, dtype=torch.int64, device="cuda"))
        self.eng.build_tables(t)
        out = {k: torch.zeros(n, self.hkv, 128, dtype=torch.bfloat16, device="cuda") for k in ("k_out", "v_out")}
        return self.eng.gather(self.cache | out | dict(slot_map=t["slot_map"]))

    def attend(self, q, out=None, lse=None):
        return self.eng.run(self.cache | dict(q=q, seq_lens=self.tab["seq_lens"], block_table=self.tab["block_table"]),
                            SCALE, out=out, lse=lse)

    def expected(self, q):
        k, v = (x.cpu().double() for x in self.read())
        g = self.hq // self.hkv
        out = torch.zeros(self.batch, self.hq, 128, dtype=torch.float64)
        at = 0
        for b, n in enumerate(self.tab["seq_lens"].tolist()):
            for h in range(self.hq):
                if n:
                    w = torch.softmax(k[at:at + n, h // g] @ q[b, h].cpu().double() * SCALE, 0)
                    out[b, h] = w @ v[at:at + n, h // g]
            at += n
        return out


def close(got, want, k):
    # the read-back rows are rounded to bf16 (2^-8 of an element) where the attention
    # takes the cached value: of a key that moves a score by at most
    # 2^-8 * scale * sum|q k|, of a value by 2^-8; then the output's own rounding
    # and the weights' (f16 2^-11 or bf16 2^-8)
    d = (got.cpu().double() - want).abs().max().item()
    assert d <= k, d


@pytest.mark.parametrize("kind", list(KINDS))
def test_prefill_then_decode_steps(kind):
    s = Server(kind)
    s.feed([3, 0, 40, 17, 1], 61)
    for step in range(20):
        q = s.feed([1] * s.batch, s.batch)
        if step % 9 in (0, 8):
            got, want = s.attend(q), s.expected(q)
            torch.cuda.synchronize()
            assert s.eng.errors() == 0
            # |k|, |v| < 6 here: scores move by at most 2^-8 * 128 * 6 * 4 / 11.3 * (their signs
            # average out; sqrt(128) of them count), weights by the same share
            close(got, want, 0.08)
    assert s.tab["seq_lens"].tolist() == [23, 20, 60, 37, 21]


@pytest.mark.parametrize("kind", ["fp4", "bf16"])
def test_decode_loop_as_one_graph(kind):
    s, ref = Server(kind), Server(kind)
    for x in (s, ref):
        x.feed([30, 5, 16, 0, 64], 115)
    b, hq, hkv = s.batch, s.hq, s.hkv
    qkv = torch.zeros(b, hq + 2 * hkv, 128, dtype=torch.bfloat16, device="cuda")
    step = dict(new_lens=torch.ones(b, dtype=torch.int32, device="cuda"), slot_map=torch.zeros(b, dtype=torch.int64, device="cuda"),
                positions=torch.zeros(b, dtype=torch.int32, device="cuda"))
    q_out = torch.zeros(b, hq, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q_out), torch.zeros(b, hq, device="cuda")

    def one():
        s.eng.build_tables(s.tab | step)
        s.eng.append(s.cache | dict(q=qkv[:, :hq], k_new=qkv[:, hq:hq + hkv], v_new=qkv[:, hq + hkv:], q_out=q_out,
                                    slot_map=step["slot_map"], positions=step["positions"], cos_sin=s.cos_sin))
        s.attend(q_out, out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            one()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(12):
        new = torch.randn(b, hq + 2 * hkv, 128, generator=ref.gen).to(torch.bfloat16).cuda()
        qkv.copy_(new)
        g.replay()
        # the same step, eagerly, on another cache
        t = dict(new_lens=step["new_lens"], slot_map=torch.zeros_like(step["slot_map"]), positions=torch.zeros_like(step["positions"]))
        ref.eng.build_tables(ref.tab | t)
        q2 = torch.zeros_like(q_out)
        ref.eng.append(ref.cache | dict(q=new[:, :hq], k_new=new[:, hq:hq + hkv], v_new=new[:, hq + hkv:], q_out=q2,
                                        slot_map=t["slot_map"], positions=t["positions"], cos_sin=ref.cos_sin))
        lse2 = torch.zeros_like(lse)
        want = ref.attend(q2, lse=lse2)
        torch.cuda.synchronize()
        assert torch.equal(q_out, q2) and torch.equal(out, want) and torch.equal(lse, lse2)
    assert s.eng.errors() == 0 and ref.eng.errors() == 0
    assert s.tab["seq_lens"].tolist() == [42, 17, 28, 12, 76] and math.isfinite(float(out.float().sum()))
