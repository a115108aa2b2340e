"""A serving loop held against a model of its own: keys, values and queries stay on the host,
are turned and quantised there by the formats' definitions, and attended to in 64 bits. The
library's tables, slots, appended rows and read-backs are on one side only.

Bounds, all from the roundings that a decode makes (half a step each): weights as bf16 (2^-8;
the bf16 cache) or f16 (2^-11, 2^-25 below 2^-14; the others), values formed in f16 (int4: the
value; token scales: code * scale), keys formed in f16 (int4), fp32 scores of 128 products, a
bf16 output. Every check of a row of less than 100 tokens also makes sure that its bound would
tell the loss of an ordinary one."""

import pytest
import torch

import decode_attention_flash_gb300 as da
from test_gpu_serving_step import KINDS, SCALE, Server

pytestmark = pytest.mark.gpu
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()


def cached(kind, x, head_scale):
    """What a row's x [T, H, 128] (fp32, bf16 values) stands for in the cache, float64, and the size
    of the shift in it. Every operation is one rounding to fp32, as the formats define them."""
    none = torch.zeros(*x.shape[:2], 1, dtype=torch.float64)
    if kind == "bf16":
        return x.double(), none
    hs = head_scale.cpu()[None, :, None] if head_scale is not None else None
    if kind == "e4m3":
        return e4m3(x * (1.0 / hs)).double() * hs.double(), none
    if kind == "fp4":
        b = x.view(*x.shape[:2], 8, 16)
        g = hs[..., None]
        sb = e4m3(b.abs().amax(-1, keepdim=True) / (6.0 * g))
        eff = sb * g
        y = (b * torch.where(eff >= 2.0 ** -126, 1.0 / eff, torch.zeros_like(eff))).double()
        m = y.abs().clamp(max=6.0)
        unit = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
        v = torch.copysign(torch.round(m / unit) * unit, y) * (sb.double() * g.double())
        return v.flatten(-2), none
    groups = 4 if kind == "int4" else 1
    b = x.view(*x.shape[:2], groups, -1)
    hi, lo = b.amax(-1, keepdim=True), b.amin(-1, keepdim=True)
    if kind == "int4":
        sh, sc = lo.half().float(), ((hi - lo) / 15.0).half().float()
    else:
        sh, sc = ((hi + lo) * 0.5).half().float(), ((hi - lo) * 0.5 / 448.0).half().float()
    sc = torch.where(sc == 0, torch.ones_like(sc), sc)
    y = (b - sh) * (1.0 / sc)
    code = torch.round(y).clamp(0, 15) if kind == "int4" else e4m3(y)
    v = code.double() * sc.double() + sh.double()
    return v.flatten(-2), sh.double().expand_as(b).abs().flatten(-2)


def turned(x, pos, cos_sin):
    """x [T, H, 128] fp32 by the angles of pos [T]: each product and sum rounded to fp32, then bf16."""
    row = cos_sin[pos][:, None]
    c, s, a, b = row[..., :64], row[..., 64:], x[..., :64], x[..., 64:]
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    return torch.cat([ac - bs, bc + as_], -1).to(torch.bfloat16).float()


class Model:
    """The rows' keys and values on the host, in order of position."""

    def __init__(self, kind, server):
        self.kind, self.hq, self.hkv, self.batch = kind, server.hq, server.hkv, server.batch
        self.scales = {n: server.cache.get(n + "_scale") for n in "kv"}
        self.cos_sin = server.cos_sin.cpu()
        self.len = [0] * self.batch
        self.rows = [[] for _ in range(self.batch)]

    def feed(self, new, qkv):
        """Tokens of the rows, row after row; their turned queries."""
        x = qkv.float()
        row = [b for b, n in enumerate(new) for _ in range(n)]
        pos = torch.tensor([self.len[b] + i for b, n in enumerate(new) for i in range(n)], dtype=torch.long)
        n = len(row)
        q, k, v = x[:n, :self.hq], x[:n, self.hq:self.hq + self.hkv], x[:n, self.hq + self.hkv:]
        k, ksh = cached(self.kind, turned(k, pos, self.cos_sin), self.scales["k"])
        v, vsh = cached(self.kind, v, self.scales["v"])
        for i, b in enumerate(row):
            self.rows[b].append((k[i], v[i], ksh[i].expand(-1, 128), vsh[i].expand(-1, 128)))
        self.len = [a + c for a, c in zip(self.len, new)]
        return turned(q, pos, self.cos_sin)

    def check(self, q, out, lse=None):
        """One query token a row: q, out [B, HQ, 128]."""
        out = out.cpu().double()
        g = self.hq // self.hkv
        for b in range(self.batch):
            if not self.rows[b]:
                assert (out[b] == 0).all()
                continue
            K, V, ksh, vsh = (torch.stack(t) for t in zip(*self.rows[b]))
            for h in range(self.hq):
                k, v, x = K[:, h // g], V[:, h // g], q[b, h].double()
                s = (k @ x) * SCALE
                size = ((k.abs() + 2 * ksh[:, h // g]) @ x.abs()) * SCALE
                l = torch.logsumexp(s, 0)
                w = torch.exp(s - l)
                want, a = w @ v, w @ v.abs()
                # 128 products and sums, then a few roundings of the score and the exponential
                delta = (160 * size.max() + 16 * s.abs().max() + 16) * 2.0 ** -24
                tol = 2.0 ** -8 * want.abs() + 2 * delta * a + 2.0 ** -30
                if self.kind == "int4":
                    # an element of a key is rounded once, to f16: a score moves by at most ds, the
                    # output by sum w ds (v - output), and 1 % of that for the terms in ds^2
                    ds = (2.0 ** -11 * (k.abs() @ x.abs()) + 2.0 ** -25 * x.abs().sum()) * SCALE
                    tol = tol + 1.01 * (w * ds) @ (v - want).abs()
                    delta = delta + ds.max()
                if self.kind == "bf16":
                    tol = tol + 2.0 ** -8 * a
                else:
                    tol = tol + 2.0 ** -11 * a + 2.0 ** -25 * v.abs().sum(0) * torch.exp(s.max() - l)
                if self.kind in ("int4", "token"):
                    tol = tol + w @ (2.0 ** -11 * (v.abs() + vsh[:, h // g]) + 2.0 ** -25)
                worst = ((out[b, h] - want).abs() / tol).max().item()
                assert worst <= 1, (b, h, worst)
                if lse is not None:
                    assert abs(lse[b, h].item() - l.item()) <= delta + 2.0 ** -20 * (1 + abs(l.item()))
                if 1 < len(w) < 100:  # (of more, one counts less than the roundings of all)
                    j = w.argsort()[len(w) // 2]
                    keep = torch.arange(len(w)) != j
                    less = (w[keep] / w[keep].sum()) @ v[keep]
                    assert ((less - want).abs() > 2 * tol).any(), (b, h, "the bound would not tell")


def tokens(server, capacity):
    return torch.randn(capacity, server.hq + 2 * server.hkv, 128, generator=server.gen).to(torch.bfloat16)


def feed(s, new, capacity, host):
    qkv = host.cuda()
    t = dict(new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"),
             slot_map=torch.zeros(capacity, dtype=torch.int64, device="cuda"),
             positions=torch.zeros(capacity, dtype=torch.int32, device="cuda"))
    s.eng.build_tables(s.tab | t)
    q_out = torch.zeros(capacity, s.hq, 128, dtype=torch.bfloat16, device="cuda")
    s.eng.append(s.cache | dict(q=qkv[:, :s.hq], k_new=qkv[:, s.hq:s.hq + s.hkv], v_new=qkv[:, s.hq + s.hkv:], q_out=q_out,
                                slot_map=t["slot_map"], positions=t["positions"], cos_sin=s.cos_sin))
    return q_out


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("prompt", [[3, 0, 40, 17, 1], [130, 5, 0, 60, 33]])
def test_prompt_and_steps_against_a_model_of_their_own(kind, prompt):
    s = Server(kind)
    m = Model(kind, s)
    host = tokens(s, sum(prompt))
    got = feed(s, prompt, sum(prompt), host)
    assert torch.equal(got.cpu().float(), m.feed(prompt, host))
    for step in range(20):
        host = tokens(s, s.batch)
        got = feed(s, [1] * s.batch, s.batch, host)
        q = m.feed([1] * s.batch, host)
        assert torch.equal(got.cpu().float(), q)
        if step % 6 in (0, 1):
            lse = torch.zeros(s.batch, s.hq, device="cuda")
            out = s.attend(got, lse=lse)
            torch.cuda.synchronize()
            assert s.eng.errors() == 0
            m.check(q, out, lse)
    assert s.tab["seq_lens"].tolist() == m.len == [n + 20 for n in prompt]


@pytest.mark.parametrize("kind", ["fp4", "bf16"])
def test_a_captured_step_against_a_model_of_its_own(kind):
    s = Server(kind)
    m = Model(kind, s)
    prompt = [30, 5, 16, 0, 64]
    host = tokens(s, sum(prompt))
    feed(s, prompt, sum(prompt), host)
    m.feed(prompt, host)
    b, hq, hkv = s.batch, s.hq, s.hkv
    qkv = torch.zeros(b, hq + 2 * hkv, 128, dtype=torch.bfloat16, device="cuda")
    step = dict(new_lens=torch.ones(b, dtype=torch.int32, device="cuda"), slot_map=torch.zeros(b, dtype=torch.int64, device="cuda"),
                positions=torch.zeros(b, dtype=torch.int32, device="cuda"))
    q_out = torch.zeros(b, hq, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q_out), torch.zeros(b, hq, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.eng.build_tables(s.tab | step)
        s.eng.append(s.cache | dict(q=qkv[:, :hq], k_new=qkv[:, hq:hq + hkv], v_new=qkv[:, hq + hkv:], q_out=q_out,
                                    slot_map=step["slot_map"], positions=step["positions"], cos_sin=s.cos_sin))
        s.attend(q_out, out, lse)
    for i in range(12):
        new = tokens(s, b)
        qkv.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        q = m.feed([1] * b, new)
        assert torch.equal(q_out.cpu().float(), q)
        if i % 4 in (0, 3):
            m.check(q, out, lse)
    assert s.eng.errors() == 0 and s.tab["seq_lens"].tolist() == m.len
