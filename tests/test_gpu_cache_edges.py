"""Calls that a server makes and a unit test easily forgets: caches larger than 32-bit
offsets, two calls at once, graphs that share a workspace, lengths that outgrow their
plan, query layouts of several tokens for the latent cache."""

import pytest
import torch

import decode_attention_flash_gb300 as da
import fp4_ref as R
from test_gpu_fp4 import SCALE, engine, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp4", "bf16"])
def test_rows_behind_four_gigabytes(kind):
    hkv, page = 8, 16
    fp4 = kind == "fp4"
    page_bytes = hkv * (1152 if fp4 else page * 256)
    pages = (1 << 32) // page_bytes + 2000
    need = 2 * pages * page_bytes
    if torch.cuda.mem_get_info()[0] < need + (2 << 30):
        pytest.skip("not enough free memory")
    eng = da.DecodeAttention(device=0, batch=1, num_q_heads=16, num_kv_heads=hkv, head_dim_qk=128, head_dim_v=128,
                             kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=pages, max_pages_per_seq=8, max_seq_len=128,
                             q_dtype=da.DA_DTYPE_BF16, kv_dtype=da.DA_DTYPE_FP4_E2M1_BLOCKS if fp4 else da.DA_DTYPE_BF16)
    cache = {k: torch.empty(pages * page_bytes, dtype=torch.uint8, device="cuda") for k in "kv"}
    if fp4:
        cache |= dict(k_scale=torch.full((hkv,), 0.003, device="cuda"), v_scale=torch.full((hkv,), 0.004, device="cuda"))
    gen = torch.Generator().manual_seed(1)
    n = 100
    table = torch.tensor([[pages - 1 - 3 * i for i in range(8)]], dtype=torch.int32)
    slots = torch.tensor([int(table[0, i // page]) * page + i % page for i in range(n)])
    x = torch.randn(n, 2 * hkv, 128, generator=gen).to(torch.bfloat16).cuda()
    k_new, v_new = x[:, :hkv].contiguous(), x[:, hkv:].contiguous()
    eng.append(cache | dict(k_new=k_new, v_new=v_new, slot_map=slots.cuda()))
    out = {k: torch.zeros(n, hkv, 128, dtype=torch.bfloat16, device="cuda") for k in ("k_out", "v_out")}
    k, v = eng.gather(cache | out | dict(slot_map=slots.cuda()))
    if not fp4:
        assert torch.equal(k, k_new) and torch.equal(v, v_new)
    q = torch.randn(1, 16, 128, generator=gen).to(torch.bfloat16).cuda()
    lse = torch.zeros(1, 16, device="cuda")
    got = eng.run(cache | dict(q=q, block_table=table.cuda(), seq_lens=torch.tensor([n], dtype=torch.int32, device="cuda")),
                  SCALE, lse=lse)
    assert eng.errors() == 0
    k, v = k.cpu().double(), v.cpu().double()
    for h in range(16):
        # the read-back rows are the cached values rounded to bf16 (2^-8): a score moves by at most
        # 2^-8 scale sum|q k|, the output by that share and 2^-8 for the values' own rounding, and is
        # itself rounded (2^-8); weights are rounded to f16 or bf16 (2^-8)
        s = k[:, h // 2] @ q[0, h].cpu().double() * SCALE
        size = (k[:, h // 2].abs() @ q[0, h].cpu().double().abs()).max().item() * SCALE
        w = torch.softmax(s, 0)
        mag = (w @ v[:, h // 2].abs())
        tol = (2 * 2.0 ** -8 * size + 3 * 2.0 ** -8) * mag
        assert ((got[0, h].cpu().double() - w @ v[:, h // 2]).abs() <= tol).all()


def test_two_decodes_at_once_on_two_streams():
    cases = []
    for i in range(2):
        t = R.make(lens=[900 + 300 * i, 40, 1500], hq=8, hkv=2, page=16, seed=50 + i)
        eng = engine(t, hq=8, hkv=2, page=16)
        want = run(eng, t)
        cases.append((eng, {k: v.cuda() for k, v in t.items()}, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for eng, dev, want, s in cases:
            with torch.cuda.stream(s):
                out, lse = torch.zeros_like(dev["q"]), torch.zeros(3, 8, device="cuda")
                eng.run(dev, SCALE, out=out, lse=lse)
                got.append((out, lse, want))
    torch.cuda.synchronize()
    for out, lse, (o, l) in got:
        assert torch.equal(out, o) and torch.equal(lse, l)
    assert all(eng.errors() == 0 for eng, *_ in cases)


def test_two_graphs_that_share_a_workspace():
    t = R.make(lens=[2000, 17, 640], hq=8, hkv=2, page=16, seed=60)
    eng = engine(t, hq=8, hkv=2, page=16)
    want = run(eng, t)
    dev = {k: v.cuda() for k, v in t.items()}
    graphs, outs = [], []
    for _ in range(2):
        out, lse = torch.zeros_like(dev["q"]), torch.zeros(3, 8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            eng.run(dev, SCALE, out=out, lse=lse)
        graphs.append(g)
        outs.append((out, lse))
    for _ in range(5):  # one after the other, on one stream
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert eng.errors() == 0
    for out, lse in outs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("planned", [[1, 1, 1], [3000, 1, 1], [0, 0, 0]])
def test_lengths_that_outgrow_their_plan(planned):
    t = R.make(lens=[2900, 800, 33], hq=8, hkv=2, page=16, seed=70)
    kw = dict(batch=3, num_q_heads=8, num_kv_heads=2, head_dim_qk=128, head_dim_v=128, q_dtype=da.DA_DTYPE_BF16,
              kv_dtype=da.DA_DTYPE_FP4_E2M1_BLOCKS, kv_layout=da.DA_KV_PAGED, page_size=16, num_pages=t["k"].shape[0],
              max_pages_per_seq=t["block_table"].shape[1], max_seq_len=t["block_table"].shape[1] * 16)
    eng = da.DecodeAttention(device=0, seq_lens_host=torch.tensor(planned), **kw)
    out, lse = run(eng, t)
    assert eng.errors() == 0
    R.check(out, lse, R.reference(t, SCALE, hq=8, hkv=2, page=16))


def test_latent_queries_of_several_tokens():
    b, q_len = 3, 4
    eng = da.DecodeAttention(device=0, batch=b, num_q_heads=128, num_kv_heads=1, head_dim_qk=576, head_dim_v=512, is_mla=1,
                             ckv_dim=512, kpe_dim=64, kv_layout=da.DA_KV_PAGED, page_size=64, num_pages=4, max_pages_per_seq=4,
                             max_seq_len=256, q_dtype=da.DA_DTYPE_BF16, kv_dtype=da.DA_DTYPE_BF16, q_len=q_len)
    gen = torch.Generator().manual_seed(3)
    n = b * q_len
    q = torch.randn(n, 128, 64, generator=gen).to(torch.bfloat16).cuda()
    a = torch.randn(50, 32, generator=gen)
    table = torch.cat([a.cos(), a.sin()], -1).cuda()
    pos = torch.randint(0, 50, (n,), generator=gen).int().cuda()
    flat, laid = torch.zeros_like(q), torch.zeros(b, 128, q_len, 64, dtype=torch.bfloat16, device="cuda")
    eng.append(dict(q=q, q_out=flat, cos_sin=table, positions=pos))
    eng.append(dict(q=q, q_out=laid, cos_sin=table, positions=pos), q_len=q_len)
    assert eng.errors() == 0
    assert torch.equal(laid.transpose(1, 2).reshape(n, 128, 64), flat) and not torch.equal(flat, q)


def test_a_misaligned_output_is_refused():
    t = R.make(lens=[20], hq=4, hkv=1, page=16, seed=80)
    eng = engine(t, hq=4, hkv=1, page=16)
    dev = {k: v.cuda() for k, v in t.items()}
    room = torch.zeros(4 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(da.DecodeAttnError) as e:
        eng.run(dev, SCALE, out=room[4:4 + 512].view(1, 4, 128))
    assert e.value.status == da.DA_ERR_INVALID_ARG


def test_one_row_of_many_new_tokens():
    n, page = 200_000, 16
    pages = n // page + 10
    eng = da.DecodeAttention(device=0, batch=1, num_q_heads=1, num_kv_heads=1, head_dim_qk=128, head_dim_v=128,
                             kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=pages, max_pages_per_seq=pages,
                             max_seq_len=pages * page, q_dtype=da.DA_DTYPE_BF16, kv_dtype=da.DA_DTYPE_BF16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int().cuda()
    lens, nf = i32([5]), i32([pages - 1])
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = free[pages - 1]
    t = dict(seq_lens=lens, new_lens=i32([n]), seq_lens_out=lens, free_pages=free, num_free=nf, num_free_out=nf,
             block_table=table, slot_map=torch.zeros(n, dtype=torch.int64, device="cuda"),
             positions=torch.zeros(n, dtype=torch.int32, device="cuda"))
    eng.build_tables(t)
    assert eng.errors() == 0 and lens.item() == n + 5
    used = -(-(n + 5) // page) - 1
    assert nf.item() == pages - 1 - used
    pos = torch.arange(5, n + 5, device="cuda")
    assert torch.equal(t["positions"].long(), pos)
    assert torch.equal(table[0, 1:1 + used], free[:pages - 1].flip(0)[:used])
    assert torch.equal(t["slot_map"], table[0, pos // page].long() * page + pos % page)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 40, 3000])
def test_every_call_reads_what_the_one_before_wrote(kind, n):
    """The same rows written and read back over and over, nothing waited for in between: a call
    that starts early must not see what an SM had of a row from the call before the last."""
    steps, hkv = 60, 2
    dtype = da.DA_DTYPE_BF16 if kind == "bf16" else da.DA_DTYPE_FP8_E4M3
    eng = da.DecodeAttention(device=0, batch=1, num_q_heads=2, num_kv_heads=hkv, head_dim_qk=128, head_dim_v=128,
                             q_dtype=da.DA_DTYPE_BF16, kv_dtype=dtype, kv_layout=da.DA_KV_PAGED, page_size=16,
                             num_pages=200, max_pages_per_seq=200, max_seq_len=3200)
    kb, vb, _ = eng._cache_sizes()
    cache = dict(k=torch.zeros(kb, dtype=torch.uint8, device="cuda"), v=torch.zeros(vb, dtype=torch.uint8, device="cuda"))
    if kind != "bf16":
        cache |= dict(k_scale=torch.ones(hkv, device="cuda"), v_scale=torch.ones(hkv, device="cuda"))
    value = [(1 + i % 16) * (-1) ** (i // 16) for i in range(steps)]  # exact in e4m3
    x = torch.tensor(value, dtype=torch.bfloat16, device="cuda")[:, None, None, None].expand(steps, n, hkv, 128).contiguous()
    maps = [torch.randperm(3200, generator=torch.Generator().manual_seed(s))[:n].cuda() for s in range(2)]
    out = torch.zeros(2, steps, n, hkv, 128, dtype=torch.bfloat16, device="cuda")

    def loop():
        for i in range(steps):
            slots = maps[i % 3 == 0]
            eng.append(cache | dict(k_new=x[i], v_new=-x[i], slot_map=slots))
            eng.gather(cache | dict(slot_map=slots, k_out=out[0, i], v_out=out[1, i]))

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        loop()
    for go in (loop, graph.replay, graph.replay):
        out.zero_()
        go()
        torch.cuda.synchronize()
        assert eng.errors() == 0
        assert torch.equal(out[0], x) and torch.equal(out[1], -x)
