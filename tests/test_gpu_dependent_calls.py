"""Serving steps with nothing waited for in between: tables with lengths in place, queries
turned in place, then the decode, which may start on an SM while the append is still
reading there. A twin with buffers of its own, waited for after every call, says what each
step has to give, bit for bit; the last step is held against 64 bits too."""

import pytest
import torch

import decode_attention_flash_gb300 as da
import fp4_ref as R

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
B, HQ, HKV, PAGE, COLS, PAGES = 6, 16, 2, 16, 64, 300
STEPS = 25


def engine(kind):
    dtype = da.DA_DTYPE_FP4_E2M1_BLOCKS if kind == "fp4" else da.DA_DTYPE_BF16
    return da.DecodeAttention(device=0, batch=B, num_q_heads=HQ, num_kv_heads=HKV, head_dim_qk=128, head_dim_v=128,
                              kv_layout=da.DA_KV_PAGED, page_size=PAGE, max_seq_len=COLS * PAGE, max_pages_per_seq=COLS,
                              num_pages=PAGES, q_dtype=da.DA_DTYPE_BF16, kv_dtype=dtype)


def state(kind, eng, capacity):
    size = eng._cache_sizes()[0]
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(k=torch.zeros(size, dtype=torch.uint8, device="cuda"), v=torch.zeros(size, dtype=torch.uint8, device="cuda"),
             seq_lens=i32(B), block_table=i32(B, COLS), num_free=i32(1), positions=i32(capacity),
             slot_map=torch.zeros(capacity, dtype=torch.int64, device="cuda"),
             free_pages=torch.randperm(PAGES, generator=torch.Generator().manual_seed(3)).int().cuda())
    if kind == "fp4":
        s |= {n: torch.full((HKV,), 0.003, device="cuda") for n in ("k_scale", "v_scale")}
    return s | dict(seq_lens_out=s["seq_lens"], num_free_out=s["num_free"])


def reset(s):
    for n in ("k", "v", "seq_lens", "block_table"):
        s[n].zero_()
    s["num_free"].fill_(PAGES)


def steps_of():
    gen = torch.Generator().manual_seed(5)
    new = torch.randint(0, 12, (STEPS, B), generator=gen).int()
    new[3] = 0
    n = int(new.sum(1).max())
    qkv = torch.randn(STEPS, n, HQ + 2 * HKV, 128, generator=gen).to(torch.bfloat16)
    return new.cuda(), qkv.cuda(), n


def table():
    inv = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    a = torch.arange(COLS * PAGE, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], -1).float().cuda()


@pytest.mark.parametrize("kind", ["fp4", "bf16"])
# (more slots than tokens put a block of the tables, which reads the lengths, on one SM or on all)
@pytest.mark.parametrize("capacity", [0, 80000])
def test_steps_in_place_with_nothing_waited_for(kind, capacity):
    new, qkv, n = steps_of()
    capacity = max(capacity, n)
    cos_sin = table()
    fast, slow = engine(kind), engine(kind)
    a, b = state(kind, fast, capacity), state(kind, slow, capacity)
    q = torch.zeros(max(n, B), HQ, 128, dtype=torch.bfloat16, device="cuda")
    outs = torch.zeros(2, STEPS, B, HQ, 128, dtype=torch.bfloat16, device="cuda")
    turned = torch.zeros(2, STEPS, n, HQ, 128, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(2, 2, STEPS, n, HKV, 128, dtype=torch.bfloat16, device="cuda")
    x = [(qkv[i, :, :HQ], qkv[i, :, HQ:HQ + HKV], qkv[i, :, HQ + HKV:]) for i in range(STEPS)]

    def loop():
        for i in range(STEPS):
            q[:n].copy_(x[i][0])
            fast.build_tables(a | dict(new_lens=new[i]))
            some = dict(slot_map=a["slot_map"][:n], positions=a["positions"][:n])
            fast.append(a | some | dict(q=q[:n], q_out=q[:n], k_new=x[i][1], v_new=x[i][2], cos_sin=cos_sin))
            fast.run(a | dict(q=q[:B]), SCALE, out=outs[0, i])
            fast.gather(a | some | dict(k_out=rows[0, 0, i], v_out=rows[0, 1, i]))
            turned[0, i].copy_(q[:n])

    reset(b)
    for i in range(STEPS):
        torch.cuda.synchronize()
        slow.build_tables(b | dict(new_lens=new[i]))
        torch.cuda.synchronize()
        some = dict(slot_map=b["slot_map"][:n].clone(), positions=b["positions"][:n].clone())
        mine = x[i][0].contiguous().clone()  # (tokens without a slot keep their rows)
        torch.cuda.synchronize()
        slow.append(b | some | dict(q=x[i][0], q_out=mine, k_new=x[i][1], v_new=x[i][2], cos_sin=cos_sin))
        torch.cuda.synchronize()
        slow.run(b | dict(q=mine[:B].clone()), SCALE, out=outs[1, i])
        torch.cuda.synchronize()
        slow.gather(b | some | dict(k_out=rows[1, 0, i], v_out=rows[1, 1, i]))
        turned[1, i].copy_(mine)
    torch.cuda.synchronize()
    assert slow.errors() == 0 and b["seq_lens"].tolist() == new.sum(0).tolist()
    if kind == "fp4":
        t = {k: b[k].cpu() for k in ("k_scale", "v_scale", "seq_lens", "block_table")}
        t |= {k: b[k].cpu().view(PAGES, HKV, 1, 1152) for k in "kv"} | dict(q=turned[1, -1, :B].cpu())
        out, _, tol, _ = R.reference(t, SCALE, hq=HQ, hkv=HKV, page=PAGE)
        assert ((outs[1, -1].cpu().double() - out[:, :, 0]).abs() <= tol[:, :, 0]).all()

    reset(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop()
    for go in (loop, loop, graph.replay, graph.replay):
        for y in (outs, turned, rows):
            y[0].zero_()
        reset(a)
        go()
        torch.cuda.synchronize()
        assert fast.errors() == 0
        assert torch.equal(a["seq_lens"], b["seq_lens"]) and torch.equal(a["block_table"], b["block_table"])
        for name, y in (("queries", turned), ("rows", rows), ("outputs", outs)):
            assert torch.equal(y[0], y[1]), name


@pytest.mark.parametrize("capacity", [16, 80000])
def test_tables_then_the_decode(capacity):
    """The decode right behind the tables: lengths and pages as they have just become."""
    eng, ref = engine("fp4"), engine("fp4")
    gen = torch.Generator().manual_seed(9)
    new = torch.randint(0, 40, (STEPS, B), generator=gen).int()
    new = new.clamp(max=2).cuda() if capacity == 16 else new.cuda()
    a = state("fp4", eng, capacity)
    raw = [torch.randint(0, 256, (PAGES, HKV, 1152), generator=gen).to(torch.uint8) for _ in "kv"]
    for r in raw:  # any codes, scales below 2
        r[..., 1024:] &= 0x3F
    q = torch.randn(STEPS, B, HQ, 128, generator=gen).to(torch.bfloat16).cuda()
    out = torch.zeros(2, STEPS, B, HQ, 128, dtype=torch.bfloat16, device="cuda")

    def loop(e, k, wait):
        for i in range(STEPS):
            e.build_tables(a | dict(new_lens=new[i]))
            if wait:
                torch.cuda.synchronize()
            lens = a["seq_lens"].clone() if wait else a["seq_lens"]
            tab = a["block_table"].clone() if wait else a["block_table"]
            if wait:
                torch.cuda.synchronize()
            e.run(a | dict(seq_lens=lens, block_table=tab, q=q[i]), SCALE, out=out[k, i])
            if wait:
                torch.cuda.synchronize()

    def start():
        reset(a)
        for n, r in zip("kv", raw):
            a[n].copy_(r.flatten())
        out[0].zero_()
        torch.cuda.synchronize()

    start()
    loop(ref, 1, True)
    assert ref.errors() == 0
    graph = torch.cuda.CUDAGraph()
    start()
    with torch.cuda.graph(graph):
        loop(eng, 0, False)
    for go in (lambda: loop(eng, 0, False), graph.replay, graph.replay):
        start()
        go()
        torch.cuda.synchronize()
        assert eng.errors() == 0 and a["seq_lens"].tolist() == new.sum(0).tolist()
        assert torch.equal(out[0], out[1])
