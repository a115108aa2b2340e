"""Calls on two streams that wait for each other by events, eagerly and captured as a graph with
branches: a kernel launched as a dependent of its own stream's last kernel waits for the
other stream's as well."""

import pytest
import torch

import decode_attention_flash_gb300 as da

pytestmark = pytest.mark.gpu
STEPS, N, HKV, PAGES = 30, 3000, 2, 200


@pytest.mark.parametrize("between", ["nothing", "kernel", "copy"])
def test_append_on_one_stream_and_read_back_on_another(between):
    eng = da.DecodeAttention(device=0, batch=1, num_q_heads=2, num_kv_heads=HKV, head_dim_qk=128, head_dim_v=128,
                             q_dtype=da.DA_DTYPE_BF16, kv_dtype=da.DA_DTYPE_BF16, kv_layout=da.DA_KV_PAGED, page_size=16,
                             num_pages=PAGES, max_pages_per_seq=PAGES, max_seq_len=PAGES * 16)
    size = eng._cache_sizes()[0]
    cache = {n: torch.zeros(size, dtype=torch.uint8, device="cuda") for n in "kv"}
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(STEPS, N, HKV, 128, generator=gen).to(torch.bfloat16).cuda()
    maps = torch.stack([torch.randperm(PAGES * 16, generator=gen)[:N] for _ in range(STEPS)]).cuda()
    slots = torch.zeros(N, dtype=torch.int64, device="cuda")
    out = torch.zeros(2, STEPS, N, HKV, 128, dtype=torch.bfloat16, device="cuda")
    scrap = torch.zeros(2, 1 << 20, device="cuda")
    other = torch.cuda.Stream()

    def loop():
        main = torch.cuda.current_stream()
        for i in range(STEPS):
            slots.copy_(maps[i])  # (a copy, not a kernel)
            if between == "kernel":
                scrap[0].add_(1.0)
            eng.append(cache | dict(k_new=x[i], v_new=-x[i], slot_map=slots))
            other.wait_stream(main)
            with torch.cuda.stream(other):
                if between == "kernel":
                    scrap[1].add_(1.0)
                if between == "copy":
                    scrap[1, : 1 << 19].copy_(scrap[1, 1 << 19:])
                eng.gather(cache | dict(slot_map=slots, k_out=out[0, i], v_out=out[1, i]))
            main.wait_stream(other)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop()
    for go in (loop, loop, graph.replay, graph.replay):
        out.zero_()
        for n in "kv":
            cache[n].zero_()
        torch.cuda.synchronize()
        go()
        torch.cuda.synchronize()
        assert eng.errors() == 0
        assert torch.equal(out[0], x) and torch.equal(out[1], -x)


def test_two_branches_that_meet():
    """Two appends on two streams, then one read-back that waits for both."""
    engs = [da.DecodeAttention(device=0, batch=1, num_q_heads=2, num_kv_heads=HKV, head_dim_qk=128, head_dim_v=128,
                               q_dtype=da.DA_DTYPE_BF16, kv_dtype=da.DA_DTYPE_BF16, kv_layout=da.DA_KV_PAGED, page_size=16,
                               num_pages=PAGES, max_pages_per_seq=PAGES, max_seq_len=PAGES * 16) for _ in range(2)]
    size = engs[0]._cache_sizes()[0]
    cache = {n: torch.zeros(size, dtype=torch.uint8, device="cuda") for n in "kv"}
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(STEPS, N, HKV, 128, generator=gen).to(torch.bfloat16).cuda()
    slots = torch.randperm(PAGES * 16, generator=gen)[:N].cuda()
    out = torch.zeros(2, STEPS, N, HKV, 128, dtype=torch.bfloat16, device="cuda")
    other = torch.cuda.Stream()
    h = N // 2 + 7

    def loop():
        main = torch.cuda.current_stream()
        for i in range(STEPS):
            other.wait_stream(main)
            with torch.cuda.stream(other):
                engs[1].append(cache | dict(k_new=x[i, h:], v_new=-x[i, h:], slot_map=slots[h:]))
            engs[0].append(cache | dict(k_new=x[i, :h], v_new=-x[i, :h], slot_map=slots[:h]))
            main.wait_stream(other)
            engs[0].gather(cache | dict(slot_map=slots, k_out=out[0, i], v_out=out[1, i]))

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop()
    for go in (loop, loop, graph.replay, graph.replay):
        out.zero_()
        torch.cuda.synchronize()
        go()
        torch.cuda.synchronize()
        assert engs[0].errors() == 0 and engs[1].errors() == 0
        assert torch.equal(out[0], x) and torch.equal(out[1], -x)
