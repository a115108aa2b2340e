"""Blocks started anew and read at once, over and over with nothing waited for: every decode has to see the scale
that the append just before it wrote, on whatever SM, though an earlier decode there read the old one. The values are
small integers times a power of two, which both kinds of code hold exactly, and one position a row is its own mean, so
outputs are compared bit for bit."""

import pytest
import torch

import block8_ref as B
import decode_attention_flash_gb300 as da

pytestmark = pytest.mark.gpu
ROWS, HKV, PAGE, STEPS = 230, 8, 16, 60


def setup(kind, q_heads, block=16):
    eng = da.DecodeAttention(device=0, batch=ROWS, num_q_heads=q_heads, num_kv_heads=HKV, head_dim_qk=128, head_dim_v=128,
                             kv_layout=da.DA_KV_PAGED, page_size=PAGE, num_pages=ROWS, max_pages_per_seq=1, max_seq_len=PAGE,
                             kv_dtype=B.KINDS[kind], kv_groups=block)
    gen = torch.Generator().manual_seed(1)
    cache = {s: torch.zeros(ROWS, HKV, PAGE, 128, dtype=B.DTYPE[kind], device="cuda") for s in ("k", "v")}
    cache |= {s + "_scale": torch.zeros(ROWS, HKV, PAGE // block, device="cuda") for s in ("k", "v")}
    t = dict(block_table=torch.randperm(ROWS, generator=gen).int()[:, None].contiguous().cuda(),
             seq_lens=torch.ones(ROWS, dtype=torch.int32, device="cuda"),
             q=torch.randn(ROWS, q_heads, 128, generator=gen).to(torch.bfloat16).cuda())
    rows = torch.randint(-8, 9, (STEPS, ROWS, HKV, 128), generator=gen).float()
    rows[..., 0] = 8
    size = torch.exp2(torch.randint(-6, 7, (STEPS, ROWS, HKV, 1), generator=gen).float())
    new = (rows * size).to(torch.bfloat16).cuda()
    out = torch.zeros(STEPS, ROWS, q_heads, 128, dtype=torch.bfloat16, device="cuda")
    slots = t["block_table"][:, 0].long() * PAGE
    appends = [da.make_append_args({**cache, "k_new": new[i], "v_new": new[i], "slot_map": slots}) for i in range(STEPS)]
    runs = [da.make_args({**cache, **t}, 128 ** -0.5, out[i]) for i in range(STEPS)]
    return eng, appends, runs, new, out, (cache, t, slots)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [1, 16])
@pytest.mark.parametrize("captured", [False, True])
def test_every_decode_sees_the_scales_just_written(kind, group, captured):
    eng, appends, runs, new, out, alive = setup(kind, HKV * group)

    def steps():
        for a, r in zip(appends, runs):
            da.decode_attn_append(eng.ctx, a, eng.workspace)
            da.decode_attn_run(eng.ctx, r, eng.workspace)

    steps()
    torch.cuda.synchronize()
    if captured:
        out.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            steps()
        for _ in range(5):
            g.replay()
        torch.cuda.synchronize()
    assert eng.errors() == 0
    want = new.repeat_interleave(group, 2)
    assert torch.equal(out, want), f"{int((out != want).sum())} of {out.numel()}"
    assert alive
