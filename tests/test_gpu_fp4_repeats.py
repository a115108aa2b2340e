"""The same call gives the same bits, whatever order the blocks of a launch finish in."""

import pytest
import torch

import decode_attention_flash_gb300 as da

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,q_len", [(16, 1), (20, 1), (32, 1), (48, 1), (16, 4)])
@pytest.mark.parametrize("b", [38, 11])
def test_a_decode_repeats_itself(hq, q_len, b):
    """152 or 44 units that end inside the ranges of blocks: most are the sum of two to four blocks'
    pieces, made by the block that comes last, which may be last for two units at once, or for one."""
    hkv, page, cols = 4, 64, 60
    gen = torch.Generator().manual_seed(hq)
    pages = b * cols
    kw = dict(batch=b, num_q_heads=hq, num_kv_heads=hkv, head_dim_qk=128, head_dim_v=128, q_dtype=da.DA_DTYPE_BF16,
              kv_dtype=da.DA_DTYPE_FP4_E2M1_BLOCKS, kv_layout=da.DA_KV_PAGED, page_size=page, num_pages=pages,
              max_pages_per_seq=cols, max_seq_len=cols * page, q_len=q_len)
    eng = da.DecodeAttention(device=0, **kw)
    assert eng.plan["writes_final"] == 0
    t = dict(block_table=torch.randperm(pages, generator=gen).int().view(b, cols).cuda(),
             seq_lens=torch.randint(2500, 3800, (b,), generator=gen).int().cuda())
    for n in "kv":
        raw = torch.randint(0, 256, (pages, hkv, page // 16, 1152), dtype=torch.uint8, generator=gen)
        raw[..., 1024:] &= 0x3F  # scales below 2
        t[n], t[n + "_scale"] = raw.cuda(), torch.full((hkv,), 0.1, device="cuda")
    lead = (b, hq, q_len) if q_len > 1 else (b, hq)
    t["q"] = torch.randn(*lead, 128, generator=gen).to(torch.bfloat16).cuda()
    outs = torch.zeros(24, *lead, 128, dtype=torch.bfloat16, device="cuda")
    lses = torch.zeros(24, *lead, device="cuda")
    other = torch.zeros(1 << 24, device="cuda")
    for i in range(24):
        if i % 2:  # with and without other work before it
            other[: 1 << (i % 24)].add_(1.0)
        eng.run(t, 128 ** -0.5, out=outs[i], lse=lses[i])
    torch.cuda.synchronize()
    assert eng.errors() == 0
    assert torch.isfinite(outs.float()).all()
    assert all(torch.equal(outs[i], outs[0]) and torch.equal(lses[i], lses[0]) for i in range(24))
