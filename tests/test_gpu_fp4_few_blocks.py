"""Few blocks for many ragged units of a 4-bit float cache: a plan made for hardly any token has a
block or a few, and the lengths that come then lay several units, their heads and their tails
into the range of one warp."""

import pytest
import torch

import decode_attention_flash_gb300 as da
import fp4_ref as R
from test_gpu_fp4 import SCALE, run

pytestmark = pytest.mark.gpu
ROWS = [[333, 64, 1200, 31, 95, 2, 800], [1, 2, 3, 0, 5, 6, 0], [2000, 0, 0, 1, 0, 33, 32], [640, 640, 640, 640, 640, 640, 640],
        [17, 900, 18, 900, 19, 900, 20]]


def few(t, planned, *, hq, hkv, page, q_len=1):
    """An engine planned for `planned`, two splits asked for (so that no unit has a block of its own)."""
    cols = t["block_table"].shape[1]
    return da.DecodeAttention(device=0, seq_lens_host=torch.tensor(planned), num_splits_override=2, batch=len(planned),
                              num_q_heads=hq, num_kv_heads=hkv, head_dim_qk=128, head_dim_v=128, q_dtype=da.DA_DTYPE_BF16,
                              kv_dtype=da.DA_DTYPE_FP4_E2M1_BLOCKS, q_len=q_len, kv_layout=da.DA_KV_PAGED, page_size=page,
                              num_pages=t["k"].shape[0], max_pages_per_seq=cols, max_seq_len=cols * page)


@pytest.mark.parametrize("lens", ROWS)
@pytest.mark.parametrize("hq,hkv,q_len", [(8, 1, 1), (12, 1, 1), (8, 2, 4), (2, 1, 1)])
@pytest.mark.parametrize("blocks", [1, 2, 3, 7])
def test_units_inside_the_ranges_of_warps(lens, hq, hkv, q_len, blocks):
    t = R.make(lens=lens, hq=hq, hkv=hkv, page=32, q_len=q_len, seed=len(lens) + hq)
    eng = few(t, [32] * blocks + [0] * (7 - blocks), hq=hq, hkv=hkv, page=32, q_len=q_len)
    assert eng.plan["grid_x"] == blocks * hkv and eng.plan["writes_final"] == 0 and eng.plan["num_units"] == 7 * hkv
    ref = R.reference(t, SCALE, hq=hq, hkv=hkv, page=32, q_len=q_len)
    for _ in range(2):  # the counters are back at zero
        out, lse = run(eng, t)
        assert eng.errors() == 0
        R.check(out, lse, ref)


@pytest.mark.parametrize("blocks", [1, 5])
def test_hundreds_of_units_in_a_block(blocks):
    gen = torch.Generator().manual_seed(blocks)
    lens = torch.randint(0, 70, (150,), generator=gen).tolist()
    lens[0] = 3000
    t = R.make(lens=lens, hq=4, hkv=2, page=16, seed=blocks)
    eng = few(t, [32] * blocks + [0] * (150 - blocks), hq=4, hkv=2, page=16)
    assert eng.plan["grid_x"] == 2 * blocks and eng.plan["writes_final"] == 0
    ref = R.reference(t, SCALE, hq=4, hkv=2, page=16)
    out, lse = run(eng, t)
    assert eng.errors() == 0
    R.check(out, lse, ref)
