"""One forced split over a 4-bit float cache needs no more than the workspace's header."""

import pytest
import torch

import decode_attention_flash_gb300 as da
import fp4_ref as R
from test_gpu_fp4 import SCALE, engine

pytestmark = pytest.mark.gpu
LENS = [1, 0, 33, 700, 1200, 64]


@pytest.mark.parametrize("hq,hkv,q_len", [(8, 2, 1), (32, 2, 1), (40, 2, 1), (8, 2, 4)])
@pytest.mark.parametrize("page", [16, 64, 0])
def test_nothing_behind_the_header_is_written(hq, hkv, q_len, page):
    t = R.make(lens=LENS, hq=hq, hkv=hkv, page=page, q_len=q_len, seed=hq)
    eng = engine(t, hq=hq, hkv=hkv, page=page, q_len=q_len, splits=1)
    assert eng.workspace.numel() == 256 and eng.plan["writes_final"] == 1
    room = torch.full((1 << 20,), 0x5A, dtype=torch.uint8, device="cuda")
    room[:256] = 0
    dev = {k: v.cuda() for k, v in t.items()}
    out, lse = torch.zeros(t["q"].shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(t["q"].shape[:-1], device="cuda")
    da.decode_attn_run(eng.ctx, da.make_args(dev, SCALE, out, lse), room[:256])
    torch.cuda.synchronize()
    assert da.decode_attn_get_error(eng.ctx, room[:256]) == 0
    assert (room[256:] == 0x5A).all() and (room[:256] == 0).all()
    R.check(out, lse, R.reference(t, SCALE, hq=hq, hkv=hkv, page=page, q_len=q_len))


def test_many_rows_without_allocation():
    # 1024 rows of 64 / 8 heads: 547 MB of pieces that no block writes
    lens = [(7 * i) % 41 for i in range(1024)]
    t = R.make(lens=lens, hq=64, hkv=8, page=16, seed=3)
    eng = engine(t, hq=64, hkv=8, page=16, splits=1)
    dev = {k: v.cuda() for k, v in t.items()}
    out, lse = torch.zeros(1024, 64, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1024, 64, device="cuda")
    da.decode_attn_run_noalloc(eng.ctx, da.make_args(dev, SCALE, out, lse))
    torch.cuda.synchronize()
    assert da.decode_attn_get_error_noalloc(eng.ctx) == 0
    some = torch.arange(0, 1024, 97)
    pick = t | dict(q=t["q"][some], seq_lens=t["seq_lens"][some], block_table=t["block_table"][some])
    R.check(out[some.cuda()], lse[some.cuda()], R.reference(pick, SCALE, hq=64, hkv=8, page=16))


def test_a_wait_that_gives_up_leaves_the_header_clean():
    t = R.make(lens=LENS, hq=8, hkv=2, page=16, seed=5)
    eng = engine(t, hq=8, hkv=2, page=16, splits=1)
    dev = {k: v.cuda() for k, v in t.items()}
    out, lse = torch.zeros(t["q"].shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(t["q"].shape[:-1], device="cuda")
    assert da.load().decode_attn_test_set_stall(eng.ctx, 200_000) == da.DA_OK  # 0.2 ms
    eng.run(dev, SCALE, out=out, lse=lse)
    assert eng.errors() & da.DA_DEVERR_TIMEOUT
    assert (eng.workspace == 0).all()
    eng.run(dev, SCALE, out=out, lse=lse)
    assert eng.errors() == 0
    R.check(out, lse, R.reference(t, SCALE, hq=8, hkv=2, page=16))
