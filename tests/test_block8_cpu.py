"""Problems of the 8-bit block cache that are accepted and refused, and their plans (host only)."""

import pytest

import decode_attention_flash_gb300 as da

KINDS = [da.DA_DTYPE_FP8_E4M3_BLOCKS, da.DA_DTYPE_INT8_BLOCKS]


def plan(kind, block, lens=None, splits=0, **more):
    da.load(build_if_missing=True)
    kw = dict(batch=4, num_q_heads=32, num_kv_heads=8, head_dim_qk=128, head_dim_v=128, kv_dtype=kind, kv_groups=block,
              kv_layout=da.DA_KV_PAGED, page_size=64, num_pages=1000, max_pages_per_seq=100, max_seq_len=6400)
    return da.decode_attn_plan_info(da.make_problem(**(kw | more)), 152, lens, splits)


def status(*a, **kw):
    with pytest.raises(da.DecodeAttnError) as e:
        plan(*a, **kw)
    return e.value.status


@pytest.mark.parametrize("kind", KINDS)
def test_blocks_that_divide_a_page(kind):
    for page in (16, 32, 64, 128, 192, 256, 512):
        for block in (16, 32, 64, 128, 256):
            kw = dict(page_size=page, max_seq_len=100 * page)
            if page % block == 0:
                assert plan(kind, block, **kw)["workspace_bytes"] > 0
            else:
                assert status(kind, block, **kw) == da.DA_ERR_INVALID_ARG


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block", [0, 1, 8, 24, 48, 512, -16])
def test_other_blocks_are_refused(kind, block):
    assert status(kind, block, page_size=512 * 3, max_seq_len=0) == da.DA_ERR_INVALID_ARG


@pytest.mark.parametrize("kind", KINDS)
def test_contiguous_lengths(kind):
    kw = dict(kv_layout=da.DA_KV_CONTIGUOUS, page_size=0, num_pages=0, max_pages_per_seq=0)
    assert plan(kind, 16, max_seq_len=4080, **kw)["num_units"] == 32
    assert status(kind, 32, max_seq_len=4080, **kw) == da.DA_ERR_INVALID_ARG
    assert status(kind, 16, max_seq_len=4088, **kw) == da.DA_ERR_INVALID_ARG


@pytest.mark.parametrize("kind", KINDS)
def test_other_refusals(kind):
    assert status(kind, 16, head_dim_qk=64) == da.DA_ERR_UNSUPPORTED
    assert status(kind, 16, num_q_heads=40, num_kv_heads=8, q_len=4) == da.DA_ERR_UNSUPPORTED  # 20 rows a head
    assert status(kind, 16, num_q_heads=256, num_kv_heads=1) == da.DA_ERR_UNSUPPORTED
    assert status(kind, 16, fp8_mma=1) == da.DA_ERR_UNSUPPORTED
    assert status(kind, 16, max_pages_per_seq=1 << 26, max_seq_len=0) == da.DA_ERR_UNSUPPORTED  # 2^32 positions
    assert status(kind, 16, batch=1 << 20, max_pages_per_seq=1 << 20, max_seq_len=0) == da.DA_ERR_UNSUPPORTED
    assert plan(kind, 16, num_q_heads=128, num_kv_heads=1)["num_units"] == 32  # 8 passes of 16 rows


@pytest.mark.parametrize("kind", KINDS)
def test_plans_keep_their_pieces(kind):
    one = plan(kind, 16, [40] * 4, splits=1)
    assert one["writes_final"] == 1 and one["grid_x"] == 32 and one["workspace_bytes"] == 256
    p = plan(kind, 16, [6000] * 4)
    pieces = (p["num_units"] + p["grid_x"]) * p["rows_per_unit"]
    assert p["partial_lse_offset"] - p["partial_o_offset"] >= pieces * 512
    assert p["workspace_bytes"] >= p["partial_lse_offset"] + pieces * 4 + p["grid_x"] * p["rows_per_unit"] * 512
