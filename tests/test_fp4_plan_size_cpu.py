"""The workspace of a 4-bit float plan holds what its kernel writes there: with one forced
split every unit has a block of its own, no piece leaves a block, and the header is all."""

import pytest

import decode_attention_flash_gb300 as da

NOALLOC = 32 << 20


def plan(lens, batch, hq, hkv, splits, **more):
    kw = dict(batch=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim_qk=128, head_dim_v=128,
              kv_dtype=da.DA_DTYPE_FP4_E2M1_BLOCKS, kv_layout=da.DA_KV_PAGED, num_pages=100000, max_pages_per_seq=100,
              page_size=16, max_seq_len=1600)
    return da.decode_attn_plan_info(da.make_problem(**(kw | more)), 152, lens, splits)


@pytest.mark.parametrize("batch,hq,hkv", [(1, 4, 1), (1024, 64, 8), (4000, 128, 8), (8000, 64, 8), (3, 128, 1)])
@pytest.mark.parametrize("lens", [None, 40])
def test_one_forced_split_takes_the_header(batch, hq, hkv, lens):
    da.load(build_if_missing=True)
    p = plan(None if lens is None else [lens] * batch, batch, hq, hkv, 1)
    assert p["writes_final"] == 1 and p["grid_x"] == p["num_units"]
    assert p["workspace_bytes"] == 256 <= NOALLOC
    assert p["counters_offset"] == p["partial_o_offset"] == p["partial_lse_offset"] == 256


def test_other_plans_keep_their_pieces():
    da.load(build_if_missing=True)
    for splits in (0, 2, 3):
        p = plan([40, 2000], 2, 32, 8, splits)
        pieces = (p["num_units"] + p["grid_x"]) * p["rows_per_unit"]
        assert p["partial_lse_offset"] - p["partial_o_offset"] >= pieces * 512
        assert p["workspace_bytes"] >= p["partial_lse_offset"] + pieces * 4 + p["grid_x"] * 15 * p["rows_per_unit"] * 512
    # more units than a grid holds are shared among 1024 blocks, split or not
    p = plan(None, 9000, 64, 8, 1)
    assert p["writes_final"] == 0 and p["grid_x"] == 1024 and p["workspace_bytes"] > 9000 * 8 * 8 * 512
