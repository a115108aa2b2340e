"""CPU-side checks of the cache calls and of the 4-bit float cache: refusals that
need no device, the planner, the binding, and the tests' own 64-bit definitions
pinned by hand."""

import ctypes

import pytest
import torch

import decode_attention_flash_gb300 as da
import fp4_ref as R


@pytest.fixture(scope="module")
def lib():
    return da.load(build_if_missing=True)


FP4 = dict(batch=4, num_q_heads=8, num_kv_heads=2, head_dim_qk=128, head_dim_v=128,
           kv_dtype=da.DA_DTYPE_FP4_E2M1_BLOCKS)


def plan(lens=None, splits=0, **kw):
    return da.decode_attn_plan_info(da.make_problem(**(FP4 | kw)), 152, lens, splits)


def refused(**kw):
    with pytest.raises(da.DecodeAttnError) as e:
        plan(**kw)
    return e.value.status


def test_fp4_problems_are_validated(lib):
    paged = dict(kv_layout=da.DA_KV_PAGED, num_pages=100, max_pages_per_seq=10)
    for page in (16, 32, 64, 192):
        plan(**paged, page_size=page)
    assert refused(**paged, page_size=8) == da.DA_ERR_UNSUPPORTED
    plan(max_seq_len=208)
    assert refused(max_seq_len=200) == da.DA_ERR_UNSUPPORTED   # granules of 16 rows
    assert refused(max_seq_len=208, fp8_mma=1) == da.DA_ERR_UNSUPPORTED
    assert refused(max_seq_len=208, num_q_heads=34) == da.DA_ERR_UNSUPPORTED  # 17 rows a head
    assert refused(max_seq_len=208, num_q_heads=8, q_len=5) == da.DA_ERR_UNSUPPORTED
    assert refused(batch=4, num_q_heads=128, num_kv_heads=1, is_mla=1, ckv_dim=512, kpe_dim=64, head_dim_qk=576,
                   head_dim_v=512, **paged, page_size=64) == da.DA_ERR_UNSUPPORTED
    # positions and tiles are counted in 32 bits; rows beyond the tensor maps' limit are fine
    assert refused(**(paged | dict(max_pages_per_seq=1 << 27)), page_size=16) == da.DA_ERR_UNSUPPORTED
    plan(**(paged | dict(num_pages=1 << 27, max_pages_per_seq=1 << 20)), page_size=16)


def test_fp4_heads_of_many_queries_are_split(lib):
    for hq, units, rows in ((32, 2, 16), (20, 2, 10), (48, 4, 12), (64, 4, 16), (128, 8, 16)):
        got = plan([100], batch=1, num_q_heads=hq, num_kv_heads=1, max_seq_len=208)
        assert (got["num_units"], got["rows_per_unit"]) == (units, rows)
    for more in (dict(num_q_heads=19), dict(num_q_heads=144), dict(num_q_heads=32, q_len=2),
                 dict(num_q_heads=32, max_seq_len=256, sparse_block_size=64, max_sparse_blocks=4),
                 dict(num_q_heads=32, kv_dtype=da.DA_DTYPE_BF16)):
        assert refused(**(dict(batch=1, num_kv_heads=1, max_seq_len=208) | more)) == da.DA_ERR_UNSUPPORTED


def test_fp4_plan_takes_a_block_for_every_unit_where_that_is_shorter(lib):
    kw = dict(kv_layout=da.DA_KV_PAGED, num_pages=5000, max_pages_per_seq=1000, page_size=16)
    short = plan([700, 1, 64, 0], **kw)
    assert short["grid_x"] == short["num_units"] == 8 and short["writes_final"] == 1
    one_long = plan([9000, 1, 64, 0], **kw)
    assert one_long["grid_x"] == 152 and one_long["writes_final"] == 0
    many = plan([40] * 200, batch=200, **kw)   # more units than SMs
    assert many["grid_x"] == 152 and many["writes_final"] == 0
    assert plan(None, **kw)["writes_final"] == 0   # lengths not known
    assert plan([9000, 1, 64, 0], splits=1, **kw)["writes_final"] == 1
    assert plan([9000, 1, 64, 0], splits=3, **kw)["grid_x"] == 24
    for p in (short, one_long):
        units, ctas, rows = p["num_units"], p["grid_x"], p["rows_per_unit"]
        lse_end = p["partial_lse_offset"] + (units + ctas) * rows * 4
        assert p["workspace_bytes"] >= lse_end + ctas * 15 * rows * 512


def test_fp4_plan_has_no_more_pieces_than_two_levels_of_32_merge(lib):
    kw = dict(kv_layout=da.DA_KV_PAGED, num_pages=5000, max_pages_per_seq=5000, page_size=64)
    for splits in (1024, 1025, 4000, 1 << 30):
        assert plan([200000], batch=1, splits=splits, num_q_heads=4, num_kv_heads=1, **kw)["grid_x"] == 1024
    assert plan([200000, 5], batch=2, splits=1000, **kw)["grid_x"] == 1024
    assert plan([5] * 3000, batch=3000, splits=1, **kw)["grid_x"] == 6000  # a CTA a unit: nothing to merge


def test_calls_refuse_null_and_report_it(lib):
    for name, args in (("build_tables", da.TableArgs()), ("append", da.AppendArgs()), ("gather", da.GatherArgs())):
        fn = getattr(lib, "decode_attn_" + name)
        assert fn(None, ctypes.byref(args), None, 0, None) == da.DA_ERR_INVALID_ARG
        assert fn(None, None, None, 0, None) == da.DA_ERR_INVALID_ARG


def test_binding_refuses_wrong_tensors():
    i = torch.zeros(3, dtype=torch.int32)
    s = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="device memory"):
        da.make_table_args(dict(seq_lens=i, new_lens=i, seq_lens_out=i, slot_map=s))
    with pytest.raises(ValueError, match="int32"):
        da.make_table_args(dict(seq_lens=i.long(), new_lens=i, seq_lens_out=i, slot_map=s))
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device memory"):
        da.make_append_args(dict(k_new=x, v_new=x, slot_map=s))
    with pytest.raises(ValueError, match="rows"):
        da.make_gather_args(dict(slot_map=s, k_out=x[:2], v_out=x))


def test_the_reference_format_by_hand():
    # codes 0..15: 0 .5 1 1.5 2 3 4 6 and negatives; scale byte 0x38 is 1.0, 0x40 2.0, 0x01 2^-9
    codes = torch.zeros(1, 64, dtype=torch.uint8)
    codes[0, :8] = torch.tensor([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE])
    codes[0, 8:16] = codes[0, :8]
    codes[0, 16:24] = codes[0, :8]
    scales = torch.tensor([[0x38, 0x40, 0x01, 0, 0, 0, 0, 0x7F]], dtype=torch.uint8)
    v = R.values(codes, scales, torch.tensor([0.25]))[0]
    grid = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert v[:16].tolist() == [x * .25 for x in grid]
    assert v[16:32].tolist() == [x * .5 for x in grid]
    assert v[32:48].tolist() == [x * 2.0 ** -11 for x in grid]
    assert (v[48:112] == 0).all() and torch.isnan(v[112:]).all()
    # and back: the grid is its own quantisation, halves go to the even code
    x = torch.zeros(1, 1, 128, dtype=torch.float64)
    x[0, 0, :16] = torch.tensor(grid, dtype=torch.float64)
    x[0, 0, 16:24] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5], dtype=torch.float64)
    c, b = R.quantise(x, torch.tensor([1.0]))
    assert b[0, 0].tolist() == [0x38, 0x38] + [0] * 6
    got = R.values(c, b, torch.tensor([[1.0]]))[0, 0]
    assert got[:16].tolist() == [abs(g) if g == 0 else g for g in grid]
    assert got[16:24].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]


def test_the_reference_attention_by_hand():
    # two keys of equal score: the mean of the values; a masked one: the other's value
    q = torch.ones(128, dtype=torch.float64)
    k = torch.stack([q, q]) * 0.5
    v = torch.stack([q * 2, q * 4])
    out, lse, _, _ = R.attend_row(q, k, v, torch.tensor([True, True]), 0.25)
    assert torch.allclose(out, q * 3) and abs(lse - (16 + 0.6931471805599453)) < 1e-12
    out, lse, _, _ = R.attend_row(q, k, v, torch.tensor([False, True]), 0.25)
    assert torch.equal(out, q * 4) and lse == 16.0
    out, lse, _, _ = R.attend_row(q, k, v, torch.tensor([False, False]), 0.25)
    assert torch.equal(out, q * 0) and lse == float("-inf")
