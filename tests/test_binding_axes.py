"""How the binding hands over rotary axes and positions (what it refuses needs no GPU)."""

import pytest
import torch

import decode_attention_flash_gb300 as da


def args(monkeypatch, pair_axis=None, positions=None, n=3, rope=16):
    """make_append_args on host tensors, whose addresses are taken as device pointers."""
    monkeypatch.setattr(da, "_ptr", lambda t: None if t is None else t.data_ptr())
    t = dict(slot_map=torch.zeros(n, dtype=torch.int64), cos_sin=torch.zeros(4, rope),
             positions=torch.zeros(n, dtype=torch.int32) if positions is None else positions)
    return da.make_append_args(t, pair_axis=pair_axis)


@pytest.mark.parametrize("bad", [256, -1, 255 + 256, 1 << 40])
def test_an_axis_outside_a_byte_is_refused(monkeypatch, bad):
    with pytest.raises(ValueError, match="pair_axis"):
        args(monkeypatch, pair_axis=[0, 1, 0, 1, 0, 1, 0, bad])
    with pytest.raises(ValueError, match="pair_axis"):
        args(monkeypatch, pair_axis=torch.tensor([bad] + [0] * 7))


@pytest.mark.parametrize("axes", [[0, 1, 2, 0, 1, 2, 0, 1], [255] * 8, torch.tensor([2, 0, 1, 1, 0, 0, 0, 2])])
def test_axes_are_handed_over_as_they_are(monkeypatch, axes):
    a = args(monkeypatch, pair_axis=axes)
    assert [a._pairs[i] for i in range(8)] == [int(x) for x in axes]


def test_nothing_to_turn_takes_no_axes(monkeypatch):
    assert args(monkeypatch, pair_axis=[], rope=0).rope_dim == 0


def test_positions_may_be_a_column_range(monkeypatch):
    wide = torch.arange(30, dtype=torch.int32).view(3, 10)
    part = wide[:, 4:7]
    a = args(monkeypatch, positions=part)
    assert (a.positions, a.position_stride, a.rope_axes) == (part.data_ptr(), 10, 3)
    a = args(monkeypatch, positions=wide[:, 4:5], n=1)
    assert (a.positions, a.position_stride, a.rope_axes) == (wide[:, 4:5].data_ptr(), 10, 3)
    a = args(monkeypatch, positions=wide.contiguous()[:, :], n=10)
    assert (a.position_stride, a.rope_axes) == (10, 3)
    a = args(monkeypatch, positions=wide[1:2, 4:7])
    assert (a.positions, a.position_stride, a.rope_axes) == (wide[1:2, 4:7].data_ptr(), 3, 1)
    a = args(monkeypatch, positions=wide[1, 4:7])
    assert (a.positions, a.position_stride, a.rope_axes) == (wide[1, 4:7].data_ptr(), 3, 1)


@pytest.mark.parametrize("positions", [torch.zeros(3, 3, dtype=torch.int32).t()[:, :3], torch.zeros(6, dtype=torch.int32)[::2],
                                       torch.zeros(1, dtype=torch.int32).expand(3), torch.zeros(3), torch.zeros(3, dtype=torch.int64),
                                       torch.zeros(4, dtype=torch.int32), torch.zeros(2, 2, 3, dtype=torch.int32)])
def test_other_positions_are_refused(monkeypatch, positions):
    with pytest.raises(ValueError, match="positions"):
        args(monkeypatch, positions=positions)


@pytest.mark.gpu
def test_a_column_range_turns_as_its_copy_does():
    eng = da.DecodeAttention(device=0, batch=1, num_q_heads=2, num_kv_heads=1, head_dim_qk=128, head_dim_v=128,
                             kv_layout=da.DA_KV_PAGED, page_size=16, num_pages=4, max_pages_per_seq=4, max_seq_len=64,
                             q_dtype=da.DA_DTYPE_BF16, kv_dtype=da.DA_DTYPE_BF16)
    gen = torch.Generator().manual_seed(1)
    wide = torch.randint(0, 50, (3, 100), generator=gen).int().cuda()
    a = torch.randn(50, 64, generator=gen)
    table = torch.cat([a.cos(), a.sin()], -1).cuda()
    for at, n in ((0, 40), (17, 40), (99, 1), (60, 40)):
        q = torch.randn(n, 2, 128, generator=gen).to(torch.bfloat16).cuda()
        out = torch.zeros(2, n, 2, 128, dtype=torch.bfloat16, device="cuda")
        for k, pos in enumerate((wide[:, at:at + n], wide[:, at:at + n].contiguous())):
            eng.append(dict(q=q, q_out=out[k], cos_sin=table, positions=pos), pair_axis=[i % 3 for i in range(64)])
        assert eng.errors() == 0 and torch.equal(out[0], out[1]) and not torch.equal(out[0], q)
    # the same axis over and over is no memory of tokens side by side: the library refuses it
    with pytest.raises(da.DecodeAttnError) as e:
        eng.append(dict(q=q, q_out=out[0], cos_sin=table, positions=wide[:1, :40].expand(3, 40)), pair_axis=[0] * 64)
    assert e.value.status == da.DA_ERR_INVALID_ARG
