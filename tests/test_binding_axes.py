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
