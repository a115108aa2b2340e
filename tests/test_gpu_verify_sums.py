"""Running sums of a vocabulary where one weight is great and the others are all alike and just too small to
change a float of its size: each is a rounding error of the sum so far, and they all err to the same side. Borders are
chosen nearer to a token's end than such errors would add up to, yet 2^-40 of the sum away from it, which is what the
call promises; tokens come from whole numbers on the host."""

from fractions import Fraction

import pytest
import torch

from test_gpu_verify import engine, run

pytestmark = pytest.mark.gpu
W = float.fromhex("0x1.f8298p-33")


def borders(vocab, great, want):
    """Random numbers r in [0, 1) whose border r * sum lies between 2^-40 and 2^-37 of the sum from a token's end, and
    the first token past it. The great weight is 1, at `great`."""
    w = Fraction(W)
    total = 1 + (vocab - 1) * w
    near, far = total / 2 ** 40, total / 2 ** 37
    out = []
    lo = int((1 - 1 / total) * 2 ** 24)
    # the border past the great weight, or (where that comes last) anywhere below it
    for m in range(1, lo) if great == 0 else range(2 ** 24 - 1, 2 ** 24 - lo, -1):
        r = 1 - Fraction(m, 2 ** 24)
        border = r * total
        ahead = border - 1 if great == 0 else border  # made of small weights
        if ahead < 0 or ahead > (vocab - 1) * w:
            continue
        k = ahead // w  # small weights that end at or below it
        gap = min(ahead - k * w, (k + 1) * w - ahead)
        if near < gap < far and k < vocab - 1:
            out.append((float(r), int(k) + (1 if great == 0 else 0)))
    step = max(1, len(out) // want)
    return out[::step][:want]


@pytest.mark.parametrize("batch,vocab", [(310, 1 << 21), (160, 1 << 21), (5, 1 << 21), (1250, 1200000), (300, 1200001)])
@pytest.mark.parametrize("great", [0, -1])
def test_a_great_weight_and_many_that_round_to_nothing(batch, vocab, great):
    some = borders(vocab, great, 150)
    assert len(some) > 50
    p = torch.full((batch, 1, vocab), W, device="cuda")
    p[..., great] = 1.0
    eng = engine(batch, pages=16, cols=1)
    u = torch.zeros(batch, 1, device="cuda")
    wrong = 0
    for at in range(0, len(some), batch):
        part = (some[at:at + batch] * batch)[:batch]
        u[:, 0] = torch.tensor([r for r, _ in part])
        got = run(eng, dict(target_probs=p, draft_tokens=torch.zeros(batch, 0, dtype=torch.int32), uniforms=u))
        wrong += int((got["tokens_out"][:, 0].cpu() != torch.tensor([k for _, k in part])).sum())
    assert eng.errors() == 0 and wrong == 0
