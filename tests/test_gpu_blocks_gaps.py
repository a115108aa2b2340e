"""Appends to 8-bit blocks whose slots have holes: padding, slots outside the cache and positions outside the table
between the tokens of one block, few and many of them. The tokens that are left are written as if the holes were not
there: codes and scales bit for bit those of the model on the host."""

import pytest
import torch

import decode_attention_flash_gb300 as da
from test_gpu_blocks_append import Cache, rows

pytestmark = pytest.mark.gpu
both = pytest.mark.parametrize("kind", ["e4m3", "int8"])


def append(c, k, v, slots, flags=0, **more):
    c.eng.append({**c.t, "k_new": k.cuda(), "v_new": v.cuda(), "slot_map": slots.cuda(), **more})
    assert c.eng.errors() == flags
    c.model("k", k, slots)
    c.model("v", v, slots)
    c.same()


def with_holes(slots, holes, gen, bad):
    """`slots` with holes[i] entries of no slot after entry i (bad: some outside the cache instead of padding)."""
    parts = []
    for s, n in zip(slots.tolist(), holes):
        parts.append(torch.tensor([s]))
        h = torch.full((n,), -1)
        if bad:
            h[torch.rand(n, generator=gen) < 0.5] = 1 << 40
        parts.append(h)
    return torch.cat(parts)


@both
@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("block", [16, 64, 256])
@pytest.mark.parametrize("gap", [1, 2, 29, 31, 64, 300, 1000])
def test_one_hole_in_a_block(kind, block, gap, bad):
    c = Cache(kind, 3, 3, block=block, page=256, pages=4, seed=gap)
    gen = torch.Generator().manual_seed(block + gap)
    for first, n, at in ((0, 9, 4), (9, 2, 0), (12, block, 1), (12 + block, block + 5, block - 14), (300, 200, 199)):
        slots = torch.arange(first, first + n)
        holes = [gap if i == at else 0 for i in range(n)]
        s = with_holes(slots, holes, gen, bad)
        flags = da.DA_DEVERR_SLOT if bool((s > 1 << 30).any()) else 0
        append(c, rows(s.numel(), 3, gen) * 2.0 ** (first % 5), rows(s.numel(), 3, gen), s, flags)


@both
@pytest.mark.parametrize("block,n", [(16, 40), (32, 250), (64, 700), (256, 700)])
def test_holes_of_many_lengths(kind, block, n):
    """Holes after a third of the tokens, more of them than the block has positions among them; rows of two
    sequences in turn, the second one's written in no order."""
    c = Cache(kind, 2, 2, block=block, page=256, pages=8, seed=n)
    gen = torch.Generator().manual_seed(n)
    for step in range(3):
        a = torch.arange(3 + step, 3 + step + n // 2)
        b = 4 * 256 + torch.arange(n // 2)
        b = b.reshape(-1)[:n // 2 // 8 * 8].reshape(-1, 8).flip(1).reshape(-1)
        slots = torch.cat([a, b])
        odd = torch.rand(slots.numel(), generator=gen) < 0.33
        many = torch.randint(1, 5, odd.shape, generator=gen) * torch.where(torch.rand(odd.shape, generator=gen) < 0.05, 40, 1)
        s = with_holes(slots, torch.where(odd, many, 0).tolist(), gen, step == 1)
        if step == 2:
            s = torch.cat([torch.full((77,), -1), s, torch.full((500,), -1)])
        append(c, rows(s.numel(), 2, gen), rows(s.numel(), 2, gen) * 4.0, s, da.DA_DEVERR_SLOT if step == 1 else 0)


@both
def test_ragged_drafts_in_the_layout_of_query_tokens(kind):
    """[rows, q_len] tokens, each row's last ones padding, rows of length 0 among them."""
    b, q = 40, 5
    c = Cache(kind, 4, 2, block=16, page=16, pages=200, batch=b, q_len=q, seed=1)
    gen = torch.Generator().manual_seed(2)
    at = torch.zeros(b, dtype=torch.long)
    perm = torch.randperm(200, generator=gen).reshape(b, 5)
    for _ in range(12):
        n = torch.randint(0, q + 1, (b,), generator=gen)
        pos = at[:, None] + torch.arange(q)
        s = torch.where(torch.arange(q) < n[:, None], perm.gather(1, pos // 16) * 16 + pos % 16, -1).reshape(-1)
        append(c, rows(b * q, 2, gen), rows(b * q, 2, gen), s)
        at += n


@both
@pytest.mark.parametrize("n", [60, 600])
def test_bad_positions_between_holes(kind, n):
    c = Cache(kind, 1, 1, block=64, page=64, pages=16, seed=3)
    gen = torch.Generator().manual_seed(n)
    s = torch.arange(5, 5 + n)
    s[torch.rand(n, generator=gen) < 0.3] = -1
    pos = torch.where(torch.rand(n, generator=gen) < 0.2, 99, 7).int()
    t = dict(cos_sin=torch.cat([torch.ones(50, 64), torch.zeros(50, 64)], -1).cuda(), positions=pos.cuda())
    k, v = rows(n, 1, gen), rows(n, 1, gen)
    c.eng.append({**c.t, "k_new": k.cuda(), "v_new": v.cuda(), "slot_map": s.cuda(), **t})
    assert c.eng.errors() == da.DA_DEVERR_POSITION
    s[pos == 99] = -1
    c.model("k", k, s)
    c.model("v", v, s)
    c.same()


@both
def test_a_block_filled_and_its_neighbours(kind):
    """A whole block in one call with a hole after each token, between two blocks that get one token each."""
    c = Cache(kind, 8, 8, block=32, page=32, pages=8, seed=4)
    gen = torch.Generator().manual_seed(5)
    slots = torch.cat([torch.tensor([31]), torch.arange(32, 64), torch.tensor([64])])
    s = with_holes(slots, [i % 3 for i in range(slots.numel())], gen, False)
    append(c, rows(s.numel(), 8, gen), rows(s.numel(), 8, gen), s)


@both
def test_a_captured_append_with_holes(kind):
    """The same graph over slots that change: full, half of them padding, padding alone."""
    n = 96
    c = Cache(kind, 2, 2, block=32, page=32, pages=6, seed=6)
    gen = torch.Generator().manual_seed(7)
    k, v, s = rows(n, 2, gen).cuda(), rows(n, 2, gen).cuda(), torch.full((n,), -1).cuda()
    call = {**c.t, "k_new": k, "v_new": v, "slot_map": s}
    c.eng.append(call)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.eng.append(call)
    for keep in (1.0, 0.5, 0.0, 0.9):
        slots = torch.where(torch.rand(n, generator=gen) < keep, torch.arange(40, 40 + n), -1)
        hk, hv = rows(n, 2, gen), rows(n, 2, gen)
        k.copy_(hk), v.copy_(hv), s.copy_(slots)
        g.replay()
        torch.cuda.synchronize()
        c.model("k", hk, slots)
        c.model("v", hv, slots)
        c.same()
    assert c.eng.errors() == 0
