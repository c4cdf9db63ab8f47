"""The weights' gradients of the norm of Q and K heads over many tokens: sums of whole
numbers, which are exact in any order, so that one head left out or taken twice shows;
and sums of ordinary values within the roundings that the order of the sums allows.
"""
import pytest
import torch

from . import heads_ref as hr
from . import train_ref as tr
from .test_qk_norm_gpu import BF, DEV, EPS, F32, case, gen, mbx, rnd  # noqa: F401

pytestmark = pytest.mark.gpu

# (batch, tokens, Q heads, K heads): tokens of few heads, several to a warp; of many, shared by warps; more rounds of
# the grid than one, the last not whole; K alone in a block's work
COUNTS = [(1, 1, 1, 1), (1, 2, 3, 1), (3, 7, 5, 2), (2, 37, 4, 2), (2, 1501, 1, 1), (2, 1501, 2, 1), (2, 1501, 4, 3),
          (2, 77, 16, 4), (24, 1, 32, 8), (3, 2731, 3, 1), (1, 20011, 1, 1), (1, 20011, 5, 2), (1, 20011, 32, 1),
          (2, 4352, 24, 24), (1, 9000, 1, 33)]
# (elements, those that turn, in halves)
HEADS = [(64, 64, False), (64, 32, True), (128, 128, False), (128, 64, True), (80, 40, False), (72, 72, False), (96, 96, True),
         (100, 50, True), (127, 60, False), (32, 32, False), (256, 128, False), (255, 2, True), (2, 2, False)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("hd,turn,halves", HEADS)
def test_whole_numbers(mbx, hd, turn, halves, dt):  # noqa: F811
    """x = 2^-4 or -2^-4 and eps = 1 - 2^-8: the mean of the squares is 2^-8 to 2^-32, with eps it rounds to 1 and
    the norm leaves x as it is (the forward call says so).  At position 0 nothing turns.  So a term is a whole number
    of sixteenths, at most 1/2, and sums of up to 2^21 of them are exact in binary32."""
    g = torch.Generator(device=DEV).manual_seed(hd)
    eps, fr = 1.0 - 2.0 ** -8, mbx.rope_axis_freqs((turn,))
    w = torch.rand(hd, generator=g, device=DEV) + 0.5
    for B, S, hq, hk in COUNTS:
        x = [(torch.randint(0, 2, (B, S, H, hd), generator=g, device=DEV) * 2 - 1).div(16).to(dt) for H in (hq, hk)]
        do = [torch.randint(-8, 9, t.shape, generator=g, device=DEV).to(dt) for t in x]
        pos = torch.zeros((S, 1), dtype=torch.int32, device=DEV)
        out = mbx.qk_norm_rope(*x, None, None, pos, fr, (turn,), not halves, eps)
        assert torch.equal(out[0], x[0]) and torch.equal(out[1], x[1])
        dw = mbx.qk_norm_rope_backward(*do, *x, w, w, pos, fr, (turn,), not halves, eps)[2:]
        for got, d, t in zip(dw, do, x):
            assert torch.equal(got.double(), (d.double() * t.double()).sum((0, 1, 2))), (B, S, hq, hk)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("B,S,hq,hk", [(3, 2731, 3, 1), (1, 20011, 5, 2), (1, 20011, 32, 1)])
def test_many_terms(mbx, B, S, hq, hk, dt):  # noqa: F811
    """A term passes fewer additions than there are terms: those of its lane (20011 tokens of 32 heads: 9 tokens of a
    warp, 8 heads each), of a warp's groups (32), of a block's warps (8) and of the join (two parts on each of at most
    160 SMs): 450 with the 24 of its own value.  That is well below the sums themselves."""
    g = gen(S + hq)
    axes, fr = (16, 24, 24), mbx.rope_axis_freqs((16, 24, 24))
    q, k = case(g, B, S, hq, hk, 64, dt)
    do = [rnd(g, t.shape, dt, 0.1) for t in (q, k)]
    w = rnd(g, (64,), F32, 0.1, 1.0)
    pos = torch.randint(0, 200, (S, 3), generator=g).int()
    dw = mbx.qk_norm_rope_backward(*do, q, k, w, w, pos.to(DEV), fr, axes, True, EPS)[2:]
    for got, d, t in zip(dw, do, (q, k)):
        _, (want, tol) = hr.norm_rope_backward(d, t, w, pos, axes, fr, True, EPS)
        tol = tol / (24 + t.shape[0] * t.shape[1] * t.shape[2]) * 450
        assert tol.max() < 0.05 * want.abs().max()
        tr.assert_close(got, want, tol)
