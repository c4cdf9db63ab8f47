"""The cosines and sines of the norm and rotation of Q and K heads, read out of heads of
ones and zeros, against the exact product of position and frequency in whole numbers.
"""
import math
from fractions import Fraction

import pytest
import torch

from .test_qk_norm_gpu import BF, DEV, F32, mbx  # noqa: F401

pytestmark = pytest.mark.gpu

# the largest error over all remainders that there are, multiples of 2^-32 of a turn up to an eighth: 1.7262 * 2^-24
LIMIT = 1.73 * 2.0 ** -24 + 2.0 ** -50


def _inverse_of_2pi(bits):
    """floor(2^bits / (2 pi)), pi by Machin's formula."""
    def arctan(n):  # of 1/n, in units of 2^-(bits+64)
        t = s = (1 << (bits + 64)) // n
        k = 1
        while t:
            t = -t // (n * n)
            k += 2
            s += t // k
            if t == -1:
                break
        return s
    pi = 4 * (4 * arctan(5) - arctan(239))
    return (1 << (2 * bits + 64)) // (2 * pi)


BITS = 700
INVERSE = Fraction(_inverse_of_2pi(BITS), 1 << BITS)
FREQS = [1.0, -1.0, 0.0, 7.5, 50.0, 1e-9, 1e-300, -3.3e5, 2.0 ** 40, 1e-320, 2.0 ** 52 + 1, -(2.0 ** 53), math.nextafter(2.0 ** 54, 0),
         math.pi, math.pi / 2, 1e10 / 3, -0.1, 2.0 ** -64, 2.0 ** -11, 2.0 ** -12, -2.0 ** -13, 123456789.125]
WHOLE = [0, 1, -1, 12345, 2 ** 31 - 1, -2 ** 31, 99, -7, 1 << 30, 1000003, 65535, 32759, -4351, 3, 7, 1 << 16]
PART = [0.0, -0.0, 0.7109375, -1234.56, 1e-12, 1e-40, 3e7, -5.5, 1e9, 16777216.0, 2.0 ** 60, -3.7e20, 1.5 * 2.0 ** 89, 1e-30, 0.1, 8388607.5]


def _exact(positions, freqs):
    c, s = [], []
    for p in positions:
        for f in freqs:
            turns = Fraction(p) * Fraction(f) * INVERSE
            a = float((turns - round(turns)) * 1) * 2.0 * math.pi
            c.append(math.cos(a))
            s.append(math.sin(a))
    return (torch.tensor(v, dtype=torch.float64).view(len(positions), len(freqs)) for v in (c, s))


def test_the_inverse():
    assert abs(float(INVERSE) - 1 / (2 * math.pi)) < 1e-16
    # pi rounded to 53 bits is 1.2246467991473532e-16 short
    assert abs(float((Fraction(1) / INVERSE / 2 - Fraction(math.pi))) - 1.2246467991473532e-16) < 1e-30


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("kind", ["whole", "part"])
def test_cosines_and_sines(mbx, kind, interleaved):  # noqa: F811
    """A head whose pairs are (1, 0): the mean of the squares is 1/2 and eps 1/2, so the norm leaves it as it is and the
    rotation writes its cosines and sines.  The gradients' pass turns the other way: of incoming (1, 0) it has
    g = (cos, -sin), dw = g * x at a single token."""
    g = torch.Generator().manual_seed(2)
    mag = torch.rand(32 - len(FREQS), generator=g, dtype=torch.float64) * 113 - 60
    freqs = FREQS + [float(v) for v in torch.exp2(mag)]
    values = WHOLE if kind == "whole" else PART
    pos = torch.tensor(values, dtype=torch.int32 if kind == "whole" else F32)
    n = len(freqs)
    c, s = _exact(values if kind == "whole" else [float(v) for v in pos], freqs)
    even, odd = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    for heads in (1, 3, 40):
        x = torch.zeros((1, len(values), heads, 2 * n), device=DEV)
        x[..., even] = 1.0
        fr = torch.tensor(freqs, dtype=torch.float64, device=DEV)
        out, _ = mbx.qk_norm_rope(x, None, None, None, pos[:, None].to(DEV), fr, (2 * n,), interleaved, 0.5)
        out = out.double().cpu()
        for h in range(heads):
            assert (out[0, :, h, even] - c).abs().max() <= LIMIT and (out[0, :, h, odd] - s).abs().max() <= LIMIT
    ones, w = torch.ones((1, 1, 1, 2 * n), device=DEV), torch.ones(2 * n, device=DEV)
    do = torch.zeros_like(ones)
    do[..., even] = 1.0
    for i in range(len(values)):
        # x of ones: the mean of the squares is 1, eps 3: rstd = 1/2
        dw = mbx.qk_norm_rope_backward(do, None, ones, None, w, None, pos[i:i + 1, None].to(DEV), fr, (2 * n,), interleaved, 3.0)[2]
        dw = 2 * dw.double().cpu()
        assert (dw[even] - c[i]).abs().max() <= LIMIT and (dw[odd] + s[i]).abs().max() <= LIMIT


def test_frequencies_past_the_range(mbx):  # noqa: F811
    """2^54 radians per position and more, infinities and NaN: NaN in their own pair."""
    fr = torch.tensor([0.5, 2.0 ** 54, -1e300, float("inf"), float("nan"), -0.25], dtype=torch.float64, device=DEV)
    x = torch.ones((1, 3, 2, 12), dtype=BF, device=DEV)
    pos = torch.tensor([[1], [0], [-5]], dtype=torch.int32, device=DEV)
    out, _ = mbx.qk_norm_rope(x, None, None, None, pos, fr, (12,))
    assert out[..., 2:10].isnan().all() and out[..., :2].isfinite().all() and out[..., 10:].isfinite().all()
