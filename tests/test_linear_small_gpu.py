"""Products with NVFP4 weights of activations next to zero: an output has the stated
precision however small x is, down to binary32's own smallest step.
"""
import pytest
import torch

from . import linear_ref as lr
from . import train_ref as tr
from .test_linear_nvfp4_gpu import BF, DEV, F32, gen, mbx, weight  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K", [1024, 1040])
@pytest.mark.parametrize("rows", [3, 16])
def test_activations_next_to_zero(mbx, rows, K, dt):  # noqa: F811
    """Rows of 2^-90 to 2^-145 (subnormal below 2^-126) under a global scale that makes the outputs ordinary numbers.
    Beside the relative bounds: a slice's sum is rounded once to a multiple of 2^-149, at most K / 256 slices, whose
    sum is then exact there."""
    g = gen(rows + K)
    w4, sf, gs = weight(mbx, g, 300, K)
    for k in (90, 100, 105, 110, 115, 120, 125, 128, 132, 140, 145):
        x = (torch.randn((rows, K), generator=g).double() * 2.0 ** -k).to(dt)
        x[0, 32:48] = 0.0
        x[1, ::3] *= 2.0 ** -6
        small = (gs.double() * 2.0 ** -min(k, 118)).float()  # normal itself
        out = torch.empty((rows, 300), dtype=F32, device=DEV)
        mbx.linear_nvfp4(x.to(DEV), w4, sf, small.to(DEV), out=out)
        want, tol = lr.linear(x, w4, sf, small, None, False)
        tr.assert_close(out, want, tol + -(-K // 256) * 2.0 ** -150 / float(small), what=f"2^-{k}")


def test_a_small_row_keeps_its_bits(mbx):  # noqa: F811
    """2^-k times a row gives 2^-k times its outputs, bit for bit, as long as nothing is subnormal."""
    g = gen(1)
    w4, sf, gs = weight(mbx, g, 300, 1024)
    x = torch.randn((3, 1024), generator=g)
    x = torch.where(x.abs() < 2.0 ** -10, torch.zeros_like(x), x).to(DEV)
    want = mbx.linear_nvfp4(x, w4, sf, gs)
    want = torch.where(want.abs() < 2.0 ** -20, torch.zeros_like(want), want)
    for k in (60, 85, 95, 103, 110):
        got = mbx.linear_nvfp4(x * 2.0 ** -k, w4, sf, gs * 2.0 ** -k)
        assert torch.equal(torch.where(got.abs() < 2.0 ** -20, torch.zeros_like(got), got), want), k
