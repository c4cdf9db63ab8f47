"""Plain 64-bit reference of the products with NVFP4 weights, on the CPU, with the
error scale that the tests' tolerances are made of.

u = 2^-24.  Sums: a block's 16 products, the blocks and the lanes are below 45
roundings; the tensor cores add K/64 times to a binary32 sum, and each addition
may cut off 2u of the magnitudes, once for each of the parts that x is cut into,
of which the highest carries all but 1/8: T = 48 + 3*K/64 roundings of sum |a*w|.
SiLU: exp 2u, a sum, a division: 4u of a.  The parts of x keep each value to 2^-22
of the largest of its 16, and no finer than 2^-39 of the row's largest.
"""
import torch

from .train_ref import U, d

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0] + [-0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def e4m3(b):
    return b.contiguous().view(torch.float8_e4m3fn).double()


def weight(w4, sf):
    """Values times block scales, [N, K] float64."""
    w4, sf = w4.cpu(), sf.cpu().view(torch.uint8)
    N, K = w4.shape[0], w4.shape[1] * 2
    codes = torch.stack([w4 & 15, w4 >> 4], dim=-1).reshape(N, K).int()
    n, b = torch.arange(N)[:, None], torch.arange(K // 16)[None]
    at = ((n // 128) * (sf.shape[1] // 4) + b // 4) * 512 + n % 32 * 16 + n % 128 // 32 * 4 + b % 4
    return E2M1[codes] * e4m3(sf.reshape(-1)[at]).repeat_interleave(16, 1)


def linear(x, w4, sf, gs, bias, silu):
    """(out, tolerance) of rows x [rows, K]"""
    a, w = d(x), weight(w4, sf)
    K = a.shape[1]
    if silu:
        a = a / (1 + torch.exp(-a))
    b = torch.zeros(w.shape[0], dtype=torch.float64) if bias is None else d(bias)
    g = float(gs)
    out = (a[:, None, :] * w[None]).sum(-1) if not a.isfinite().all() else a @ w.t()
    m = torch.where(a.isfinite(), a, 0.0).abs()
    blk = m.unflatten(1, (K // 16, 16)).amax(-1)
    coarse = torch.maximum(blk * 2.0 ** -22, m.amax(-1, keepdim=True) * 2.0 ** -39).repeat_interleave(16, 1)
    wa = w.abs()
    tol = ((48 + 3 * K / 64) * U * m + 4 * U * m + coarse) @ torch.nan_to_num(wa).t()
    return out / g + b, tol / abs(g) + 4 * U * ((out / g).abs().nan_to_num(0, 0, 0) + b.abs())
