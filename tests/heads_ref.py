"""Plain 64-bit references of the norm and rotation of Q and K heads, on the CPU,
with the error scales that the tests' tolerances are made of.

u = 2^-24.  A head's sum of squares is a chain of at most 16 multiply-adds in a
lane and 5 shuffle steps, 21 roundings of terms of one sign; with the mean, eps,
the square root and the division rstd is off by (21 + 2 + 1)/2 + 2 = 14u.  A
turned value is off by 8u of its pair's magnitudes (train_ref.rope).
  forward   n = x*rstd*w: 14u + 2u, and the turn: 24u of |n0| + |n1|; KF = 32
  backward  g: 8u of G = |d0| + |d1|.  gy*rstd: 8 + 14 + 3.  mean(gy*xh): chain 21,
            products 2, g 8, 1/hd 2, rstd 14; times xh 15, rstd 15: 77.  KB = 96
  dw        g*xh: 8 + 15 + 1, and fewer roundings than terms in the sum
"""
import torch

from .train_ref import U, d

KF, KB = 32.0, 96.0


def _angles(pos, S, axes, freqs):
    which = torch.tensor([a for a, w in enumerate(axes) for _ in range(w // 2)])
    ang = d(pos).reshape(-1, S, len(axes))[:, :, which] * d(freqs)
    return torch.cos(ang)[:, :, None], torch.sin(ang)[:, :, None]


def _turn(x, c, s, n, interleaved):
    """(x turned, the magnitudes of each element's pair; of a passing element its own)"""
    i0 = torch.arange(n) * 2 if interleaved else torch.arange(n)
    i1 = i0 + 1 if interleaved else i0 + n
    out, mag = x.clone(), x.abs()
    out[..., i0] = x[..., i0] * c - x[..., i1] * s
    out[..., i1] = x[..., i0] * s + x[..., i1] * c
    mag[..., i0] = mag[..., i1] = x[..., i0].abs() + x[..., i1].abs()
    return out, mag


def _weight(w, hd):
    return torch.ones(hd, dtype=torch.float64) if w is None else d(w)


def norm_rope(x, w, pos, axes, freqs, interleaved, eps):
    """(out, tolerance)"""
    xd = d(x)
    c, s = _angles(pos, x.shape[1], axes, freqs)
    n = xd / torch.sqrt(xd.square().mean(-1, keepdim=True) + eps) * _weight(w, x.shape[-1])
    out, mag = _turn(n, c, s, sum(axes) // 2, interleaved)
    return out, KF * U * mag


def norm_rope_backward(dout, x, w, pos, axes, freqs, interleaved, eps):
    """((dx, tolerance), (dw, tolerance))"""
    xd, wd = d(x), _weight(w, x.shape[-1])
    c, s = _angles(pos, x.shape[1], axes, freqs)
    g, G = _turn(d(dout), c, -s, sum(axes) // 2, interleaved)
    rstd = 1.0 / torch.sqrt(xd.square().mean(-1, keepdim=True) + eps)
    xh, gy = xd * rstd, g * wd
    dx = rstd * (gy - xh * (gy * xh).mean(-1, keepdim=True))
    Gw = G * wd.abs()
    tol = KB * U * rstd * (Gw + xh.abs() * (Gw * xh.abs()).mean(-1, keepdim=True))
    terms = x.shape[0] * x.shape[1] * x.shape[2]
    dw = (g * xh).sum((0, 1, 2))
    return (dx, tol), (dw, (24 + terms) * U * (G * xh.abs()).sum((0, 1, 2)))
