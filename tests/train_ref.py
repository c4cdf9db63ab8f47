"""Plain 64-bit references of the training path, on the CPU, with the error
scales that the tests' tolerances are made of.

u = 2^-24 is the rounding of a binary32 operation and half(T) the one rounding
of an output to its type.  Every sum over a row is a chain of at most 16
additions in a thread, 5 shuffle steps and at most 16 warps: below 40 roundings,
so a row sum is off by at most 40u times the sum of the magnitudes.  The mean is
off by 40u*mean|x|, hence xh = (x - mean)*rstd by about
    dxh = 40u*X + (rstd's relative error, below 24u, + 3u)*|xh|,   X = mean|x|*rstd
and K = 64 covers both factors (40 and 27) with the products' own roundings.
"""
import numpy as np
import torch

U = 2.0 ** -24
K = 64.0
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32)}


def d(t):
    return t.detach().cpu().double()


def ln_stats(x, eps):
    x = d(x)
    mean = x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    return (x - mean) * rstd, rstd, x.abs().mean(-1, keepdim=True) * rstd


def layer_norm(x, w, b, eps):
    """(out, scale of its binary32 error)"""
    xh, _, X = ln_stats(x, eps)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else d(w)
    b = torch.zeros(x.shape[-1], dtype=torch.float64) if b is None else d(b)
    return xh * w + b, K * U * ((xh.abs() + X) * w.abs() + b.abs())


def ln_backward(dout, x, f, eps, dres=None):
    """f [mod_rows, D]: weight, or 1 + scale.  Returns ((dx, tol), (df, tol), (dshift, tol))
    with df and dshift summed over each modulation row's rows."""
    xh, rstd, X = ln_stats(x, eps)
    m, D = f.shape
    rows = x.shape[0]
    f = d(f).repeat_interleave(rows // m, 0)
    dy = d(dout)
    gy = dy * f
    c1, c2 = gy.mean(-1, keepdim=True), (gy * xh).mean(-1, keepdim=True)
    dx = rstd * (gy - c1 - xh * c2)
    a = xh.abs() + X
    tol = K * U * rstd * (gy.abs() + gy.abs().mean(-1, keepdim=True) + a * (gy.abs() * a).mean(-1, keepdim=True))
    if dres is not None:
        dx = dx + d(dres)
        tol = tol + 2 * U * dx.abs()
    seq = rows // m
    part = lambda t: t.reshape(m, seq, D).sum(1)
    # a column sum of seq terms: fewer than seq roundings, on top of the terms' own errors
    df_tol = (K + seq) * U * part(dy.abs() * a)
    ds_tol = (4 + seq) * U * part(dy.abs())
    return (dx, tol), (part(dy * xh), df_tol), (part(dy), ds_tol)


def philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 on arrays of uint32 words held in uint64."""
    c = [np.asarray(v, dtype=np.uint64) for v in (c0, c1, c2, c3)]
    m32 = np.uint64(0xFFFFFFFF)
    for r in range(10):
        pa, pb = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        ka, kb = np.uint64((k0 + r * 0x9E3779B9) % 2 ** 32), np.uint64((k1 + r * 0xBB67AE85) % 2 ** 32)
        c = [(pb >> np.uint64(32)) ^ c[1] ^ ka, pb & m32, (pa >> np.uint64(32)) ^ c[3] ^ kb, pa & m32]
    return c


def keep_mask(rows, cols, p, seed, counter, row0=0):
    quads = -(-cols // 4)
    q, r = np.meshgrid(np.arange(quads), np.arange(row0, row0 + rows))
    counter %= 2 ** 64
    seed %= 2 ** 64
    w = philox(q, r, np.full_like(q, counter % 2 ** 32, dtype=np.uint64),
               np.full_like(q, counter >> 32, dtype=np.uint64), seed % 2 ** 32, seed >> 32)
    words = np.stack(w, axis=-1).reshape(rows, quads * 4)[:, :cols]
    return torch.from_numpy(words >= np.uint64(int(p * 2.0 ** 32)))


def rope(t, pos, axes, freqs, interleaved, inverse):
    """t [B, S, H, hd]; pos [S, A] or [B, S, A].  Returns (out, tol)."""
    x = d(t)
    B, S, H, hd = x.shape
    n = sum(axes) // 2
    which = torch.tensor([a for a, w in enumerate(axes) for _ in range(w // 2)])
    ang = d(pos).reshape(-1, S, len(axes))[:, :, which] * d(freqs)
    c, s = torch.cos(ang)[:, :, None], torch.sin(ang)[:, :, None]
    if inverse:
        s = -s
    i0 = torch.arange(n) * 2 if interleaved else torch.arange(n)
    i1 = i0 + 1 if interleaved else i0 + n
    out = x.clone()
    out[..., i0] = x[..., i0] * c - x[..., i1] * s
    out[..., i1] = x[..., i0] * s + x[..., i1] * c
    tol = torch.zeros_like(x)
    # sine and cosine: the remainder's and the function's roundings, 4u; two products and a sum, 3u
    tol[..., i0] = tol[..., i1] = 8 * U * (x[..., i0].abs() + x[..., i1].abs())
    return out, tol


def assert_close(got, want, tol, what=""):
    """|got - want| <= half(T)*|want| + tol (grown by the rounding of the perturbed value)."""
    g = d(got).reshape(want.shape)
    h = HALF[got.dtype]
    lim = h * want.abs() + tol * (1 + h) + torch.finfo(got.dtype).tiny
    bad = ~((g - want).abs() <= lim) & ~(g.isnan() & want.isnan()) & ~(g == want)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {want.numel()} beyond the bound; first at {i}: got "
                             f"{g[i]!r} want {want[i]!r} bound {lim[i]!r}")
