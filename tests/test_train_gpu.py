"""The training path on the GPU against plain 64-bit references (train_ref.py):
widths that are no multiple of a chunk, padded and misaligned rows, one row and
many, parameters shared by the batch, a sample or a token, both activation
types, values that are infinite, constant or far from zero.
"""
import numpy as np
import pytest
import torch

from . import train_ref as tr

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
TYPES = [(BF, BF), (BF, F32), (F32, F32)]
# one thread each of a warp, a warp's share and one over, several warps a row, the largest
WIDTHS = [1, 7, 8, 64, 257, 264, 520, 1030, 2048, 5120, 8191, 8192]


@pytest.fixture(scope="module")
def mbx():
    import modulation_bit_exact_gb300 as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, shape, dt, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dt).to(DEV)


def padded(t, pad=24, fill=float("nan")):
    """The same rows inside a wider buffer whose padding holds `fill`."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf, buf[:, :t.shape[1]]


def misaligned(t):
    """The same rows starting one element past a 16-byte boundary."""
    buf = torch.zeros(t.numel() + 16, dtype=t.dtype, device=t.device)
    v = buf[1:1 + t.numel()].view(t.shape)
    v.copy_(t)
    return v


def acts(g, rows, D, dt):
    """N(0, 1) with rows of a far mean, a constant row and a zero row among them."""
    x = torch.randn(rows, D, generator=g)
    if rows > 3:
        x[1] += 300.0
        x[2] = 0.7
        x[3] = 0.0
    return x.to(dt).to(DEV)


# ---------------------------------------------------------------- LayerNorm


@pytest.mark.parametrize("dt,pdt", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_layer_norm(mbx, D, dt, pdt):
    g = gen(D)
    for rows in (1, 5, 333):
        x, w, b = acts(g, rows, D, dt), rnd(g, (D,), pdt, 0.05, 1.0), rnd(g, (D,), pdt, 0.1)
        for ww, bb in ((w, b), (None, b), (w, None), (None, None)):
            tr.assert_close(mbx.layer_norm(x, ww, bb, EPS), *tr.layer_norm(x, ww, bb, EPS), what=f"rows {rows}")


@pytest.mark.parametrize("dt", [BF, F32])
def test_layer_norm_views(mbx, dt):
    g = gen(3)
    x, w, b = acts(g, 37, 768, dt), rnd(g, (768,), dt, 0.05, 1.0), rnd(g, (768,), dt, 0.1)
    want = tr.layer_norm(x, w, b, EPS)
    obuf, out = padded(torch.zeros_like(x), fill=7.0)
    mbx.layer_norm(padded(x)[1], w, b, EPS, out=out)
    tr.assert_close(out, *want)
    assert torch.all(obuf[:, 768:] == 7.0)
    tr.assert_close(mbx.layer_norm(misaligned(x), w, b, EPS), *want)
    tr.assert_close(mbx.layer_norm(x, misaligned(w[None])[0], b, EPS), *want)
    assert torch.equal(mbx.layer_norm(x.view(37, 1, 768), w, b, EPS).view(37, 768), mbx.layer_norm(x, w, b, EPS))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [40, 200, 520, 1021, 4096])
def test_layer_norm_many_rows(mbx, D, dt):
    """Enough rows for every SM to take two at a time, and one over."""
    g = gen(17)
    x, w, b = acts(g, 2433, D, dt), rnd(g, (D,), dt, 0.05, 1.0), rnd(g, (D,), dt, 0.1)
    tr.assert_close(mbx.layer_norm(x, w, b, EPS), *tr.layer_norm(x, w, b, EPS))


def test_layer_norm_one_row_tensor(mbx):
    x = rnd(gen(18), (768,), BF)
    tr.assert_close(mbx.layer_norm(x), *tr.layer_norm(x[None], None, None, EPS))


def test_layer_norm_non_finite_rows_stay_alone(mbx):
    x = acts(gen(4), 9, 512, BF)
    x[5, 100], x[7, 3] = float("inf"), float("nan")
    out = mbx.layer_norm(x)
    assert out[5].isnan().all() and out[7].isnan().all()
    keep = [0, 1, 2, 3, 4, 6, 8]
    tr.assert_close(out[keep], *tr.layer_norm(x[keep], None, None, EPS))


def check_ln_backward(mbx, x, do, f, dres, scale=None, weight=None, **out):
    if scale is not None:
        got = mbx.ln_modulate_backward(do, x, scale, EPS, dres, **out)
    else:
        got = mbx.layer_norm_backward(do, x, weight, EPS, dres, **out)
    rows = lambda t: t.reshape(-1, t.shape[-1])
    want = tr.ln_backward(rows(do), rows(x), f, EPS, None if dres is None else rows(dres))
    for name, gt, (w, tol) in zip(("dx", "dfactor", "dshift"), got, want):
        tr.assert_close(gt, w, tol, what=name)
    return got


@pytest.mark.parametrize("dt,pdt", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_layer_norm_backward(mbx, D, dt, pdt):
    g = gen(100 + D)
    for rows in (1, 2, 5, 333):
        x, do = acts(g, rows, D, dt), rnd(g, (rows, D), dt, 0.1)
        w = rnd(g, (D,), pdt, 0.05, 1.0)
        dres = rnd(g, (rows, D), dt, 0.1) if rows != 5 else None
        check_ln_backward(mbx, x, do, tr.d(w)[None], dres, weight=w)
        dx, dw, db = mbx.layer_norm_backward(do, x, None, EPS, dres)
        (want, tol), _, _ = tr.ln_backward(do, x, torch.ones(1, D), EPS, dres)
        assert dw is None and db is None
        tr.assert_close(dx, want, tol)


@pytest.mark.parametrize("dt,pdt", TYPES)
@pytest.mark.parametrize("D", [1, 40, 257, 520, 1030, 4096, 8192])
@pytest.mark.parametrize("mod_rows,seq", [(1, 700), (2, 350), (5, 7), (40, 3), (123, 1), (300, 40)])
def test_ln_modulate_backward(mbx, D, dt, pdt, mod_rows, seq):
    if mod_rows * seq * D > 8_000_000:
        seq = max(2, 8_000_000 // (mod_rows * D))
    g = gen(D * 7 + mod_rows)
    rows = mod_rows * seq
    x, do = acts(g, rows, D, dt), rnd(g, (rows, D), dt, 0.1)
    sc = rnd(g, (mod_rows, D), pdt, 0.1)
    dres = rnd(g, (rows, D), dt, 0.1) if seq % 2 else None
    check_ln_backward(mbx, x, do, 1 + tr.d(sc), dres, scale=sc)


def inside(t, shift, stride, fill):
    """The same rows `shift` elements behind a 16-byte boundary, `stride` apart, in a buffer of `fill`."""
    rows, D = t.shape
    buf = torch.full((rows * stride + 32,), fill, dtype=t.dtype, device=t.device)
    v = buf[8 + shift:8 + shift + rows * stride].view(rows, stride)[:, :D]
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D,pad", [(1, 0), (2, 3), (9, 2), (121, 0), (561, 6), (1027, 1), (4099, 0), (8185, 1)])
def test_rows_at_every_start(mbx, D, pad, dt):
    """All operands of a row start at the same byte, at each of a 16-byte piece's and from row to
    row another; NaN lies around every input, and nothing around an output is written."""
    g = gen(D + pad)
    rows, stride = (3001 if D < 2000 else 700), D + pad
    x, do, dres, f = (rnd(g, (rows, D), dt, s, m) for s, m in ((1.0, 0.5), (0.1, 0.0), (0.1, 0.0), (0.1, 0.0)))
    w, b = rnd(g, (D,), dt, 0.05, 1.0), rnd(g, (D,), dt, 0.1)
    want = tr.layer_norm(x, w, b, EPS)
    grads, alone = tr.ln_backward(do, x, 1 + tr.d(f), EPS, dres), tr.ln_backward(do, x, 1 + tr.d(f), EPS)[0]
    nan = float("nan")

    def clean(buf, v):
        v.fill_(7.0)
        return bool((buf == 7.0).all())

    for shift in (range(8) if D < 2000 else (0, 1, 5, 6)):
        xi, doi, ri, fi = (inside(t, shift, stride, nan)[1] for t in (x, do, dres, f))
        ob, o = inside(x, shift, stride, 7.0)
        mbx.layer_norm(xi, w, b, EPS, out=o)
        tr.assert_close(o, *want, what=f"shift {shift}")
        assert clean(ob, o)
        outs = [inside(x, shift, stride, 7.0) for _ in range(3)]
        mbx.ln_modulate_backward(doi, xi, fi, EPS, ri, *[v for _, v in outs])
        for (buf, v), (wv, tol), name in zip(outs, grads, ("dx", "dscale", "dshift")):
            tr.assert_close(v, wv, tol, what=f"{name} shift {shift}")
            assert clean(buf, v)
        mbx.ln_modulate_backward(doi, xi, fi, EPS, None, *[v for _, v in outs])
        tr.assert_close(outs[0][1], *alone, what=f"no residual, shift {shift}")
        # in place on the residual's gradient
        mbx.ln_modulate_backward(doi, xi, fi, EPS, ri, ri, *[v for _, v in outs[1:]])
        tr.assert_close(ri, *grads[0], what=f"in place, shift {shift}")
    # one operand apart from the others
    mbx.layer_norm(inside(x, 1, stride, nan)[1], w, b, EPS, out=o)
    tr.assert_close(o, *want)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [16, 64, 72, 128, 264, 1024, 4096, 5120, 8192])
def test_a_row_keeps_its_bits(mbx, D, dt):
    """A row's output does not depend on where it starts, nor on the rows beside it."""
    g = gen(D)
    rows = 1300 if D > 300 else 3000
    x, do = acts(g, rows, D, dt), rnd(g, (rows, D), dt, 0.1)
    w, b = rnd(g, (D,), dt, 0.05, 1.0), rnd(g, (D,), dt, 0.1)
    some = slice(5, 12)
    y = mbx.layer_norm(x, w, b)
    assert torch.equal(mbx.layer_norm(x[some], w, b), y[some])
    assert torch.equal(mbx.layer_norm(misaligned(x), w, b), y)
    dx = mbx.layer_norm_backward(do, x, w)[0]
    assert torch.equal(mbx.layer_norm_backward(do[some], x[some], w)[0], dx[some])
    assert torch.equal(mbx.layer_norm_backward(do, misaligned(x), w)[0], dx)
    sc = w.expand(rows, D).contiguous() - 1.0
    token = mbx.ln_modulate_backward(do, x, sc)
    for a, t in zip(mbx.ln_modulate_backward(do, misaligned(x), sc), token):
        assert torch.equal(a, t)
    for a, t in zip(mbx.ln_modulate_backward(do[some], x[some], sc[some]), token):
        assert torch.equal(a, t[some])


@pytest.mark.parametrize("D", [64, 257, 520, 4096])
@pytest.mark.parametrize("mod_rows,seq", [(3, 200), (40, 50), (64, 33), (100, 300), (153, 70), (310, 40)])
def test_gradients_of_many_segments(mbx, D, mod_rows, seq):
    """One part a segment and several, few and many of them, more segments than the device has blocks."""
    seq = max(2, min(seq, 16_000_000 // (mod_rows * D)))
    g = gen(D + mod_rows)
    rows = mod_rows * seq
    x, do = acts(g, rows, D, BF), rnd(g, (rows, D), BF, 0.1)
    sc = rnd(g, (mod_rows, D), BF, 0.1)
    base = check_ln_backward(mbx, x, do, 1 + tr.d(sc), None, scale=sc)
    assert all(torch.equal(a, b) for a, b in zip(mbx.ln_modulate_backward(do, x, sc, EPS), base))
    rng = state(6, 1)
    keep = tr.keep_mask(rows, D, 0.25, 6, 1)
    _, dg = mbx.dropout_gate_add_backward(do, sc, x, 0.25, rng)
    terms = torch.where(keep, tr.d(do) * tr.d(x) / 0.75, 0.0).reshape(mod_rows, seq, D)
    tr.assert_close(dg, terms.sum(1), (8 + seq) * tr.U * terms.abs().sum(1))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [8, 40, 64, 72, 96, 128, 136])
def test_layer_norm_of_narrow_rows(mbx, D, dt):
    """Rows of a head's width: many to a block, several parts, a last part that is not full."""
    g = gen(D)
    for rows in (3, 129, 20011):
        x, do, dres = acts(g, rows, D, dt), rnd(g, (rows, D), dt, 0.1), rnd(g, (rows, D), dt, 0.1)
        w, b = rnd(g, (D,), F32, 0.05, 1.0), rnd(g, (D,), F32, 0.1)
        want, tol = tr.layer_norm(x, w, b, EPS)
        tr.assert_close(mbx.layer_norm(x, w, b, EPS), want, tol)
        check_ln_backward(mbx, x, do, tr.d(w)[None], None, weight=w)
        check_ln_backward(mbx, x, do, tr.d(w)[None], dres, weight=w)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("D,mod_rows,seq", [(4104, 1, 1601), (4608, 3, 333), (5112, 160, 6), (5120, 200, 3)])
def test_ln_modulate_backward_wide_rows(mbx, D, mod_rows, seq, residual):
    """Two rows in work on an SM: odd counts of rows, one part a segment and several."""
    g = gen(D + mod_rows)
    rows = mod_rows * seq
    x, do = acts(g, rows, D, BF), rnd(g, (rows, D), BF, 0.1)
    sc = rnd(g, (mod_rows, D), BF, 0.1)
    dres = rnd(g, (rows, D), BF, 0.1) if residual else None
    base = check_ln_backward(mbx, x, do, 1 + tr.d(sc), dres, scale=sc)
    if residual:
        got = mbx.ln_modulate_backward(do, x, sc, EPS, dres, dx=dres)
        assert all(torch.equal(a, b) for a, b in zip(got, base))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mod_rows", [1, 3, 36])
def test_ln_backward_views_and_in_place(mbx, dt, mod_rows):
    g = gen(9)
    rows, D = 36, 1024
    x, do, dres = acts(g, rows, D, dt), rnd(g, (rows, D), dt, 0.1), rnd(g, (rows, D), dt, 0.1)
    sc = rnd(g, (mod_rows, D), dt, 0.1)
    f = 1 + tr.d(sc)
    base = check_ln_backward(mbx, x, do, f, dres, scale=sc)
    buf, dx = padded(torch.zeros_like(x), fill=7.0)
    sbuf, dsc = padded(torch.zeros_like(sc), fill=7.0)
    hbuf, dsh = padded(torch.zeros_like(sc), fill=7.0)
    got = check_ln_backward(mbx, padded(x)[1], padded(do)[1], f, padded(dres)[1], scale=padded(sc)[1], dx=dx,
                            dscale=dsc, dshift=dsh)
    for b in (buf, sbuf, hbuf):
        assert torch.all(b[:, D:] == 7.0)
    for a, b in zip(base, got):
        assert torch.equal(a, b)                      # padding changes no bit
    check_ln_backward(mbx, misaligned(x), do, f, dres, scale=sc)
    r2 = dres.clone()
    got = mbx.ln_modulate_backward(do, x, sc, EPS, r2, dx=r2)  # in place on the stream's gradient
    assert torch.equal(got[0], base[0]) and got[0].data_ptr() == r2.data_ptr()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mod_rows", [1, 40])
@pytest.mark.parametrize("D", [7, 561, 1027])
def test_ln_backward_unaligned_rows(mbx, D, mod_rows, dt):
    """Rows that all lie differently to 16 bytes; each operand another way; in place."""
    g = gen(D)
    rows = 40
    x, do, dres = acts(g, rows, D, dt), rnd(g, (rows, D), dt, 0.1), rnd(g, (rows, D), dt, 0.1)
    sc = rnd(g, (mod_rows, D), dt, 0.1)
    f = 1 + tr.d(sc)
    base = check_ln_backward(mbx, x, do, f, dres, scale=sc)
    bufs = [padded(torch.zeros_like(t), pad=k, fill=7.0) for t, k in ((x, 3), (sc, 1), (sc, 2))]
    got = check_ln_backward(mbx, padded(x, 5)[1], misaligned(do), f, padded(dres, 8)[1], scale=padded(sc, 2)[1],
                            dx=bufs[0][1], dscale=bufs[1][1], dshift=bufs[2][1])
    assert all(torch.equal(a, b) for a, b in zip(base, got))
    for b, v in bufs:
        assert torch.all(b[:, D:] == 7.0)
    r2 = dres.clone()
    got = mbx.ln_modulate_backward(do, x, sc, EPS, r2, dx=r2)
    assert torch.equal(got[0], base[0])


def test_ln_backward_rows_beyond_32_bits(mbx):
    """Three rows 2^31 - 8 elements apart: every offset past the first row needs 64 bits."""
    stride, D = 2 ** 31 - 8, 256
    buf = torch.empty(2 * stride + D, dtype=BF, device=DEV)
    x = torch.as_strided(buf, (3, D), (stride, 1))
    g = gen(19)
    small = rnd(g, (3, D), BF)
    x.copy_(small)
    do, w = rnd(g, (3, D), BF), rnd(g, (D,), BF, 0.05, 1.0)
    for a, b in zip(mbx.layer_norm_backward(do, x, w), mbx.layer_norm_backward(do, small, w)):
        assert torch.equal(a, b)
    assert torch.equal(mbx.layer_norm(x, w), mbx.layer_norm(small, w))
    s = state(1, 1)
    assert torch.equal(mbx.dropout(x, 0.5, s), mbx.dropout(small, 0.5, s))


def test_ln_backward_is_deterministic_and_chained(mbx):
    g = gen(11)
    x, do, sc = acts(g, 5000, 640, BF), rnd(g, (5000, 640), BF), rnd(g, (2, 640), BF, 0.1)
    first = mbx.ln_modulate_backward(do, x, sc)
    for _ in range(20):  # back to back: each reads the previous call's output
        again = mbx.ln_modulate_backward(do, x, sc)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_gradient_against_differences(mbx):
    """Directional differences of the 64-bit forward formula, of the binary32 gradients:
    each gradient is within its own bound, so the product with v is within their sum."""
    g = gen(12)
    rows, D, m, h = 12, 200, 3, 1e-5
    x, do, sc = rnd(g, (rows, D), F32), rnd(g, (rows, D), F32), rnd(g, (m, D), F32, 0.1)
    sh = torch.zeros(m, D, dtype=torch.float64)
    got = mbx.ln_modulate_backward(do, x, sc, EPS)
    tols = tr.ln_backward(do, x, 1 + tr.d(sc), EPS)

    def loss(x, sc, sh):
        xh, _, _ = tr.ln_stats(x, EPS)
        return ((xh.reshape(m, -1, D) * (1 + sc[:, None]) + sh[:, None]).reshape(rows, D) * tr.d(do)).sum()

    args = [tr.d(x), tr.d(sc), sh]
    for k in range(3):
        v = torch.randn(args[k].shape, generator=gen(k), dtype=torch.float64)
        lo, hi = list(args), list(args)
        lo[k], hi[k] = args[k] - h * v, args[k] + h * v
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        gk = tr.d(got[k])
        bound = ((tols[k][1] + tr.U * gk.abs()) * v.abs()).sum() + 1e-6 * (gk * v).abs().sum()
        assert abs(num - (gk * v).sum()) <= bound


# ---------------------------------------------------------------- dropout


def state(seed, counter):
    return torch.tensor([seed, counter], dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", WIDTHS)
def test_dropout_mask_and_values(mbx, D, dt):
    g = gen(D)
    for rows, p, seed, ctr, off in ((1, 0.5, 1, 0, 0), (41, 0.1, -5, 2 ** 40, 3), (41, 0.0, 7, 7, 7),
                                    (9, 0.999, 2 ** 62, -1, 1)):
        x = rnd(g, (rows, D), dt) + 5.0 if dt == F32 else (rnd(g, (rows, D), F32) + 5.0).to(dt)
        x = x.clamp_min(0.5)
        got = mbx.dropout(x, p, state(seed, ctr), off)
        keep = tr.keep_mask(rows, D, p, seed, ctr + off)
        assert torch.equal((got != 0).cpu(), keep)
        want = torch.where(keep, tr.d(x) / (1 - p), 0.0)
        tr.assert_close(got, want, 4 * tr.U * want.abs())
        y = x.clone()
        assert torch.equal(mbx.dropout(y, p, state(seed, ctr), off, out=y), got)   # in place
        assert torch.equal(mbx.dropout(misaligned(x), p, state(seed, ctr), off), got)  # the mask knows no address


@pytest.mark.parametrize("dt,pdt", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_dropout_gate_add_and_gradients(mbx, D, dt, pdt):
    g = gen(31 + D)
    for m, seq, p in ((1, 1, 0.1), (1, 201, 0.1), (3, 50, 0.5), (77, 1, 0.25), (30, 3, 0.0)):
        rows = m * seq
        x, y, do = (rnd(g, (rows, D), dt) for _ in range(3))
        gate = rnd(g, (m, D), pdt, 0.3)
        s = state(99, 5)
        keep = tr.keep_mask(rows, D, p, 99, 5 + 2)
        gr = tr.d(gate).repeat_interleave(seq, 0)
        z = gr * tr.d(y) / (1 - p)
        out = mbx.dropout_gate_add(x, gate, y, p, s, 2)
        tr.assert_close(out, torch.where(keep, tr.d(x) + z, tr.d(x)), 8 * tr.U * (tr.d(x).abs() + z.abs()), "out")
        assert torch.equal(out.cpu()[~keep], x.cpu()[~keep])
        dy, dgate = mbx.dropout_gate_add_backward(do, gate, y, p, s, 2)
        want = torch.where(keep, tr.d(do) * gr / (1 - p), 0.0)
        tr.assert_close(dy, want, 4 * tr.U * want.abs(), "dy")
        t = torch.where(keep, tr.d(do) * tr.d(y) / (1 - p), 0.0).reshape(m, seq, D)
        tr.assert_close(dgate, t.sum(1), (8 + seq) * tr.U * t.abs().sum(1), "dgate")
        x2 = x.clone()
        assert torch.equal(mbx.dropout_gate_add(x2, gate, y, p, s, 2, out=x2), out)


def test_dropout_drops_non_finite_values(mbx):
    g = gen(8)
    x, y, do, gate = rnd(g, (16, 256), F32), rnd(g, (16, 256), F32), rnd(g, (16, 256), F32), rnd(g, (1, 256), F32)
    keep = tr.keep_mask(16, 256, 0.5, 3, 0).to(DEV)
    bad = torch.where(keep, y, float("inf"))
    bad_do = torch.where(keep, do, float("nan"))
    s = state(3, 0)
    assert torch.equal(mbx.dropout(bad, 0.5, s), mbx.dropout(y, 0.5, s))
    assert torch.equal(mbx.dropout_gate_add(x, gate, bad, 0.5, s), mbx.dropout_gate_add(x, gate, y, 0.5, s))
    for a, b in zip(mbx.dropout_gate_add_backward(bad_do, gate, bad, 0.5, s),
                    mbx.dropout_gate_add_backward(do, gate, y, 0.5, s)):
        assert torch.equal(a, b)


def test_dropout_views(mbx):
    g = gen(14)
    x, y, do, gate = (rnd(g, s, BF) for s in ((30, 512), (30, 512), (30, 512), (3, 512)))
    s = state(4, 4)
    want = mbx.dropout_gate_add(x, gate, y, 0.2, s)
    buf, out = padded(torch.zeros_like(x), fill=7.0)
    mbx.dropout_gate_add(padded(x)[1], padded(gate)[1], padded(y)[1], 0.2, s, out=out)
    assert torch.equal(out, want) and torch.all(buf[:, 512:] == 7.0)
    dy, dg = mbx.dropout_gate_add_backward(do, gate, y, 0.2, s)
    buf, dy2 = padded(torch.zeros_like(x), fill=7.0)
    _, dg2 = mbx.dropout_gate_add_backward(padded(do)[1], gate, padded(y)[1], 0.2, s, dy=dy2)
    assert torch.equal(dy, dy2) and torch.equal(dg, dg2) and torch.all(buf[:, 512:] == 7.0)
    # a batch of shape [B, S, D] has the mask of its rows
    assert torch.equal(mbx.dropout(x.view(3, 10, 512), 0.2, s).view(30, 512), mbx.dropout(x, 0.2, s))


def test_dropout_far_rows(mbx):
    """Rows beyond 2^16 and element offsets beyond 2^31: the tail's mask."""
    D = 7750
    rows = 2 ** 31 // D + 5000
    x = torch.ones((rows, D), dtype=BF, device=DEV)
    got = mbx.dropout(x, 0.5, state(6, 6))
    keep = tr.keep_mask(40, D, 0.5, 6, 6, row0=rows - 40)
    assert torch.equal((got[-40:] != 0).cpu(), keep)


# ---------------------------------------------------------------- rotary positions


def rope_case(g, B, S, hq, hk, hd, dt, order):
    def make(h):
        t = rnd(g, (B, S, h, hd), dt)
        return t if order == "bshd" else t.transpose(1, 2).contiguous().transpose(1, 2)
    return make(hq), make(hk)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("hd,axes", [(128, (44, 42, 42)), (128, (16, 56, 56)), (64, (32, 32)), (256, (128, 64, 32, 32)),
                                     (80, (16, 16)), (80, (80,)), (72, (24, 24, 24)), (6, (2, 2)), (2, (2,)),
                                     (255, (2,)), (50, (20, 10, 20))])
def test_rope(mbx, hd, axes, interleaved, dt):
    g = gen(hd + len(axes))
    fr = mbx.rope_axis_freqs(axes)
    for B, S, hq, hk, order in ((1, 1, 1, 1, "bshd"), (2, 37, 4, 2, "bshd"), (3, 5, 6, 1, "bhsd"), (1, 130, 3, 3, "bhsd")):
        q, k = rope_case(g, B, S, hq, hk, hd, dt, order)
        for pos in (torch.randint(0, 200, (S, len(axes)), generator=g).int(),
                    torch.randint(-10 ** 6, 10 ** 6, (B, S, len(axes)), generator=g).int(),
                    torch.rand(S, len(axes), generator=g) * 100):
            for inverse in (False, True):
                qo, ko = mbx.rope_axes(q, k, pos.to(DEV), fr, axes, interleaved, inverse)
                for t, o in ((q, qo), (k, ko)):
                    tr.assert_close(o, *tr.rope(t, pos, axes, fr, interleaved, inverse))
        only, none = mbx.rope_axes(q, None, pos.to(DEV), fr, axes, interleaved, True)
        assert none is None and torch.equal(only, qo)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("order", ["bshd", "bhsd", "bsh3d"])
def test_rope_in_place_in_a_merged_buffer(mbx, order, interleaved):
    g = gen(2)
    B, S, hd, axes = 2, 33, 128, (44, 42, 42)
    if order == "bshd":
        buf = rnd(g, (B, S, 12, hd), BF)
        q, k = buf[:, :, :6], buf[:, :, 6:9]
    elif order == "bsh3d":
        buf = rnd(g, (B, S, 12, hd), BF)
        q, k = buf.view(B, S, 4, 3, hd)[:, :, :, 0], buf.view(B, S, 4, 3, hd)[:, :, :, 1]
    else:
        buf = rnd(g, (B, 12, S, hd), BF)
        q, k = buf[:, :6].transpose(1, 2), buf[:, 6:9].transpose(1, 2)
    before = buf.clone()
    pos, fr = torch.randint(0, 64, (S, 3), generator=g).int().to(DEV), mbx.rope_axis_freqs(axes)
    want = mbx.rope_axes(q, k, pos, fr, axes, interleaved)
    mbx.rope_axes(q, k, pos, fr, axes, interleaved, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    v = {"bshd": (slice(None), slice(None), slice(9, None)), "bhsd": (slice(None), slice(9, None)),
         "bsh3d": (slice(None), slice(None), slice(2, None, 3))}[order]
    assert torch.equal(buf[v], before[v])             # V is left as it was


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dt", [BF, F32])
def test_rope_keeps_its_bits(mbx, dt, interleaved):
    """A head's output depends neither on the access width that its place allows nor on the other heads."""
    g = gen(31)
    q = rnd(g, (1, 50, 6, 64), dt)
    pos, fr = torch.randint(0, 200, (50, 2), generator=g).int().to(DEV), mbx.rope_axis_freqs((32, 32))
    want, _ = mbx.rope_axes(q, None, pos, fr, (32, 32), interleaved)
    for lead in (1, 8 // q.element_size(), 16 // q.element_size()):
        buf = torch.zeros(q.numel() + lead, dtype=dt, device=DEV)
        v = buf[lead:].view(q.shape)
        v.copy_(q)
        got, _ = mbx.rope_axes(v, None, pos, fr, (32, 32), interleaved)
        assert torch.equal(got, want)
    assert torch.equal(mbx.rope_axes(q[:, 3:9, 2:3], None, pos[3:9], fr, (32, 32), interleaved)[0], want[:, 3:9, 2:3])


def test_rope_misaligned_and_gradient(mbx):
    """A slice that starts at no 16-byte boundary; and <rope(q), r> = <q, inverse(r)>."""
    g = gen(21)
    axes = (16, 24, 24)
    pos, fr = torch.randint(0, 500, (19, 3), generator=g).int().to(DEV), mbx.rope_axis_freqs(axes)
    q, r = rnd(g, (1, 19, 3, 64), F32), rnd(g, (1, 19, 3, 64), F32)
    a, _ = mbx.rope_axes(q, None, pos, fr, axes)
    m = misaligned(q.reshape(19, 192)).view(1, 19, 3, 64)
    b, _ = mbx.rope_axes(m, None, pos, fr, axes)
    assert torch.equal(a, b)
    c, _ = mbx.rope_axes(r, None, pos, fr, axes, inverse=True)
    lhs, rhs = (tr.d(a) * tr.d(r)).sum(), (tr.d(q) * tr.d(c)).sum()
    pair = lambda t: tr.d(t).abs().unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(-1, -1, -1, -1, 2).flatten(-2)
    assert abs(lhs - rhs) <= 9 * tr.U * ((pair(q) * tr.d(r).abs()) + (pair(r) * tr.d(q).abs())).sum()


def test_rope_broadcast_batch_and_positions(mbx):
    """A batch of stride 0 (an input only), positions given for the batch, three-dimensional Q."""
    g = gen(23)
    axes, fr = (16, 24, 24), mbx.rope_axis_freqs((16, 24, 24))
    q = rnd(g, (1, 9, 4, 64), BF)
    pos = torch.randint(0, 50, (9, 3), generator=g).int().to(DEV)
    one, _ = mbx.rope_axes(q, None, pos, fr, axes)
    four, _ = mbx.rope_axes(q.expand(4, -1, -1, -1), None, pos[None].expand(4, -1, -1).contiguous(), fr, axes)
    assert torch.equal(four, one.expand(4, -1, -1, -1))
    three, _ = mbx.rope_axes(q[0], None, pos, fr, axes)
    assert three.shape == (9, 4, 64) and torch.equal(three, one[0])


def test_rope_infinite_position_stays_alone(mbx):
    pos = torch.tensor([[0.0], [float("inf")], [2.0]], device=DEV)
    fr = mbx.rope_axis_freqs((8,))
    q = torch.ones((1, 3, 2, 8), device=DEV)
    o, _ = mbx.rope_axes(q, None, pos, fr, (8,))
    assert o[0, 1].isnan().all() and not o[0, [0, 2]].isnan().any() and torch.equal(o[0, 0], q[0, 0])


# ---------------------------------------------------------------- as they are used together


def test_block_of_gradients_on_a_side_stream_and_in_a_graph(mbx):
    """A pre-norm block's half: LN + modulate, rotation, gated residual with dropout, forward and
    backward; eager on a side stream and captured, replayed twice with a new counter in between."""
    g = gen(77)
    B, S, H, hd, p = 2, 24, 4, 64, 0.2
    D, rows = H * hd, B * S
    axes = (16, 24, 24)
    x, y, do = rnd(g, (rows, D), BF), rnd(g, (rows, D), BF), rnd(g, (rows, D), BF, 0.1)
    sc, sh, gate = (rnd(g, (B, D), BF, 0.1) for _ in range(3))
    pos, fr = torch.randint(0, 64, (S, 3), generator=g).int().to(DEV), mbx.rope_axis_freqs(axes)
    rng = state(5, 0)

    def block():
        n = mbx.ln_modulate(x, sc, sh, EPS, "high")
        q, _ = mbx.rope_axes(n.view(B, S, H, hd), None, pos, fr, axes)
        out = mbx.dropout_gate_add(x, gate, q.view(rows, D), p, rng, 1)
        dq, dgate = mbx.dropout_gate_add_backward(do, gate, q.view(rows, D), p, rng, 1)
        dn, _ = mbx.rope_axes(dq.view(B, S, H, hd), None, pos, fr, axes, inverse=True)
        dx, dsc, dsh = mbx.ln_modulate_backward(dn.view(rows, D), x, sc, EPS, dresidual=do)
        return out, dgate, dx, dsc, dsh

    want = block()
    n = mbx.ln_modulate(x, sc, sh, EPS, "high")
    q, _ = mbx.rope_axes(n.view(B, S, H, hd), None, pos, fr, axes)
    dq, _ = mbx.dropout_gate_add_backward(do, gate, q.view(rows, D), p, rng, 1)
    dn, _ = mbx.rope_axes(dq.view(B, S, H, hd), None, pos, fr, axes, inverse=True)
    for got, (w, tol) in zip(want[2:], tr.ln_backward(dn.view(rows, D), x, 1 + tr.d(sc), EPS, do)):
        tr.assert_close(got, w, tol)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block()
    for counter in (0, 9):
        rng[1] = counter
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, block()))


def test_two_graphs_of_one_call_keep_their_workspaces(mbx):
    g = gen(78)
    x, sc = rnd(g, (3000, 512), BF), rnd(g, (1, 512), BF, 0.1)
    dos = [rnd(g, (3000, 512), BF) for _ in range(2)]
    want = [mbx.ln_modulate_backward(d_, x, sc) for d_ in dos]
    graphs, outs = [], []
    for d_ in dos:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(mbx.ln_modulate_backward(d_, x, sc))
        graphs.append(gr)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


@pytest.mark.parametrize("D", [520, 561, 5120])
@pytest.mark.parametrize("mod_rows,seq", [(1, 900), (40, 3), (120, 1)])
def test_gradients_that_are_not_wanted(mbx, D, mod_rows, seq):
    """The C entry points take null for a parameter gradient; the others keep their bits."""
    g = gen(D + seq)
    rows = mod_rows * seq
    x, y, do = rnd(g, (rows, D), BF), rnd(g, (rows, D), BF), rnd(g, (rows, D), BF, 0.1)
    f = rnd(g, (mod_rows, D), BF, 0.1)
    rng = state(3, 4)
    L, v, s = mbx.lib(), mbx._view, torch.cuda.current_stream().cuda_stream
    full = mbx.ln_modulate_backward(do, x, f, EPS)
    need = mbx.param_grad_workspace(rows, D, mod_rows, BF)
    ws = torch.empty(max(need, 4) // 4, device=DEV)
    for want in ((True, False), (False, True), (False, False)):
        dx = torch.full_like(x, float("nan"))
        dp = [torch.full_like(f, float("nan")) if w else None for w in want]
        wargs = (ws.data_ptr(), need) if any(want) and need else (None, 0)
        st = L.mbx_ln_modulate_backward(v(dx), *[None if t is None else v(t) for t in dp], v(do), v(x), v(f), None, EPS,
                                        *wargs, s)
        assert st == 0 and torch.equal(dx, full[0])
        assert all(t is None or torch.equal(t, full[1 + i]) for i, t in enumerate(dp))
    dy = torch.full_like(y, float("nan"))
    assert L.mbx_dropout_gate_add_backward(v(dy), None, v(do), v(f), v(y), 0.3, rng.data_ptr(), 0, None, 0, s) == 0
    assert torch.equal(dy, mbx.dropout_gate_add_backward(do, f, y, 0.3, rng)[0])


def test_workspace_is_checked(mbx):
    x, sc = torch.zeros((3000, 512), dtype=BF, device=DEV), torch.zeros((1, 512), dtype=BF, device=DEV)
    need = mbx.param_grad_workspace(3000, 512, 1, BF)
    assert need > 0 and mbx.param_grad_workspace(3000, 512, 3000, BF) == 0
    out = [torch.empty_like(x), torch.empty_like(sc), torch.empty_like(sc)]
    ws = torch.empty(need // 4, device=DEV)
    chk = lambda w: mbx.check_ln_modulate_backward(*out, x, x.clone(), sc, workspace=w)
    assert chk(ws) == 0 and chk(None) == -1 and chk(ws[:-1]) == -10 and chk(torch.empty(need // 4 + 1, device=DEV)[1:]) == -7


def test_calls_from_several_threads(mbx):
    """Host threads with a stream each, the same kernels for the first time at once."""
    from concurrent.futures import ThreadPoolExecutor
    g = gen(91)
    x, do = rnd(g, (4000, 1536), BF), rnd(g, (4000, 1536), BF)
    scs = [rnd(g, (1, 1536), BF, 0.1) for _ in range(6)]

    def work(sc):
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(st):
            for _ in range(10):
                r = mbx.ln_modulate_backward(do, x, sc)
        st.synchronize()
        return r

    torch.cuda.synchronize()
    with ThreadPoolExecutor(6) as ex:
        got = list(ex.map(work, scs))
    for sc, r in zip(scs, got):
        assert all(torch.equal(a, b) for a, b in zip(r, mbx.ln_modulate_backward(do, x, sc)))


COLD = """
import torch, modulation_bit_exact_gb300 as mbx
x = torch.randn(3000, 512, device="cuda").bfloat16()
sc = torch.zeros(1, 512, device="cuda").bfloat16()
rng = torch.tensor([1, 2], device="cuda")
pos = torch.zeros(3000, 1, dtype=torch.int32, device="cuda")
fr = mbx.rope_axis_freqs((64,))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = mbx.layer_norm(x)
    b = mbx.ln_modulate_backward(x, x, sc)
    c = mbx.dropout_gate_add(x, sc, x, 0.5, rng)
    d = mbx.dropout_gate_add_backward(x, sc, x, 0.5, rng)
    e = mbx.rope_axes(x.view(1, 3000, 8, 64), None, pos, fr, (64,))
g.replay()
torch.cuda.synchronize()
want = (mbx.layer_norm(x), *mbx.ln_modulate_backward(x, x, sc), mbx.dropout_gate_add(x, sc, x, 0.5, rng),
        *mbx.dropout_gate_add_backward(x, sc, x, 0.5, rng))
assert all(torch.equal(p, q) for p, q in zip((a, *b, c, *d), want))
"""


def test_first_calls_inside_a_capture(mbx):
    """A program whose first calls are captured: nothing needs a warm-up outside."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", COLD], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_state_on_the_host_is_refused(mbx):
    x = torch.zeros((4, 64), device=DEV)
    with pytest.raises(mbx.MbxError) as e:
        mbx.dropout(x, 0.5, torch.zeros(2, dtype=torch.int64))
    assert e.value.status == -9
    with pytest.raises(mbx.MbxError) as e:
        mbx.layer_norm(x, torch.ones(64))  # a weight on the host
    assert e.value.status == -9
