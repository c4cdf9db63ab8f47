"""Properties of the training path that its bounds against binary64 cannot show: results that are
exact, and results that two calls have to share bit for bit.
"""
import pytest
import torch

from . import train_ref as tr

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mbx():
    import modulation_bit_exact_gb300 as m
    m.lib()
    return m


EPS = 1e-6


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, shape, dt, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dt).to(DEV)


@pytest.mark.parametrize("dt,pdt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("D", [64, 257, 520, 4096])
@pytest.mark.parametrize("p", [0.1, 0.25, 1 / 3])
def test_gated_dropout_gradients_are_the_formulas_products(mbx, p, D, dt, pdt):
    """dy = dout * gate * inv and, a row each, dgate = dout * (y * inv), inv = 1 / (1 - p) in
    binary32: every product rounded, in this order, so equal bit for bit to the same products in
    torch."""
    g = gen(D)
    for m, seq in ((2, 150), (300, 1)):
        do, y, gate = rnd(g, (m * seq, D), dt), rnd(g, (m * seq, D), dt), rnd(g, (m, D), pdt, 0.1)
        rng = torch.tensor([12, 34], device=DEV)
        keep = tr.keep_mask(m * seq, D, p, 12, 34).to(DEV)
        inv = torch.tensor(1.0 / (1.0 - p), dtype=torch.float64).float().to(DEV)
        dy, dgate = mbx.dropout_gate_add_backward(do, gate, y, p, rng)
        zero = torch.zeros((), device=DEV)
        want = torch.where(keep, do.float() * gate.float().repeat_interleave(seq, 0) * inv, zero).to(dt)
        assert torch.equal(dy, want)
        if seq == 1:
            assert torch.equal(dgate, torch.where(keep, do.float() * (y.float() * inv), zero).to(pdt))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [8, 64, 72, 96, 121, 128, 136, 1024])
def test_a_row_keeps_its_bits_whoever_shares_its_factor(mbx, D, dt):
    """dx of a row alone, among others, and with a factor of its own."""
    g = gen(D)
    rows = 300
    x, do, dres, w = rnd(g, (rows, D), dt), rnd(g, (rows, D), dt), rnd(g, (rows, D), dt), rnd(g, (D,), dt, 0.05, 1.0)
    sc = rnd(g, (1, D), dt, 0.1)
    for r in (None, dres):
        dx = mbx.layer_norm_backward(do, x, w, dresidual=r)[0]
        for i in range(0, rows, 7):
            one = slice(i, i + 1)
            alone = mbx.layer_norm_backward(do[one], x[one], w, dresidual=None if r is None else r[one])[0]
            assert torch.equal(alone, dx[one])
        shared = mbx.ln_modulate_backward(do, x, sc, dresidual=r)[0]
        token = mbx.ln_modulate_backward(do, x, sc.expand(rows, D).contiguous(), dresidual=r)
        assert torch.equal(token[0], shared)
        pairs = sc.expand(rows // 2, D).contiguous()
        assert torch.equal(mbx.ln_modulate_backward(do, x, pairs, dresidual=r)[0], shared)


def far_rows(D, dt):
    """Rows of a far mean: constant ones, and ones whose elements lie within a factor of two."""
    g = gen(D)
    rows = [torch.full((1, D), v) for v in (0.7, 300.0, -1000.0, 10000.0)]
    rows += [m + m * s * torch.randn(1, D, generator=g).clamp(-4, 4)
             for m, s in ((1000.0, 2.0 ** -6), (-300.0, 0.08), (20.0, 0.05), (1e6, 2.0 ** -7))]
    if dt == F32:
        rows += [m + s * torch.randn(1, D, generator=g) for m, s in ((1000.0, 0.01), (-30000.0, 1.0), (5.0, 1e-3))]
    return torch.cat(rows).to(dt).to(DEV)


def far_scale(x):
    """With e = 41u * mean|x| * rstd, the error of a rounded mean in standard deviations (40 roundings
    of the sum, one of 1/D): the deviations from the rounded mean are e away at most; their own mean,
    which is taken off, is known to 42u * (1 + e), and the variance to 45u * (1 + e)^2 and 84u * e.  So
    xh is off by less than 64u * (1 + e)^2 * (|xh| + 1), whatever the mean."""
    xh, rstd, X = tr.ln_stats(x, EPS)
    return xh, rstd, (1 + 41 * tr.U * X).square()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [40, 64, 104, 112, 120, 1000, 1031, 2056, 5120, 8192])
def test_rows_far_from_zero(mbx, D, dt):
    x = far_rows(D, dt)
    rows = len(x)
    g = gen(D + 1)
    w, b = rnd(g, (D,), dt, 0.05, 1.0), rnd(g, (D,), dt, 0.1)
    xh, rstd, e2 = far_scale(x)
    want = xh * tr.d(w) + tr.d(b)
    many = x.repeat(620 // rows + 60, 1)  # enough for two rows at a time
    for t in (x, many):
        got = mbx.layer_norm(t, w, b, EPS)
        tr.assert_close(got[:rows], want, tr.K * tr.U * (e2 * (xh.abs() + 1) * tr.d(w).abs() + tr.d(b).abs()))
        assert torch.equal(got[-rows:], got[:rows])
    do, dres = rnd(g, (rows, D), dt, 0.1), rnd(g, (rows, D), dt, 0.1)
    gy = tr.d(do) * tr.d(w)
    a = e2 * (xh.abs() + 1)
    c1, c2 = gy.mean(-1, keepdim=True), (gy * xh).mean(-1, keepdim=True)
    dx = rstd * (gy - c1 - xh * c2)
    tol = tr.K * tr.U * rstd * (gy.abs() + e2 * gy.abs().mean(-1, keepdim=True) + a * (gy.abs() * a).mean(-1, keepdim=True))
    sc = (w.float() - 1.0)
    for r in (None, dres):
        want = dx if r is None else dx + tr.d(r)
        lim = tol if r is None else tol + 2 * tr.U * want.abs()
        gx, gw, gb = mbx.layer_norm_backward(do, x, w, EPS, r)
        tr.assert_close(gx, want, lim, "dx")
        tr.assert_close(gw, (tr.d(do) * xh).sum(0), (tr.K + rows) * tr.U * (tr.d(do).abs() * a).sum(0), "dweight")
        # a row each: the factor 1 + (w - 1) in binary32
        f = 1 + tr.d(sc)
        gy1 = tr.d(do) * f
        c1t, c2t = gy1.mean(-1, keepdim=True), (gy1 * xh).mean(-1, keepdim=True)
        want1 = rstd * (gy1 - c1t - xh * c2t)
        want1 = want1 if r is None else want1 + tr.d(r)
        gx, gs, gh = mbx.ln_modulate_backward(do, x, sc.expand(rows, D).contiguous(), EPS, r)
        tr.assert_close(gx, want1, lim + 2 * tr.U * (rstd * gy1.abs()), "dx, a row each")
        tr.assert_close(gs, tr.d(do) * xh, tr.K * tr.U * tr.d(do).abs() * a, "dscale")


@pytest.mark.parametrize("D", [64, 104, 1000, 5120, 8192])
def test_a_constant_bfloat16_row_is_zero(mbx, D):
    """The sum of equal bfloat16 values is exact: each deviation is 2u of the value at most (the mean's
    rounding, that of 1/D), and is known to 4u (1/D and three products)."""
    x = torch.tensor([[1000.0], [10000.0], [-0.3], [3e-5]], device=DEV).to(BF).expand(4, D).contiguous()
    y = mbx.layer_norm(x, None, None, EPS)
    X = tr.d(x).abs() / EPS ** 0.5
    assert (tr.d(y).abs() <= 9 * tr.U * tr.U * X).all()


@pytest.mark.parametrize("D", [64, 1000, 4096, 8192])
def test_only_few_segments_are_split(mbx, D):
    """A second kernel joins the parts of a segment, with the segment as a block row of its grid: more
    than four segments an SM are one part each, however many rows they have."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for seq in (2, 40, 3000, 100_000):
        for m in (4 * sms + 1, 5 * sms, 7 * sms + 3, 32768, 65535, 65536, 1_000_000):
            if m * seq < 2 ** 32:
                assert mbx.param_grad_workspace(m * seq, D, m, BF) == 0


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [8, 62, 64, 96, 128, 562, 1024, 4096, 4106, 5120, 8192])
def test_parameter_gradients_count_every_row_once(mbx, D, dt):
    """Whole numbers whose sums are exact in any order: with rows of +-1 in equal numbers and eps = 0,
    xh is +-1, and with p = 1/2 a kept element counts twice.  One part and many, parts and rounds that
    are not full, more segments than blocks."""
    g = torch.Generator(device=DEV).manual_seed(D)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g, device=DEV).to(dt)
    rng = torch.tensor([5, 6], device=DEV)
    half = torch.ones(D, device=DEV)
    half[D // 2:] = -1.0
    for m, seq in ((1, 20011), (1, 701), (2, 9), (3, 333), (40, 50), (64, 131), (153, 70), (310, 3), (700, 2)):
        seq = max(2, min(seq, 24_000_000 // (m * D)))
        rows = m * seq
        sign = torch.randint(0, 2, (rows, 1), generator=g, device=DEV) * 2 - 1
        xh = half * sign
        x, do, y, dres = xh.to(dt), whole(rows, D), whole(rows, D), whole(rows, D)
        sc = torch.zeros(m, D, device=DEV)
        seg = lambda t: t.float().view(m, seq, D).sum(1)
        for r in (None, dres):
            _, dsc, dsh = mbx.ln_modulate_backward(do, x, sc, 0.0, r)
            assert torch.equal(dsc, seg(do.float() * xh)), (m, seq)
            assert torch.equal(dsh, seg(do)), (m, seq)
        if m == 1:
            _, dw, db = mbx.layer_norm_backward(do, x, torch.ones(D, device=DEV), 0.0)
            assert torch.equal(dw, dsc[0]) and torch.equal(db, dsh[0])
        keep = mbx.dropout(torch.ones(rows, D, device=DEV), 0.5, rng)  # 2 or 0
        _, dg = mbx.dropout_gate_add_backward(do, sc, y, 0.5, rng)
        assert torch.equal(dg, seg(do.float() * y.float() * keep)), (m, seq)


@pytest.mark.parametrize("dt,pdt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("D", [8, 72, 561, 4104])
def test_gradient_of_a_bias_alone(mbx, D, dt, pdt):
    g = gen(D)
    for rows in (1, 2, 40, 3001):
        x, do = rnd(g, (rows, D), dt), rnd(g, (rows, D), dt)
        db = torch.full((D,), float("nan"), dtype=pdt, device=DEV)
        dx, dw, out = mbx.layer_norm_backward(do, x, None, EPS, dbias=db)
        assert dw is None and out.data_ptr() == db.data_ptr()
        want = mbx.layer_norm_backward(do, x, torch.ones(D, dtype=pdt, device=DEV), EPS)
        assert torch.equal(db, want[2]) and torch.equal(dx, want[0])
        assert torch.equal(mbx.layer_norm_backward(do, x, None, EPS)[0], dx)


def test_calls_record_no_graph_and_serve_a_function(mbx):
    """Outputs carry no grad_fn; a torch.autograd.Function around a pair of calls has the gradients."""

    class LayerNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias):
            ctx.save_for_backward(x, weight)
            return mbx.layer_norm(x, weight, bias)

        @staticmethod
        def backward(ctx, dout):
            return mbx.layer_norm_backward(dout.contiguous(), *ctx.saved_tensors)

    g = gen(3)
    leaves = [rnd(g, s, F32) for s in ((30, 200), (200,), (200,))]
    for t in leaves:
        t.requires_grad_()
    assert mbx.layer_norm(*leaves).grad_fn is None and not mbx.layer_norm(*leaves).requires_grad
    loss = LayerNorm.apply(*leaves).sum()                                  # its gradient is expanded from one number
    got = torch.autograd.grad(loss, leaves)
    ones = torch.ones(30, 200)
    (dx, tol), (dw, wtol), (db, btol) = tr.ln_backward(ones, leaves[0], leaves[1].detach()[None], EPS)
    tr.assert_close(got[0], dx, tol)
    tr.assert_close(got[1], dw[0], wtol[0])
    tr.assert_close(got[2], db[0], btol[0])


def test_row_shards_of_the_training_path(mbx):
    """What shard.py says of blocks of rows: dx and per-token gradients are the unsharded call's, the
    parts of a shared parameter's gradient add up to it, and a block's dropout mask is that of its own
    rows, the same for equal states, another for another seed."""
    from modulation_bit_exact_gb300.shard import row_shard
    g = gen(8)
    rows, D, world = 96, 136, 4
    x, y = rnd(g, (rows, D), BF), rnd(g, (rows, D), BF)
    do = torch.randint(-3, 4, (rows, D), generator=g).to(BF).to(DEV)
    sc = rnd(g, (2, D), F32, 0.1)
    dx, dsc, dsh = mbx.ln_modulate_backward(do, x, sc)
    parts, masks = torch.zeros_like(dsh), []
    for rank in range(world):
        lo, hi, m0, m1 = row_shard(rows, 2, world, rank)
        sx, _, sh = mbx.ln_modulate_backward(do[lo:hi], x[lo:hi], sc[m0:m1])
        assert torch.equal(sx, dx[lo:hi])
        parts[m0:m1] += sh
        mask = lambda seed: mbx.dropout(torch.ones_like(x[lo:hi]), 0.5, torch.tensor([seed, 3], device=DEV)) != 0
        assert torch.equal(mask(9).cpu(), tr.keep_mask(hi - lo, D, 0.5, 9, 3))
        masks.append(mask(100 + rank))
        rng = torch.tensor([100 + rank, 3], device=DEV)
        out = mbx.dropout_gate_add(torch.zeros_like(y[lo:hi]), sc[m0:m1], torch.ones_like(y[lo:hi]), 0.5, rng)
        dy, _ = mbx.dropout_gate_add_backward(torch.ones_like(y[lo:hi]), sc[m0:m1], y[lo:hi], 0.5, rng)
        assert torch.equal(out, dy) and torch.equal(dy != 0, masks[-1])
    assert torch.equal(parts, dsh)                                         # whole numbers: exact in any order
    assert not any(torch.equal(masks[0], m) for m in masks[1:])


def test_masks_of_steps_and_layers_differ(mbx):
    """A counter that each step advances by the number of layers, a layer's offset on top: no two calls
    share a mask, and rng[1] + offset alone decides."""
    ones, layers, seen = torch.ones(8, 256, device=DEV), 3, {}
    for step in range(4):
        for layer in range(layers):
            rng = torch.tensor([7, step * layers], device=DEV)
            seen[step, layer] = mbx.dropout(ones, 0.5, rng, offset=layer)
    all_ = list(seen.values())
    assert not any(torch.equal(a, b) for i, a in enumerate(all_) for b in all_[:i])
    assert torch.equal(seen[1, 1], mbx.dropout(ones, 0.5, torch.tensor([7, layers + 1], device=DEV)))
