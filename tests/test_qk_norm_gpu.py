"""The norm and rotation of Q and K heads, and its gradients, on the GPU against
plain 64-bit references: heads of every width class, grouped K heads, all head
layouts, one token and many, both types, values where a norm goes wrong.
"""
import pytest
import torch

from . import heads_ref as hr
from . import train_ref as tr

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
TYPES = [(BF, BF), (BF, F32), (F32, F32)]
# one pair; partial turns; widths of 16, 8 and single-element accesses, odd ones; every group size
SHAPES = [(2, (2,)), (8, (2, 2, 4)), (40, (40,)), (64, (16, 24, 24)), (72, (36,)), (80, (8, 16, 16)), (96, (32, 32)),
          (100, (50,)), (127, (60,)), (128, (44, 42, 42)), (128, (64, 8, 8, 8)), (192, (64, 64)), (250, (100, 150)),
          (255, (2,)), (256, (64, 96, 96)), (256, (128,))]


@pytest.fixture(scope="module")
def mbx():
    import modulation_bit_exact_gb300 as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, shape, dt, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dt).to(DEV)


def layout(t, order):
    """t [B, S, H, hd] with its values in another order in memory."""
    if order == "bhsd":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if order == "merged":  # Q, K and V side by side in a token
        buf = torch.full((*t.shape[:2], t.shape[2] + 3, t.shape[3]), float("nan"), dtype=t.dtype, device=t.device)
        buf[:, :, 2:2 + t.shape[2]] = t
        return buf[:, :, 2:2 + t.shape[2]]
    if order == "odd":  # no head starts at a 16-byte boundary but by chance
        buf = torch.full((*t.shape[:3], t.shape[3] + 1), float("nan"), dtype=t.dtype, device=t.device)
        buf[..., 1:] = t
        return buf[..., 1:]
    return t


def case(g, B, S, hq, hk, hd, dt, order="bshd"):
    """Heads of different sizes, a zero one and one with an outlier among them."""
    def one(H):
        t = torch.randn((B, S, H, hd), generator=g) * (torch.rand((H, 1), generator=g) * 4 + 0.05)
        t[0, S // 2, H // 2] = 0.0
        t[B - 1, S - 1, H - 1, hd - 1] = 300.0
        return layout(t.to(dt).to(DEV), order)
    return one(hq), one(hk)


def positions(g, B, S, n):
    return [torch.randint(0, 200, (S, n), generator=g).int(),
            torch.randint(-10 ** 6, 10 ** 6, (B, S, n), generator=g).int(), torch.rand(S, n, generator=g) * 100]


SIZES = ((1, 1, 1, 1, "bshd"), (2, 37, 4, 2, "merged"), (3, 5, 6, 1, "bhsd"), (1, 130, 3, 9, "odd"))


@pytest.mark.parametrize("dt,wdt", TYPES)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("hd,axes", SHAPES)
def test_forward(mbx, hd, axes, interleaved, dt, wdt):
    g = gen(hd + len(axes))
    fr = mbx.rope_axis_freqs(axes)
    wq, wk = rnd(g, (hd,), wdt, 0.1, 1.0), rnd(g, (hd,), wdt, 0.1, 1.0)
    for B, S, hq, hk, order in SIZES:
        q, k = case(g, B, S, hq, hk, hd, dt, order)
        for pos in positions(g, B, S, len(axes)):
            qo, ko = mbx.qk_norm_rope(q, k, wq, wk, pos.to(DEV), fr, axes, interleaved, EPS)
            for t, w, o in ((q, wq, qo), (k, wk, ko)):
                tr.assert_close(o, *hr.norm_rope(t, w, pos, axes, fr, interleaved, EPS), what=f"{B, S, hq, hk, order}")
        only, none = mbx.qk_norm_rope(q, None, None, None, pos.to(DEV), fr, axes, interleaved, 0.25)
        assert none is None
        tr.assert_close(only, *hr.norm_rope(q, None, pos, axes, fr, interleaved, 0.25))


@pytest.mark.parametrize("dt,wdt", TYPES)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("hd,axes", SHAPES)
def test_backward(mbx, hd, axes, interleaved, dt, wdt):
    g = gen(1000 + hd + len(axes))
    fr = mbx.rope_axis_freqs(axes)
    wq, wk = rnd(g, (hd,), wdt, 0.1, 1.0), rnd(g, (hd,), wdt, 0.1, 1.0)
    for B, S, hq, hk, order in SIZES:
        q, k = case(g, B, S, hq, hk, hd, dt, order)
        dq, dk = rnd(g, (B, S, hq, hd), dt, 0.1), layout(rnd(g, (B, S, hk, hd), dt, 0.1), order)
        for pos in positions(g, B, S, len(axes)):
            got = mbx.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos.to(DEV), fr, axes, interleaved, EPS)
            assert got[0].shape == q.shape and got[2].dtype == wdt and got[2].shape == (hd,)
            for i, (do, x, w) in enumerate(((dq, q, wq), (dk, k, wk))):
                (dx, tx), (dw, tw) = hr.norm_rope_backward(do, x, w, pos, axes, fr, interleaved, EPS)
                tr.assert_close(got[i], dx, tx, what=f"dx {i} {B, S, hq, hk, order}")
                tr.assert_close(got[2 + i], dw, tw, what=f"dw {i} {B, S, hq, hk, order}")
        only = mbx.qk_norm_rope_backward(dq, None, q, None, None, None, pos.to(DEV), fr, axes, interleaved, 0.25)
        assert only[1] is None and only[2] is None and only[3] is None
        (dx, tx), _ = hr.norm_rope_backward(dq, q, None, pos, axes, fr, interleaved, 0.25)
        tr.assert_close(only[0], dx, tx)


@pytest.mark.parametrize("dt", [BF, F32])
def test_backward_of_many_tokens(mbx, dt):
    """Every warp of the grid walks several tokens; the weights' gradients repeat bit for bit."""
    g = gen(5)
    axes, fr = (16, 24, 24), mbx.rope_axis_freqs((16, 24, 24))
    q, k = case(g, 3, 2731, 3, 1, 64, dt)
    dq, dk = rnd(g, q.shape, dt, 0.1), rnd(g, k.shape, dt, 0.1)
    wq, wk = rnd(g, (64,), F32, 0.1, 1.0), rnd(g, (64,), F32, 0.1, 1.0)
    pos = torch.randint(0, 200, (2731, 3), generator=g).int()
    got = mbx.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos.to(DEV), fr, axes)
    for i, (do, x, w) in enumerate(((dq, q, wq), (dk, k, wk))):
        (dx, tx), (dw, tw) = hr.norm_rope_backward(do, x, w, pos, axes, fr, True, EPS)
        tr.assert_close(got[i], dx, tx)
        tr.assert_close(got[2 + i], dw, tw)
    again = mbx.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos.to(DEV), fr, axes)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("interleaved", [True, False])
def test_backward_against_differences(mbx, interleaved):
    """<gradient, direction> against the central difference of the float32 forward call, h = 2^-7.  The third
    derivative of x/rms(x) along a direction as large as x is at most 15 of its values, so h^2/6 of it is
    2^-12.7 of them; the two calls' roundings, 32u each over 2h, are 2^-12: together below 2^-11."""
    g = gen(8)
    axes, fr, h = (8, 12, 12), mbx.rope_axis_freqs((8, 12, 12)), 2.0 ** -7
    x = rnd(g, (2, 7, 3, 40), F32) + 0.5
    w, r = rnd(g, (40,), F32, 0.1, 1.0), rnd(g, (2, 7, 3, 40), F32)
    pos = torch.randint(0, 50, (7, 3), generator=g).int().to(DEV)
    dx, _, dw, _ = mbx.qk_norm_rope_backward(r, None, x, None, w, None, pos, fr, axes, interleaved, EPS)
    ux, uw = rnd(g, x.shape, F32), rnd(g, w.shape, F32)
    f = lambda x, w: mbx.qk_norm_rope(x, None, w, None, pos, fr, axes, interleaved, EPS)[0]
    for got, terms, hi, lo in ((tr.d(dx) * tr.d(ux), tr.d(dx).abs() * tr.d(ux).abs(), f(x + h * ux, w), f(x - h * ux, w)),
                               (tr.d(dw) * tr.d(uw), tr.d(dw).abs() * tr.d(uw).abs(), f(x, w + h * uw), f(x, w - h * uw))):
        want = ((tr.d(hi) - tr.d(lo)) * tr.d(r)).sum() / (2 * h)
        scale = terms.sum() + (tr.d(hi).abs() * tr.d(r).abs()).sum()
        assert abs(got.sum() - want) <= 2.0 ** -11 * scale


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("order", ["bshd", "bhsd", "bsh3d"])
def test_in_place_in_a_merged_buffer(mbx, order, interleaved, dt):
    g = gen(2)
    B, S, hd, axes = 2, 33, 128, (44, 42, 42)
    if order == "bhsd":
        buf = rnd(g, (B, 12, S, hd), dt)
        q, k, v = buf[:, :6].transpose(1, 2), buf[:, 6:9].transpose(1, 2), buf[:, 9:]
    else:
        buf = rnd(g, (B, S, 12, hd), dt)
        q, k, v = buf[:, :, :6], buf[:, :, 6:9], buf[:, :, 9:]
        if order == "bsh3d":
            q, k, v = (buf.view(B, S, 4, 3, hd)[:, :, :, i] for i in range(3))
    before, x = v.clone(), (q.clone(), k.clone())
    w = rnd(g, (hd,), F32, 0.1, 1.0)
    pos, fr = torch.randint(0, 64, (S, 3), generator=g).int().to(DEV), mbx.rope_axis_freqs(axes)
    want = mbx.qk_norm_rope(q, k, w, w, pos, fr, axes, interleaved)
    grads = mbx.qk_norm_rope_backward(q, k, *x, w, w, pos, fr, axes, interleaved)
    again = mbx.qk_norm_rope_backward(q, k, *x, w, w, pos, fr, axes, interleaved, dq=q, dk=k)
    assert all(torch.equal(a, b) for a, b in zip(grads, again)) and torch.equal(q, grads[0])
    q.copy_(x[0]), k.copy_(x[1])
    mbx.qk_norm_rope(q, k, w, w, pos, fr, axes, interleaved, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(v, before)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dt,hd,axes", [(BF, 64, (32, 32)), (F32, 64, (32, 32)), (BF, 72, (36, 36)), (F32, 80, (8, 16, 16))])
def test_a_head_keeps_its_bits(mbx, dt, hd, axes, interleaved):
    """Wherever it lies, whatever other heads there are."""
    g = gen(31)
    q, do = rnd(g, (1, 50, 6, hd), dt), rnd(g, (1, 50, 6, hd), dt)
    w = rnd(g, (hd,), F32, 0.1, 1.0)
    pos, fr = torch.randint(0, 200, (50, len(axes)), generator=g).int().to(DEV), mbx.rope_axis_freqs(axes)
    fwd = lambda q, pos: mbx.qk_norm_rope(q, None, w, None, pos, fr, axes, interleaved)[0]
    bwd = lambda do, q, pos: mbx.qk_norm_rope_backward(do, None, q, None, w, None, pos, fr, axes, interleaved)
    want, wantg = fwd(q, pos), bwd(do, q, pos)
    for lead in (1, 8 // q.element_size(), 16 // q.element_size()):
        buf = torch.zeros(q.numel() + lead, dtype=dt, device=DEV)
        v = buf[lead:].view(q.shape)
        v.copy_(q)
        assert torch.equal(fwd(v, pos), want)
        assert all(torch.equal(a, b) for a, b in zip(bwd(do, v, pos)[::2], wantg[::2]))
    assert torch.equal(fwd(q[:, 3:9, 2:3], pos[3:9]), want[:, 3:9, 2:3])
    assert torch.equal(bwd(do[:, 3:9, 2:3], q[:, 3:9, 2:3], pos[3:9])[0], wantg[0][:, 3:9, 2:3])


@pytest.mark.parametrize("dt", [BF, F32])
def test_nothing_outside_the_heads_is_written(mbx, dt):
    g = gen(3)
    for hd, axes in ((64, (64,)), (100, (50,)), (127, (60,))):
        q, fr = rnd(g, (2, 9, 3, hd), dt), mbx.rope_axis_freqs(axes)
        pos = torch.randint(0, 20, (9, 1), generator=g).int().to(DEV)
        buf = torch.full((2, 9, 5, hd + 3), 7.0, dtype=dt, device=DEV)
        keep = torch.ones_like(buf, dtype=torch.bool)
        keep[:, :, 1:4, 2:2 + hd] = False
        mbx.qk_norm_rope(q, None, None, None, pos, fr, axes, q_out=buf[:, :, 1:4, 2:2 + hd])
        assert (buf[keep] == 7.0).all()
        mbx.qk_norm_rope_backward(q, None, q, None, None, None, pos, fr, axes, dq=buf[:, :, 1:4, 2:2 + hd])
        assert (buf[keep] == 7.0).all()


def test_non_finite_heads_stay_alone(mbx):
    g = gen(4)
    axes, fr = (16, 16), mbx.rope_axis_freqs((16, 16))
    for dt in (BF, F32):
        q, do = rnd(g, (1, 5, 4, 64), dt), rnd(g, (1, 5, 4, 64), dt)
        pos = torch.randint(0, 20, (5, 2), generator=g).int()
        clean, cleang = q.clone(), do.clone()
        q[0, 1, 2, 5], q[0, 3, 0, 40] = float("nan"), float("inf")
        do[0, 0, 1, 9] = float("nan")
        out, _ = mbx.qk_norm_rope(q, None, None, None, pos.to(DEV), fr, axes)
        dx = mbx.qk_norm_rope_backward(do, None, q, None, None, None, pos.to(DEV), fr, axes)[0]
        assert out[0, 1, 2].isnan().all() and out[0, 3, 0, 40].isnan()
        assert (out[0, 3, 0, 48:] == 0).all()  # elements that pass beside an infinite one
        assert dx[0, 1, 2].isnan().all() and dx[0, 0, 1].isnan().all()
        ok = torch.ones((1, 5, 4), dtype=torch.bool)
        ok[0, 1, 2] = ok[0, 3, 0] = False
        want, tol = hr.norm_rope(clean, None, pos, axes, fr, True, EPS)
        tr.assert_close(out[ok], want[ok], tol[ok])
        ok[0, 0, 1] = False
        (want, tol), _ = hr.norm_rope_backward(cleang, clean, None, pos, axes, fr, True, EPS)
        tr.assert_close(dx[ok], want[ok], tol[ok])


def test_broadcast_inputs(mbx):
    """A batch of stride 0, heads of stride 0 (one K head read as many), three-dimensional Q."""
    g = gen(23)
    axes, fr = (16, 24, 24), mbx.rope_axis_freqs((16, 24, 24))
    q = rnd(g, (1, 9, 1, 64), BF)
    pos = torch.randint(0, 50, (9, 3), generator=g).int().to(DEV)
    one, _ = mbx.qk_norm_rope(q, None, None, None, pos, fr, axes)
    wide = q.expand(4, -1, 5, -1)
    many, _ = mbx.qk_norm_rope(wide, None, None, None, pos[None].expand(4, -1, -1).contiguous(), fr, axes,
                               q_out=torch.empty((4, 9, 5, 64), dtype=BF, device=DEV))
    assert torch.equal(many, one.expand(4, -1, 5, -1))
    three, _ = mbx.qk_norm_rope(q[0], None, None, None, pos, fr, axes)
    assert three.shape == (9, 1, 64) and torch.equal(three, one[0])
    d1 = mbx.qk_norm_rope_backward(one, None, q, None, None, None, pos, fr, axes)[0]
    dm = mbx.qk_norm_rope_backward(one.expand(4, -1, 5, -1), None, wide, None, None, None, pos, fr, axes,
                                   dq=torch.empty((4, 9, 5, 64), dtype=BF, device=DEV))[0]
    assert torch.equal(dm, d1.expand(4, -1, 5, -1))


def test_it_is_the_norm_and_then_the_rotation(mbx):
    """float32: rope_axes of the normalised heads, within both roundings of the tolerance's scale."""
    g = gen(40)
    axes, fr = (16, 56, 56), mbx.rope_axis_freqs((16, 56, 56))
    q, k = case(g, 2, 65, 4, 2, 128, F32)
    w = rnd(g, (128,), F32, 0.1, 1.0)
    pos = torch.randint(0, 64, (65, 3), generator=g).int()
    got = mbx.qk_norm_rope(q, k, w, w, pos.to(DEV), fr, axes)
    norm = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * w
    two = mbx.rope_axes(norm(q), norm(k), pos.to(DEV), fr, axes)
    for a, b, t in zip(got, two, (q, k)):
        _, tol = hr.norm_rope(t, w, pos, axes, fr, True, EPS)
        assert ((tr.d(a) - tr.d(b)).abs() <= 2 * tol + 1e-30).all()


def test_streams_graphs_and_threads(mbx):
    """Forward and backward on a side stream, captured and replayed on new inputs, and two streams at once."""
    g = gen(77)
    axes, fr = (16, 24, 24), mbx.rope_axis_freqs((16, 24, 24))
    sets = []
    for _ in range(2):
        q, k = case(g, 2, 50, 6, 2, 64, BF)
        sets.append((q, k, rnd(g, q.shape, BF), rnd(g, k.shape, BF)))
    w = rnd(g, (64,), F32, 0.1, 1.0)
    pos = torch.randint(0, 64, (50, 3), generator=g).int().to(DEV)

    def step(q, k, dq, dk):
        return (*mbx.qk_norm_rope(q, k, w, w, pos, fr, axes),
                *mbx.qk_norm_rope_backward(dq, dk, q, k, w, w, pos, fr, axes))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for st, s in zip(streams, sets):
        with torch.cuda.stream(st):
            got.append([step(*s) for _ in range(8)][-1])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    static = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    for s, b in zip(sets, want):
        for t, v in zip(static, s):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, b))


def test_autograd_function(mbx):
    """The pair of calls inside a torch.autograd.Function, as the README shows it for LayerNorm."""
    g = gen(6)
    axes, fr = (32,), mbx.rope_axis_freqs((32,))
    pos = torch.arange(11, dtype=torch.int32, device=DEV)[:, None]

    class NormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, wq, wk):
            ctx.save_for_backward(q, k, wq, wk)
            return mbx.qk_norm_rope(q, k, wq, wk, pos, fr, axes)

        @staticmethod
        def backward(ctx, dq, dk):
            return mbx.qk_norm_rope_backward(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors, pos, fr, axes)

    leaves = [rnd(g, s, F32).requires_grad_() for s in ((2, 11, 4, 32), (2, 11, 2, 32), (32,), (32,))]
    qo, ko = NormRope.apply(*leaves)
    (qo.square().sum() + ko.mul(3).sum()).backward()
    q, k, wq, wk = (t.detach() for t in leaves)
    for x, w, do, gx, gw in ((q, wq, 2 * qo.detach(), leaves[0].grad, leaves[2].grad),
                             (k, wk, torch.full_like(k, 3.0), leaves[1].grad, leaves[3].grad)):
        (dx, tx), (dw, tw) = hr.norm_rope_backward(do, x, w, pos, axes, fr, True, EPS)
        tr.assert_close(gx, dx, tx)
        tr.assert_close(gw, dw, tw)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (3, 1), (4, 3), (5, 2), (32, 1)])
@pytest.mark.parametrize("hd,axes", [(32, (32,)), (64, (16, 24, 24)), (80, (40,)), (72, (24, 24, 24)), (128, (44, 42, 42))])
def test_few_heads(mbx, hd, axes, hq, hk, interleaved):
    """A warp takes several tokens where they have few heads; the last round's tokens are not whole; a batch's
    end inside a warp's tokens; K alone in the work of a block."""
    g = gen(hd + hq)
    fr = mbx.rope_axis_freqs(axes)
    w = rnd(g, (hd,), F32, 0.1, 1.0)
    for B, S in ((1, 2), (3, 7), (2, 1501), (1, 20011 if hd == 64 else 3)):
        q, k = case(g, B, S, hq, hk, hd, BF, "merged")
        dq, dk = rnd(g, q.shape, BF, 0.1), rnd(g, k.shape, BF, 0.1)
        pos = torch.randint(-50, 200, (B, S, len(axes)), generator=g).int()
        out = mbx.qk_norm_rope(q, k, w, w, pos.to(DEV), fr, axes, interleaved, EPS)
        got = mbx.qk_norm_rope_backward(dq, dk, q, k, w, w, pos.to(DEV), fr, axes, interleaved, EPS)
        for i, (do, x) in enumerate(((dq, q), (dk, k))):
            tr.assert_close(out[i], *hr.norm_rope(x, w, pos, axes, fr, interleaved, EPS), what=f"{i} {B, S}")
            (dx, tx), (dw, tw) = hr.norm_rope_backward(do, x, w, pos, axes, fr, interleaved, EPS)
            tr.assert_close(got[i], dx, tx, what=f"dx {i} {B, S}")
            tr.assert_close(got[2 + i], dw, tw, what=f"dw {i} {B, S}")


@pytest.mark.parametrize("interleaved", [True, False])
def test_angles(mbx, interleaved):
    """Far, fractional, tiny and negative positions; frequencies above a turn, negative, tiny and zero."""
    g = gen(50)
    n = 32
    fr = torch.cat([torch.tensor([1.0, -1.0, 0.0, 7.5, 50.0, 1e-9, 1e-300, -3.3e5, 2.0 ** 40, 1e-320], dtype=torch.float64),
                    torch.rand(n - 10, generator=g, dtype=torch.float64) * 4])
    whole = torch.tensor([0, 1, -1, 12345, 2 ** 31 - 1, -2 ** 31, 99, -7, 1 << 30, 1000003], dtype=torch.int32)
    part = torch.tensor([0.0, -0.0, 0.7109375, -1234.56, 1e-12, 1e-40, 3e7, -5.5, 1e9, 16777216.0], dtype=torch.float32)
    q = rnd(g, (1, 10, 2, 2 * n), F32)
    for pos in (whole[:, None], part[:, None]):
        out, _ = mbx.qk_norm_rope(q, None, None, None, pos.to(DEV), fr.to(DEV), (2 * n,), interleaved, EPS)
        want, tol = hr.norm_rope(q, None, pos, (2 * n,), fr, interleaved, EPS)
        # the reference's own angle: its product is rounded once, to 2^-53 of it
        ang = (tr.d(pos) * fr).abs()[None, :, None]
        slack = (ang * 2.0 ** -53).repeat_interleave(2, -1) if interleaved else torch.cat([ang, ang], -1) * 2.0 ** -53
        big = q.abs().amax().double().cpu() * 4
        keep = (slack < 1e-3).expand_as(want)
        err = (tr.d(out) - want).abs()
        assert (err <= tol * 2 + slack * big + 1e-30)[keep].all()
    for bad in (float("inf"), float("nan")):
        pos = torch.tensor([[0.0], [bad], [2.0]], device=DEV)
        o, _ = mbx.qk_norm_rope(q[:, :3], None, None, None, pos, fr.to(DEV), (2 * n,), interleaved, EPS)
        assert o[0, 1].isnan().all() and not o[0, [0, 2]].isnan().any()


def test_workspace_of_the_stated_size(mbx):
    """Nothing past it is written, what it held does not matter, and a smaller one is refused."""
    import ctypes
    g = gen(60)
    axes = (16, 24, 24)
    fr, ax = mbx.rope_axis_freqs(axes), (ctypes.c_int32 * 3)(16, 24, 24)
    L, st = mbx.lib(), torch.cuda.current_stream().cuda_stream
    for B, S, hq, hk in ((1, 1, 2, 1), (2, 77, 16, 4), (1, 9000, 1, 1), (1, 9000, 24, 24)):
        q, k = case(g, B, S, hq, hk, 64, BF)
        dq, dk, w = rnd(g, q.shape, BF, 0.1), rnd(g, k.shape, BF, 0.1), rnd(g, (64,), F32, 0.1, 1.0)
        pos = torch.randint(0, 64, (S, 3), generator=g).int().to(DEV)
        want = mbx.qk_norm_rope_backward(dq, dk, q, k, w, w, pos, fr, axes)
        need = mbx.qk_norm_grad_workspace(B, S, 64)
        out = [torch.empty_like(t) for t in want]
        for fill in (0xFF, 0x7F):
            ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
            call = lambda n: L.mbx_qk_norm_rope_backward(
                *map(mbx._heads, out[:2]), *map(mbx._view, out[2:]), *map(mbx._heads, (dq, dk, q, k)), mbx._view(w), mbx._view(w),
                mbx._view(pos), mbx._view(fr), ax, 3, 1, 1e-6, ws.data_ptr(), n, st)
            assert call(need) == 0
            assert all(torch.equal(a, b) for a, b in zip(out, want)) and (ws[need:] == fill).all()
            assert call(need - 16) == -10


def test_one_weight_gradient_alone(mbx):
    """A weight for Q or for K only; no K; a given dwq of which the rest is left alone."""
    g = gen(61)
    axes, fr = (32,), mbx.rope_axis_freqs((32,))
    q, k = case(g, 2, 21, 4, 2, 32, F32)
    dq, dk, w = rnd(g, q.shape, F32, 0.1), rnd(g, k.shape, F32, 0.1), rnd(g, (32,), F32, 0.1, 1.0)
    pos = torch.arange(21, dtype=torch.int32, device=DEV)[:, None]
    for wq, wk in ((w, None), (None, w)):
        got = mbx.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos, fr, axes)
        for i, (do, x, ww) in enumerate(((dq, q, wq), (dk, k, wk))):
            (dx, tx), (dw, tw) = hr.norm_rope_backward(do, x, ww, pos, axes, fr, True, EPS)
            tr.assert_close(got[i], dx, tx)
            if ww is None:
                assert got[2 + i] is None
            else:
                tr.assert_close(got[2 + i], dw, tw)
    buf = torch.full((40,), 7.0, device=DEV)
    a = mbx.qk_norm_rope_backward(dq, None, q, None, w, None, pos, fr, axes, dwq=buf[4:36])
    b = mbx.qk_norm_rope_backward(dq, None, q, None, w, None, pos, fr, axes)
    assert torch.equal(a[2], b[2]) and (buf[:4] == 7.0).all() and (buf[36:] == 7.0).all()
