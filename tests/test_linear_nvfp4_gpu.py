"""Products with NVFP4 weights on the GPU against a plain 64-bit reference: rows
from one to the most, widths and outputs that end inside a tile, strides and
alignments, values far apart in one row, infinities, padding that is never used.
"""
import pytest
import torch

from . import linear_ref as lr
from . import train_ref as tr

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mbx():
    import modulation_bit_exact_gb300 as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, shape, dt, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dt).to(DEV)


def weight(mbx, g, N, K, pad=0x7F):
    """A weight in NVFP4 with `pad` in the scales' padding bytes."""
    w = torch.randn((N, K), generator=g) * 0.03 * (torch.rand((N, 1), generator=g) * 3)
    w4, sf, gs = mbx.nvfp4_weight(w.bfloat16())
    mask = torch.zeros_like(sf, dtype=torch.bool)
    n, b = torch.arange(N)[:, None], torch.arange(K // 16)[None]
    mask.view(-1)[((n // 128) * (sf.shape[1] // 4) + b // 4) * 512 + n % 32 * 16 + n % 128 // 32 * 4 + b % 4] = True
    sf[~mask] = pad
    return w4.to(DEV), sf.to(DEV), gs.to(DEV)


def check(mbx, x, w, bias, silu, **kw):
    got = mbx.linear_nvfp4(x, *w, bias, silu, **kw)
    tr.assert_close(got, *lr.linear(x.reshape(-1, x.shape[-1]), *w, bias, silu), what=f"{x.shape} {w[0].shape}")
    return got


# widths: one block, ends inside a step of 64 and a piece of 256, many pieces; K/2 no multiple of 16 bytes
WIDTHS = [16, 32, 64, 80, 96, 128, 224, 256, 288, 512, 1024, 1040, 1056, 2048, 5120, 8192]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K", WIDTHS)
def test_widths(mbx, K, dt):
    g = gen(K)
    for rows, N in ((1, 300), (2, 1), (3, 127), (5, 129), (16, 384)):
        w = weight(mbx, g, N, K)
        x = rnd(g, (rows, K), dt)
        check(mbx, x, w, rnd(g, (N,), dt, 0.1), True)
        check(mbx, x, w, None, False)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 100, 256])
def test_rows(mbx, rows, dt):
    g = gen(rows)
    for N, K in ((520, 1024), (77, 336)):
        w = weight(mbx, g, N, K)
        check(mbx, rnd(g, (rows, K), dt), w, rnd(g, (N,), F32, 0.1), rows % 2 == 0)


@pytest.mark.parametrize("N,K", [(24576, 512), (19457, 256), (40000, 64), (6144, 4096), (153 * 128, 1024), (10007, 1056)])
def test_many_outputs(mbx, N, K):
    """Every SM takes several tiles of outputs, and one over."""
    g = gen(N)
    w = weight(mbx, g, N, K)
    for rows in (1, 11):
        check(mbx, rnd(g, (rows, K), BF), w, rnd(g, (N,), BF, 0.1), True)


def test_types_of_outputs_and_bias(mbx):
    g = gen(1)
    w = weight(mbx, g, 200, 320)
    x = rnd(g, (3, 320), BF)
    for bias in (None, rnd(g, (200,), BF, 0.1), rnd(g, (200,), F32, 0.1)):
        check(mbx, x, w, bias, True)
        check(mbx, x, w, bias, True, out=torch.empty((3, 200), dtype=F32, device=DEV))
        check(mbx, x.float(), w, bias, True)
    shaped = mbx.linear_nvfp4(x.view(3, 1, 320), *w)
    assert shaped.shape == (3, 1, 200) and torch.equal(shaped.view(3, 200), mbx.linear_nvfp4(x, *w))
    one = mbx.linear_nvfp4(x[0], *w)
    assert one.shape == (200,)
    e4 = mbx.linear_nvfp4(x, w[0], w[1].view(torch.float8_e4m3fn), w[2])
    assert torch.equal(e4, shaped.view(3, 200))


@pytest.mark.parametrize("K", [512, 1040])
def test_strides_and_alignment(mbx, K):
    """Rows inside wider buffers; weight rows that start at 16, 8 and single bytes; nothing outside is written."""
    g = gen(2)
    N, rows = 260, 5
    w4, sf, gs = weight(mbx, g, N, K)
    x, bias = rnd(g, (rows, K), BF), rnd(g, (N,), F32, 0.1)
    want, tol = lr.linear(x, w4, sf, gs, bias, False)
    xb = torch.full((rows, K + 9), float("nan"), dtype=BF, device=DEV)
    xb[:, 3:3 + K] = x
    ob = torch.full((rows, N + 5), 7.0, dtype=BF, device=DEV)
    mbx.linear_nvfp4(xb[:, 3:3 + K], w4, sf, gs, bias, out=ob[:, 1:1 + N])
    tr.assert_close(ob[:, 1:1 + N], want, tol)
    assert (ob[:, 0] == 7.0).all() and (ob[:, 1 + N:] == 7.0).all()
    for pad, lead in ((16, 0), (32, 16), (8, 8), (3, 1)):
        wb = torch.full((N, K // 2 + pad), 0xFF, dtype=torch.uint8, device=DEV)
        v = wb[:, lead:lead + K // 2]
        v.copy_(w4)
        tr.assert_close(mbx.linear_nvfp4(x, v, sf, gs, bias), want, tol, what=f"{pad, lead}")
    bb = torch.zeros(N + 1, dtype=F32, device=DEV)
    bb[1:] = bias
    tr.assert_close(mbx.linear_nvfp4(x, w4, sf, gs, bb[1:]), want, tol)


@pytest.mark.parametrize("K", [1024, 1040])
@pytest.mark.parametrize("dt", [BF, F32])
def test_values_far_apart(mbx, K, dt):
    """A zero row; rows of 1e30 and of 1e-30; blocks 2^40 and single elements 2^12 larger than their neighbours."""
    g = gen(3)
    x = torch.randn((6, K), generator=g)
    x[1] = 0.0
    x[2] *= 1e30
    x[3] *= 1e-30
    x[4, 32:48] *= 2.0 ** 40
    x[5, ::37] *= 4096.0
    w = weight(mbx, g, 300, K)
    x = x.to(dt).to(DEV)
    check(mbx, x, w, None, False)
    check(mbx, x[[0, 1, 3, 4, 5]], w, None, True)
    assert (mbx.linear_nvfp4(x[1:2], *w) == 0).all()


@pytest.mark.parametrize("K", [1024, 1040])
@pytest.mark.parametrize("far", [2.0 ** 10, 2.0 ** 20, 2.0 ** 40])
def test_weights_that_are_zero_where_x_is_largest(mbx, K, far):
    """Such an output has the parts' stated precision: of its 16 values, and of the row."""
    g = gen(14)
    w4, sf, gs = weight(mbx, g, 140, K)
    x = torch.randn((3, K), generator=g)
    x[1:, 40] = far
    w4[:, 20] = 0  # elements 40 and 41
    x = x.bfloat16().to(DEV)
    got = check(mbx, x, (w4, sf, gs), None, False)
    assert got.isfinite().all() and torch.equal(got[1:2], mbx.linear_nvfp4(x[1:2], w4, sf, gs))
    # rows of the fallback have no parts: binary32 products at any distance
    out = mbx.linear_nvfp4(x.float(), torch.nn.functional.pad(w4, (1, 3))[:, 1:-3], sf, gs)
    wa = lr.weight(w4, sf)
    a = x.double().cpu()
    err = (out.double().cpu() - a @ wa.t() / float(gs)).abs()
    assert (err <= (48 + 4) * tr.U * (a.abs() @ wa.abs().t()) / float(gs)).all()


@pytest.mark.parametrize("K", [1024, 1040])
@pytest.mark.parametrize("silu", [False, True])
def test_infinities_and_nan_stay_in_their_row(mbx, K, silu):
    g = gen(4)
    w = weight(mbx, g, 300, K)
    x = rnd(g, (7, K), F32)
    clean = x.clone()
    x[1, 5], x[2, K - 1], x[3, 700], x[4, 3], x[4, 600], x[5, 9] = (
        float("inf"), float("-inf"), float("nan"), float("inf"), float("-inf"), 3e38)
    got = mbx.linear_nvfp4(x, *w, None, silu)
    want, tol = lr.linear(x[[0, 6]], *w, None, silu)
    tr.assert_close(got[[0, 6]], want, tol)
    assert torch.equal(got[[0, 6]], mbx.linear_nvfp4(clean, *w, None, silu)[[0, 6]])
    want, _ = lr.linear(x[[1, 2, 3, 4]], *w, None, silu)
    bad = got[[1, 2, 3, 4]].double().cpu()
    assert torch.equal(bad.isnan(), want.isnan())
    assert torch.equal(bad[~want.isnan()], want[~want.isnan()])  # infinities of the right sign


def test_a_scale_that_is_nan_stays_in_its_output(mbx):
    g = gen(5)
    for K in (256, 272):
        w4, sf, gs = weight(mbx, g, 140, K)
        x = rnd(g, (2, K), BF)
        clean = mbx.linear_nvfp4(x, w4, sf, gs)
        sf.view(-1)[(130 // 128 * (sf.shape[1] // 4) + 0) * 512 + 130 % 32 * 16 + 2] = 0x7F  # output 130, block 2
        got = mbx.linear_nvfp4(x, w4, sf, gs)
        assert got[:, 130].isnan().all()
        keep = [n for n in range(140) if n != 130]
        assert torch.equal(got[:, keep], clean[:, keep])


@pytest.mark.parametrize("K", [2048, 2064])
def test_every_code_and_scale(mbx, K):
    """All 16 codes against all 127 scales, one block of x alive at a time."""
    g = gen(6)
    blocks = K // 16
    w4 = torch.tensor([(2 * i % 16) | ((2 * i + 1) % 16) << 4 for i in range(8)], dtype=torch.uint8).repeat(blocks).repeat(130, 1)
    sf = torch.zeros((256, -(-blocks // 4) * 4), dtype=torch.uint8)
    n, b = torch.arange(130)[:, None], torch.arange(blocks)[None]
    at = ((n // 128) * (sf.shape[1] // 4) + b // 4) * 512 + n % 32 * 16 + n % 128 // 32 * 4 + b % 4
    sf.view(-1)[at] = ((n + b) % 127).to(torch.uint8)
    x = torch.zeros((16, K))
    for i in range(16):
        x[i, 16 * (i * 7 % blocks) + i] = 1.0  # element i of some block: code i alone
    gs = torch.ones(1, device=DEV)
    w = (w4.to(DEV), sf.to(DEV), gs)
    got = mbx.linear_nvfp4(x.to(DEV), *w)
    assert torch.equal(got.double().cpu(), lr.linear(x, *w, None, False)[0])  # one product: exact


def test_a_row_keeps_its_bits(mbx):
    """Alone, in a batch, at another place in it, in padded rows; and calls repeat bit for bit."""
    g = gen(7)
    for K in (1024, 1040):
        w = weight(mbx, g, 5000, K)
        x = rnd(g, (40, K), F32)
        all_ = mbx.linear_nvfp4(x, *w, None, True)
        assert torch.equal(all_, mbx.linear_nvfp4(x, *w, None, True))
        for lo, hi in ((0, 1), (3, 4), (17, 25), (39, 40)):
            assert torch.equal(mbx.linear_nvfp4(x[lo:hi], *w, None, True), all_[lo:hi])


def test_weights_of_a_producer(mbx):
    """The NVFP4 copy that ln_modulate_nvfp4 writes is a weight: out is its product with x."""
    g = gen(8)
    m, sc = rnd(g, (200, 512), BF), rnd(g, (1, 512), BF, 0.1)
    gs = torch.tensor([400.0], device=DEV)
    _, q4, sf = mbx.ln_modulate_nvfp4(m, sc, sc, gs)
    check(mbx, rnd(g, (2, 512), BF), (q4, sf, gs), None, False)


def test_streams_and_graphs(mbx):
    """Side streams at once, a captured call replayed with new x and scale, two graphs replayed in turn."""
    g = gen(9)
    w = weight(mbx, g, 4000, 2048)
    xs = [rnd(g, (2, 2048), BF) for _ in range(3)]
    want = [mbx.linear_nvfp4(x, *w, None, True) for x in xs]
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in xs]
    for st, x in zip(streams, xs):
        with torch.cuda.stream(st):
            outs.append([mbx.linear_nvfp4(x, *w, None, True) for _ in range(20)][-1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graphs, static = [], []
    for x in xs[:2]:
        t, gr = x.clone(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = mbx.linear_nvfp4(t, *w, None, True)
        graphs.append((gr, t, o))
    for i, j in ((0, 1), (2, 0), (1, 2)):
        graphs[0][1].copy_(xs[i]), graphs[1][1].copy_(xs[j])
        graphs[0][0].replay(), graphs[1][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][2], want[i]) and torch.equal(graphs[1][2], want[j])


def test_a_blocks_modulation_and_heads(mbx):
    """As they are used together: temb -> the modulation vectors -> LayerNorm + modulate -> the QKV product (the
    caller's) -> norm and rotation of Q and K, and back; eager and captured."""
    from . import heads_ref as hr
    g = gen(10)
    B, S, H, hd = 2, 24, 4, 64
    D = H * hd
    axes, fr = (16, 24, 24), mbx.rope_axis_freqs((16, 24, 24))
    w, bias = weight(mbx, g, 3 * D, D), rnd(g, (3 * D,), BF, 0.1)
    temb, x, wqkv = rnd(g, (B, D), BF), rnd(g, (B * S, D), BF), rnd(g, (D, 3 * D), BF, D ** -0.5)
    wq, wk = rnd(g, (hd,), BF, 0.05, 1.0), rnd(g, (hd,), BF, 0.05, 1.0)
    do = rnd(g, (2, B, S, H, hd), BF, 0.1)
    pos = torch.randint(0, 64, (S, 3), generator=g).int().to(DEV)

    def block():
        m = mbx.linear_nvfp4(temb, *w, bias, silu=True)
        shift, scale, gate = m.chunk(3, dim=-1)
        n = mbx.ln_modulate(x, scale, shift, 1e-6, "high")
        qkv = (n @ wqkv).view(B, S, 3 * H, hd)
        q, k = qkv[:, :, :H], qkv[:, :, H:2 * H]
        qo, ko = mbx.qk_norm_rope(q, k, wq, wk, pos, fr, axes)
        dq, dk, dwq, dwk = mbx.qk_norm_rope_backward(do[0], do[1], q, k, wq, wk, pos, fr, axes)
        out = mbx.residual_gate_add(x, gate, qo.reshape(B * S, D))
        return m, q.clone(), k.clone(), qo, ko, dq, dk, dwq, dwk, out

    got = block()
    m, q, k, qo, ko, dq, dk, dwq, dwk, _ = got
    tr.assert_close(m, *lr.linear(temb, *w, bias, True))
    for x_, w_, o, d_, dx, dw in ((q, wq, qo, do[0], dq, dwq), (k, wk, ko, do[1], dk, dwk)):
        tr.assert_close(o, *hr.norm_rope(x_, w_, pos, axes, fr, True, 1e-6))
        (a, ta), (b, tb) = hr.norm_rope_backward(d_, x_, w_, pos, axes, fr, True, 1e-6)
        tr.assert_close(dx, a, ta)
        tr.assert_close(dw, b, tb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = block()
    for _ in range(2):
        for t in again:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, got))


def test_weight_laid_out_on_the_gpu(mbx):
    w = torch.randn((300, 208), generator=gen(11)).bfloat16()
    for a, b in zip(mbx.nvfp4_weight(w), mbx.nvfp4_weight(w.to(DEV))):
        assert b.is_cuda and torch.equal(a, b.cpu())


@pytest.mark.parametrize("rows,N,K", [(1, 3000, 2048), (16, 3000, 2048), (19, 700, 8192), (16, 300, 512)])
def test_workspace_of_the_stated_size(mbx, rows, N, K):
    """Nothing past it is written, what it held does not matter, and a smaller one is refused."""
    g = gen(12)
    w4, sf, gs = weight(mbx, g, N, K)
    x = rnd(g, (rows, K), BF)
    out = torch.empty((rows, N), dtype=BF, device=DEV)
    need = mbx.linear_nvfp4_workspace(rows, N, K)
    want = mbx.linear_nvfp4(x, w4, sf, gs)
    L, st = mbx.lib(), torch.cuda.current_stream().cuda_stream
    for fill in (0xFF, 0x7F):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
        call = lambda n: L.mbx_linear_nvfp4(mbx._view(out), mbx._view(x), *mbx._weight_views(w4, sf), gs.data_ptr(), None, 0,
                                            ws.data_ptr(), n, st)
        assert call(need) == 0
        assert torch.equal(out, want) and (ws[need:] == fill).all()
        if need:
            assert call(need - 16) == -10


def test_zero_and_extreme_scales(mbx):
    """A global scale of 0 divides by it; blocks whose scale is 0 or the largest."""
    g = gen(13)
    w4, sf, gs = weight(mbx, g, 200, 256)
    x = rnd(g, (2, 256), F32)
    out = mbx.linear_nvfp4(x, w4, sf, torch.zeros(1, device=DEV))
    assert (out.isinf() | out.isnan()).all()
    for byte in (0x00, 0x01, 0x7E):
        f = torch.full_like(sf, byte)
        check(mbx, x, (w4, f, gs), None, False)
