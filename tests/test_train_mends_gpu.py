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
