"""Host-side tests of the products with NVFP4 weights: refusals (each before any
device is touched; the pointers are fake and never dereferenced), and the weight's
layout against the oracle's NVFP4 copy.
"""
import ctypes

import numpy as np
import pytest
import torch

from . import linear_ref as lr
from .test_train_host import BASE, BF16, F32, I32, WS, V, mbx, ref  # noqa: F401

E4M3, E2M1X2 = 3, 4
GS = BASE + 0x9000000


def test_refusals(mbx):  # noqa: F811
    L = mbx.lib()

    def st(o, x, w, f, gs=GS, b=None, silu=0, ws=WS, n=1 << 40):
        a = L.mbx_check_linear_nvfp4(ref(o), ref(x), ref(w), ref(f), gs, ref(b), silu, ws, n)
        assert a == L.mbx_linear_nvfp4(ref(o), ref(x), ref(w), ref(f), gs, ref(b), silu, ws, n, None)
        return a

    o, x, w, f, b = V(0, 2, 200), V(1, 2, 64), V(2, 200, 32, dtype=E2M1X2), V(3, 256, 4, dtype=E4M3), V(4, 1, 200)
    assert st(o, x, w, f) == st(o, x, w, f, b=b, silu=1) == st(o, x, w, f, b=V(4, 1, 200, dtype=F32)) == -9
    assert st(V(0, 2, 200, dtype=F32), x, w, f) == st(V(0, 2, 200, dtype=F32), V(1, 2, 64, dtype=F32), w, f, b=b) == -9
    assert st(o, V(1, 2, 64, 80), V(2, 200, 32, 48, dtype=E2M1X2), f) == -9       # padded rows
    assert st(None, x, w, f) == st(o, None, w, f) == st(o, x, None, f) == st(o, x, w, None) == st(o, x, w, f, gs=None) == -1
    assert st(o, x, V(2, 200, 32, dtype=E2M1X2, data=False), f) == st(o, x, w, f, b=V(4, 1, 200, data=False)) == -1
    assert st(o, V(1, 2, 64, dtype=F32), w, f) == st(o, V(1, 2, 64, dtype=I32), w, f) == -2
    assert st(o, x, V(2, 200, 32), f) == st(o, x, w, V(3, 256, 4)) == st(o, x, w, f, b=V(4, 1, 200, dtype=I32)) == -2
    assert st(V(0, 0, 200), V(1, 0, 64), w, f) == st(o, x, V(2, 0, 32, dtype=E2M1X2), f) == -3
    assert st(o, V(1, 2, 8208), V(2, 200, 4104, dtype=E2M1X2), V(3, 256, 516, dtype=E4M3)) == -4
    assert st(o, V(1, 2, 72), V(2, 200, 36, dtype=E2M1X2), f) == -5                # no whole blocks
    assert st(o, V(1, 2, 80), w, f) == st(V(0, 3, 200), x, w, f) == st(V(0, 2, 199), x, w, f) == -5
    assert st(o, x, w, V(3, 200, 4, dtype=E4M3)) == st(o, x, w, V(3, 256, 8, dtype=E4M3)) == st(o, x, w, f, b=V(4, 1, 100)) == -5
    assert st(o, x, V(2, 200, 32, 16, dtype=E2M1X2), f) == st(o, x, w, V(3, 256, 4, 8, dtype=E4M3)) == -6
    assert st(o, V(1, 2, 64, 32), w, f) == st(o, x, w, f, b=V(4, 1, 200, -1)) == -6
    assert st(V(0, 2, 200, off=1), x, w, f) == st(o, x, w, f, gs=GS + 2) == -7
    for bad in (V(1, 2, 200), V(2, 2, 200), V(3, 2, 200, off=512), V(4, 2, 200)):
        assert st(bad, x, w, f, b=b) == -8
    assert st(V(9, 2, 200), x, w, f) == -8
    assert st(o, V(1, 2, 64, 2 ** 62), w, f) == -10
    assert st(V(0, 257, 200), V(1, 257, 64), w, f) == st(o, x, w, f, silu=2) == -12
    big = 2 ** 24 + 1
    assert st(V(0, 1, big), V(1, 1, 64), V(20, big, 32, dtype=E2M1X2), V(60, 2 ** 24 + 128, 4, dtype=E4M3)) == -12


def test_workspace_arguments(mbx):  # noqa: F811
    n = ctypes.c_int64()
    st = lambda r, o, k: mbx.lib().mbx_linear_nvfp4_workspace(r, o, k, ctypes.byref(n))
    assert mbx.lib().mbx_linear_nvfp4_workspace(1, 1, 16, None) == -1
    assert st(0, 1, 16) == st(1, 0, 16) == st(1, 1, 0) == -3
    assert st(1, 1, 8208) == -4
    assert st(1, 1, 24) == -5
    assert st(257, 1, 16) == st(1, 2 ** 24 + 1, 16) == -12
    assert st(1, 1, 16) in (0, -9)  # -9: no device


def test_python_call_refuses_on_the_host(mbx):  # noqa: F811
    x, w4, sf, gs = torch.zeros(2, 64), torch.zeros(200, 32, dtype=torch.uint8), torch.zeros(256, 4, dtype=torch.uint8), torch.ones(1)

    def status(*a, **kw):
        with pytest.raises(mbx.MbxError) as e:
            mbx.linear_nvfp4(*a, **kw)
        return e.value.status

    assert status(x, w4, sf, gs) == status(x.bfloat16(), w4, sf.view(torch.float8_e4m3fn), gs, torch.zeros(200), True) == -9
    assert mbx.check_linear_nvfp4(torch.zeros(2, 200), x, w4, sf, gs) == -9
    assert status(x.half(), w4, sf, gs) == status(x, w4.int(), sf, gs) == status(x, w4, sf.int(), gs) == -2
    assert status(x, w4, sf, torch.ones(2)) == status(x, w4, sf, torch.ones(1).double()) == -12
    assert status(x[:, ::2], w4[:, :16], sf, gs) == status(x, w4.t(), sf, gs) == -6
    assert status(torch.zeros(()), w4, sf, gs) == -5
    with pytest.raises(TypeError):
        mbx.linear_nvfp4(x, None, sf, gs)


@pytest.mark.parametrize("N,K", [(1, 16), (130, 80), (256, 192)])
def test_weight_is_the_oracles_copy(mbx, orc, N, K):  # noqa: F811
    g = torch.Generator().manual_seed(N)
    w = (torch.randn((N, K), generator=g) * torch.exp(torch.randn((N, 1), generator=g) * 4)).bfloat16()
    w[0, :16] = 0.0
    w[-1, 5] = -0.0
    for gs in (None, torch.tensor([37.0])):
        w4, sf, s = mbx.nvfp4_weight(w, gs)
        assert gs is None or s is gs
        want4, wantsf = orc.quant_nvfp4(w.view(torch.int16).numpy().view(np.uint16), float(s), 0)
        assert np.array_equal(w4.numpy(), want4)
        assert np.array_equal(sf.numpy().reshape(-1), wantsf)
        assert tuple(sf.shape) == mbx.nvfp4_sf_shape(N, K) and w4.is_contiguous()
    err = (lr.weight(w4, sf) / float(s) - w.double()).abs()
    # a block's values are within half the widest step (4 to 6: 1) of a scale that is at most 1/16 off amax/6, or
    # 2^-10 below e4m3's smallest normal; a value above 6 scales loses 6 times what the scale is short of amax/6
    # (6 * 1/16 of it, less than the half step, or 6 * 2^-10)
    amax = w.double().abs().unflatten(1, (-1, 16)).amax(-1)
    lim = (amax * (17 / 16) / 6 + 6 * 2.0 ** -10 / float(s)).repeat_interleave(16, 1) + 1e-30
    big = (amax * float(s) / 6 <= 448).repeat_interleave(16, 1)
    assert (err <= lim)[big].all()
    with pytest.raises(mbx.MbxError):
        mbx.nvfp4_weight(torch.zeros(4, 24))


def test_zero_weight(mbx):  # noqa: F811
    w4, sf, s = mbx.nvfp4_weight(torch.zeros(3, 32))
    assert s.item() == 1.0 and not w4.any() and not sf.any()


@pytest.mark.parametrize("largest", [1e-30, 1e-33, 1e-37, 1e-44])
def test_weight_next_to_zero(mbx, largest):  # noqa: F811
    """The global scale and its quotient by the least block scale stay finite; zero blocks stay zero."""
    w = torch.randn((5, 48), generator=torch.Generator().manual_seed(1))
    w = (w / w.abs().max() * largest).float()
    w[2, 16:32] = 0.0
    w4, sf, s = mbx.nvfp4_weight(w)
    assert 0 < s.item() <= 2.0 ** 118
    got = lr.weight(w4, sf) / float(s)
    assert got.isfinite().all() and not got[2, 16:32].any()
    # as above: half the widest step of a scale at most 1/16 off, or 2^-10 below e4m3's smallest normal
    lim = w.double().abs().max() * (17 / 16) / 6 + 6 * 2.0 ** -10 / float(s)
    assert ((got - w.double()).abs() <= lim).all()


def test_weight_refusals(mbx):  # noqa: F811
    for shape, status in (((32,), -5), ((2, 4, 32), -5), ((0, 32), -3), ((4, 0), -3)):
        with pytest.raises(mbx.MbxError) as e:
            mbx.nvfp4_weight(torch.zeros(shape))
        assert e.value.status == status


def test_scales_are_no_weight(mbx):  # noqa: F811
    """An E4M3 tensor is refused as packed E2M1 pairs; as block scales it is taken (-9: no device)."""
    x, w4, sf, gs = torch.zeros(2, 64), torch.zeros(200, 32, dtype=torch.uint8), torch.zeros(256, 4, dtype=torch.uint8), torch.ones(1)
    e4 = torch.float8_e4m3fn
    for w, f, want in ((w4.view(e4), sf, -2), (w4.view(e4), sf.view(e4), -2), (w4, sf.view(e4), -9)):
        with pytest.raises(mbx.MbxError) as e:
            mbx.linear_nvfp4(x, w, f, gs)
        assert e.value.status == want == mbx.check_linear_nvfp4(torch.zeros(2, 200), x, w, f, gs)
