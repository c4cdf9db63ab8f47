"""Host-side tests of the norm and rotation of Q and K heads: refusals (each before
any device is touched; the pointers are fake and never dereferenced), and the
plain reference against automatic differentiation.
"""
import ctypes

import pytest
import torch

from . import heads_ref as hr
from .test_train_host import BF16, F32, F64, I32, WS, H, V, mbx, ref  # noqa: F401


def W(slot, cols=64, rows=1, dtype=BF16, **kw):
    return V(slot, rows, cols, dtype=dtype, **kw)


def call_forward(L, qo, ko, q, k, wq=None, wk=None, pos=None, fr=None, axes=(16, 24, 24), il=1, eps=1e-6, n=None):
    pos, fr = pos or V(8, 3, 3, dtype=I32), fr or V(9, 1, sum(axes) // 2, dtype=F64)
    ax = (ctypes.c_int32 * len(axes))(*axes)
    args = [*map(ref, (qo, ko, q, k, wq, wk, pos, fr)), ax, len(axes) if n is None else n, il, eps]
    a = L.mbx_check_qk_norm_rope(*args)
    assert a == L.mbx_qk_norm_rope(*args, None)
    return a


def call_backward(L, dq, dk, dwq, dwk, dqo, dko, q, k, wq, wk, ws=WS, nbytes=1 << 40, axes=(16, 24, 24), eps=1e-6, il=1):
    pos, fr = V(8, 3, 3, dtype=I32), V(9, 1, sum(axes) // 2, dtype=F64)
    ax = (ctypes.c_int32 * len(axes))(*axes)
    args = [*map(ref, (dq, dk, dwq, dwk, dqo, dko, q, k, wq, wk, pos, fr)), ax, len(axes), il, eps, ws, nbytes]
    a = L.mbx_check_qk_norm_rope_backward(*args)
    assert a == L.mbx_qk_norm_rope_backward(*args, None)
    return a


def test_forward_refusals(mbx):  # noqa: F811
    L = mbx.lib()
    qo, ko, q, k = H(0), H(1, h=2), H(2), H(3, h=2)
    wq, wk = W(10), W(11)

    def st(*a, **kw):
        return call_forward(L, *a, **kw)

    assert st(qo, ko, q, k, wq, wk) == st(qo, None, q, None, wq) == st(qo, ko, q, k, None, wk) == -9
    assert st(q, k, q, k, wq, wk) == -9                                    # in place
    assert st(qo, ko, H(2, order="bhsd"), k) == st(qo, ko, q, k, axes=(8, 8, 8)) == -9
    assert st(qo, ko, q, k, W(10, dtype=F32), W(11, dtype=F32)) == -9      # binary32 weights of bf16 heads
    assert st(qo, ko, q, k, wq, wq) == -9                                  # one weight for both
    assert st(qo, None, q, k) == st(qo, ko, q, None) == st(None, ko, q, k) == -1
    assert st(qo, None, q, None, wq, wk) == st(qo, ko, q, k, W(10, data=False), wk) == -1  # a weight without heads
    f32 = [H(0, dtype=F32), None, H(2, dtype=F32), None]
    assert st(*f32, W(10, dtype=F32)) == -9
    assert st(*f32, wq) == st(qo, ko, q, k, wq, W(11, dtype=F32)) == -2
    assert st(qo, ko, q, H(3, h=2, dtype=F32)) == st(qo, ko, q, k, pos=V(8, 3, 3, dtype=F64)) == -2
    assert st(H(0, S=0), None, H(2, S=0), None) == -3
    assert st(H(0, hd=512), None, H(2, hd=512), None) == -4
    assert st(qo, ko, q, k, W(10, cols=32), wk) == st(qo, ko, q, k, W(10, rows=2), wk) == -5
    assert st(H(0, h=3), ko, q, k) == st(qo, ko, q, k, pos=V(8, 4, 3, dtype=I32)) == -5
    assert st(H(0, strides=(0, 256, 64)), ko, q, k) == st(qo, ko, H(2, strides=(768, 256, -64)), k) == -6
    assert st(H(0, off=1), ko, q, k) == st(qo, ko, q, k, W(10, off=1), wk) == -7
    assert st(H(2, off=128), ko, q, k) == st(qo, H(2, h=2), q, k) == st(qo, H(0, h=2), q, k) == -8
    assert st(qo, ko, q, k, W(0), wk) == st(qo, ko, q, k, wq, W(1, off=2)) == st(qo, ko, q, k, pos=V(0, 3, 3, dtype=I32)) == -8
    assert st(qo, ko, H(2, strides=(2 ** 62, 256, 64)), k) == -10
    assert st(qo, ko, q, k, eps=-1.0) == st(qo, ko, q, k, eps=float("nan")) == st(qo, ko, q, k, eps=float("inf")) == -12
    for axes in ((15, 24, 24), (0, 32, 32), (32, 32, 32), (16, 16, 16, 8, 8)):
        assert st(qo, ko, q, k, axes=axes) == -12
    assert st(qo, ko, q, k, n=0) == st(qo, ko, q, k, il=2) == -12


def test_backward_refusals(mbx):  # noqa: F811
    L = mbx.lib()
    dq, dk, do, dok, q, k = H(0), H(1, h=2), H(4), H(5, h=2), H(2), H(3, h=2)
    wq, wk, dwq, dwk = W(10), W(11), W(12), W(13)

    def st(*a, **kw):
        return call_backward(L, *a, **kw)

    full = (dq, dk, dwq, dwk, do, dok, q, k, wq, wk)
    put = lambda i, v: (*full[:i], v, *full[i + 1:])
    assert st(*full) == st(dq, None, dwq, None, do, None, q, None, wq, None) == -9
    assert st(*put(3, None)) == st(dq, dk, None, None, do, dok, q, k, None, None, ws=None, nbytes=0) == -9
    assert st(do, dok, dwq, dwk, do, dok, q, k, wq, wk) == -9             # in place on the incoming gradient
    assert st(q, dk, dwq, dwk, do, dok, q, k, wq, wk) == -8               # not on the heads
    assert st(*put(0, H(5))) == st(*put(0, H(1))) == st(*put(0, H(4, off=128))) == -8
    for i in (0, 1, 4, 5, 6, 7):
        assert st(*put(i, None)) == -1
    assert st(*put(8, None)) == -1                                         # a gradient without its weight
    assert st(*put(2, W(12, dtype=F32))) == st(*put(4, H(4, dtype=F32))) == st(*put(0, H(0, dtype=F32))) == -2
    assert st(*put(2, W(12, cols=32))) == st(*put(4, H(4, h=3))) == st(*put(5, H(5, h=2, S=4))) == -5
    assert st(*put(0, H(0, strides=(768, 255, 64)))) == -6
    for i, s in ((2, 10), (2, 13), (2, 2), (2, 4), (2, 0), (3, 11), (3, 8), (3, 9)):
        assert st(*put(i, W(s))) == -8
    assert st(*full, eps=-1.0) == st(*full, il=3) == st(*full, axes=(15, 24, 24)) == -12


def test_workspace_arguments(mbx):  # noqa: F811
    L = mbx.lib()
    n = ctypes.c_int64()
    st = lambda b, t, h: L.mbx_qk_norm_grad_workspace(b, t, h, ctypes.byref(n))
    assert L.mbx_qk_norm_grad_workspace(1, 1, 64, None) == -1
    assert st(0, 1, 64) == st(1, 0, 64) == st(1, 1, -1) == -3
    assert st(1, 1, 257) == -4
    assert st(2 ** 20, 2 ** 11, 64) == st(2 ** 62, 4, 64) == -12
    assert st(1, 1, 64) in (0, -9)  # -9: no device


def test_python_calls_refuse_on_the_host(mbx):  # noqa: F811
    q, fr = torch.randn(1, 4, 2, 32), mbx.rope_axis_freqs((32,), device="cpu")
    pos, w = torch.zeros(4, 1, dtype=torch.int32), torch.ones(32)

    def status(f):
        with pytest.raises(mbx.MbxError) as e:
            f()
        return e.value.status

    fwd = lambda q=q, k=None, wq=w, wk=None, axes=(32,), **kw: mbx.qk_norm_rope(q, k, wq, wk, pos, fr, axes, **kw)
    bwd = lambda dq=q, dk=None, q=q, k=None, wq=w, wk=None, axes=(32,), **kw: \
        mbx.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos, fr, axes, **kw)
    for f in (fwd, bwd):
        assert status(f) == -9
        for axes in ((), (8,) * 5, (-2,), (2 ** 40,)):
            assert status(lambda: f(axes=axes)) == -12
        assert status(lambda: f(q=q.transpose(2, 3))) == -6
        assert status(lambda: f(q=torch.randn(4, 32))) == -5
        assert status(lambda: f(wq=torch.ones(64)[::2])) == -6
        assert status(lambda: f(wk=w)) == -1
    assert status(lambda: fwd(k=q, wk=w)) == status(lambda: bwd(dk=q, k=q, wk=w)) == -9
    assert status(lambda: bwd(dk=q)) == status(lambda: bwd(k=q)) == -1
    assert mbx.check_qk_norm_rope(q, None, q, None, w, None, pos, fr, (32,)) == -9
    assert mbx.check_qk_norm_rope_backward(q, None, None, None, q, None, q, None, w, None, pos, fr, (32,)) == -8
    with pytest.raises(TypeError):
        mbx.qk_norm_rope(q, 3, w, None, pos, fr, (32,))


def test_the_reference_gradient_is_the_derivative():
    g = torch.Generator().manual_seed(1)
    axes, fr = (8, 12), torch.rand(10, generator=g, dtype=torch.float64)
    x = torch.randn(2, 5, 3, 24, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.rand(24, generator=g, dtype=torch.float64, requires_grad=True)
    r = torch.randn(2, 5, 3, 24, generator=g, dtype=torch.float64)
    pos = torch.rand(2, 5, 2, generator=g) * 9
    for il in (True, False):
        (dx, _), (dw, _) = hr.norm_rope_backward(r, x, w, pos, axes, fr, il, 0.1)
        n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 0.1) * w
        which = torch.tensor([0] * 4 + [1] * 6)
        ang = pos.double()[:, :, which] * fr
        c, s = torch.cos(ang)[:, :, None], torch.sin(ang)[:, :, None]
        a, b = (n[..., 0:20:2], n[..., 1:20:2]) if il else (n[..., :10], n[..., 10:20])
        t = torch.stack([a * c - b * s, a * s + b * c], dim=-1 if il else -2).flatten(-2)
        out = torch.cat([t, n[..., 20:]], dim=-1)
        gx, gw = torch.autograd.grad(out, (x, w), r)
        torch.testing.assert_close(out.detach(), hr.norm_rope(x, w, pos, axes, fr, il, 0.1)[0])
        torch.testing.assert_close(gx, dx)
        torch.testing.assert_close(gw, dw)
