"""Host-side tests of the training path's entry points: refusals (each before
any device is touched; the pointers are fake and never dereferenced), and the
plain references that the GPU tests compare with.
"""
import ctypes

import numpy as np
import pytest
import torch

from . import train_ref as tr

BASE = 0x10000000
BF16, F32, I32, F64 = 1, 2, 5, 6


@pytest.fixture(scope="module")
def mbx():
    from modulation_bit_exact_gb300 import _build
    _build.build()
    import modulation_bit_exact_gb300 as m
    m.lib()
    return m


def V(slot, rows=4, cols=64, stride=None, dtype=BF16, off=0, data=True):
    from modulation_bit_exact_gb300 import _View
    return _View(BASE + slot * 0x1000000 + off if data else 0, rows, cols, cols if stride is None else stride, dtype)


def ref(v):
    return None if v is None else ctypes.byref(v)


WS = BASE + 0x40000000


def test_layer_norm_refusals(mbx):
    L = mbx.lib()

    def st(o, x, w=None, b=None, eps=1e-6):
        a = L.mbx_check_layer_norm(ref(o), ref(x), ref(w), ref(b), eps)
        assert a == L.mbx_layer_norm(ref(o), ref(x), ref(w), ref(b), eps, None)
        return a

    o, x, w, b = V(0), V(1), V(2, 1), V(3, 1)
    assert st(o, x, w, b) == st(o, x) == st(o, x, None, b) == -9        # host checks pass
    assert st(V(0, dtype=F32), V(1, dtype=F32), V(2, 1, dtype=F32), V(3, 1, dtype=F32)) == -9
    assert st(o, x, V(2, 1, dtype=F32), V(3, 1, dtype=F32)) == -9       # binary32 parameters
    assert st(o, x, V(2, 1, dtype=F32), b) == -2                        # of two dtypes
    assert st(V(0, dtype=F32), V(1, dtype=F32), w, b) == -2             # bf16 parameters of f32 rows
    assert st(V(0, dtype=F32), x) == -2
    assert st(o, V(1, dtype=I32)) == -2
    assert st(None, x) == st(o, None) == st(o, V(1, data=False)) == -1
    assert st(V(0, 0), V(1, 0)) == -3
    assert st(V(0, 4, 8200), V(1, 4, 8200)) == -4
    assert st(V(0, 5), x) == st(o, x, V(2, 2)) == st(o, x, V(2, 1, 32)) == -5
    assert st(o, V(1, stride=32)) == -6
    assert st(o, V(1, off=1)) == -7
    assert st(o, V(0)) == st(o, V(0, off=64)) == st(o, x, V(0, 1)) == -8  # no in-place LayerNorm
    assert st(V(0, 2 ** 61), V(1, 2 ** 61)) == -10
    assert st(V(0, 2 ** 32), V(1, 2 ** 32)) == -12
    for eps in (float("nan"), -1.0, float("inf")):
        assert st(o, x, eps=eps) == -12


@pytest.mark.parametrize("kind", ["layer_norm_backward", "ln_modulate_backward"])
def test_ln_backward_refusals(mbx, kind):
    L = mbx.lib()
    m = 1 if kind == "layer_norm_backward" else 2

    def st(dx, dw, db, do, x, w, r=None, eps=1e-6, ws=WS, n=1 << 30):
        args = [ref(v) for v in (dx, dw, db, do, x, w, r)]
        a = getattr(L, "mbx_check_" + kind)(*args, eps, ws, n)
        assert a == getattr(L, "mbx_" + kind)(*args, eps, ws, n, None)
        return a

    dx, dw, db, do, x, w, r = V(0), V(1, m), V(2, m), V(3), V(4), V(5, m), V(6)
    assert st(dx, dw, db, do, x, w) == st(dx, dw, db, do, x, w, r) == -9   # host checks pass
    assert st(dx, None, None, do, x, w) == st(dx, dw, None, do, x, w) == -9
    assert st(V(6), dw, db, do, x, w, r) == -9                             # in place on dresidual
    assert st(V(6, off=2), dw, db, do, x, w, r) == -8
    assert st(V(6, stride=128), dw, db, do, x, w, V(6)) == -8
    assert st(V(3), dw, db, do, x, w) == st(V(4), dw, db, do, x, w) == -8
    assert st(dx, V(2, m), db, do, x, w) == st(dx, V(5, m), db, do, x, w) == -8
    assert st(dx, V(0, m), db, do, x, w) == -8
    assert st(dx, dw, db, do, x, V(5, m, dtype=F32)) == -2                 # gradients of weight's dtype
    assert st(dx, V(1, m, dtype=F32), V(2, m, dtype=F32), do, x, V(5, m, dtype=F32)) == -9
    assert st(dx, dw, db, V(3, dtype=F32), x, w) == st(V(0, dtype=F32), dw, db, do, x, w) == -2
    assert st(dx, dw, db, do, x, w, V(6, dtype=F32)) == -2
    assert st(dx, V(1, 3), db, do, x, w) == st(dx, dw, db, do, x, V(5, 3)) == -5
    assert st(dx, dw, db, V(3, 5), x, w) == st(V(0, 4, 32), dw, db, do, x, w) == -5
    assert st(dx, dw, db, do, x, w, V(6, 3)) == -5
    assert st(dx, dw, db, do, x, None) == st(dx, dw, db, V(3, data=False), x, w) == -1
    assert st(dx, dw, db, do, x, w, eps=-1.0) == -12
    if kind == "layer_norm_backward":
        assert st(dx, None, None, do, x, None) == -9                       # no weight: dx alone
        assert st(dx, dw, db, do, x, V(5, 2)) == -5
    else:
        assert st(dx, None, None, do, x, None) == -1


def test_dropout_refusals(mbx):
    L = mbx.lib()
    RNG = BASE + 0x30000000

    def st(o, x, p=0.1, rng=RNG):
        a = L.mbx_check_dropout(ref(o), ref(x), p, rng, 0)
        assert a == L.mbx_dropout(ref(o), ref(x), p, rng, 0, None)
        return a

    o, x = V(0), V(1)
    assert st(o, x) == st(o, x, 0.0) == st(x, x) == -9
    assert st(o, x, 1.0) == st(o, x, -0.1) == st(o, x, float("nan")) == -12
    assert st(o, x, rng=None) == st(o, None) == -1
    assert st(o, x, rng=RNG + 4) == -7
    assert st(o, x, rng=BASE + 64) == -8                                   # out over the state
    assert st(V(1, off=2), x) == st(V(1, stride=128), x) == -8
    assert st(V(0, dtype=F32), x) == -2
    assert st(V(0, 2 ** 32), V(1, 2 ** 32)) == -12

    def st2(o, x, g, y, p=0.1, rng=RNG):
        a = L.mbx_check_dropout_gate_add(ref(o), ref(x), ref(g), ref(y), p, rng, 0)
        assert a == L.mbx_dropout_gate_add(ref(o), ref(x), ref(g), ref(y), p, rng, 0, None)
        return a

    g, y = V(2, 2), V(3)
    assert st2(o, x, g, y) == st2(x, x, g, y) == st2(o, x, V(2, 2, dtype=F32), y) == -9
    assert st2(y, x, g, y) == st2(V(2), x, g, y) == -8
    assert st2(o, x, V(2, 3), y) == st2(o, x, g, V(3, 4, 32)) == st2(o, V(1, 3), g, y) == -5
    assert st2(o, x, None, y) == st2(o, None, g, y) == st2(o, x, g, y, rng=None) == -1

    def st3(dy, dg, do, g, y, p=0.1, rng=RNG, ws=WS, n=1 << 30):
        args = [ref(v) for v in (dy, dg, do, g, y)]
        a = L.mbx_check_dropout_gate_add_backward(*args, p, rng, 0, ws, n)
        assert a == L.mbx_dropout_gate_add_backward(*args, p, rng, 0, ws, n, None)
        return a

    dy, dg, do = V(4), V(5, 2), V(6)
    assert st3(dy, dg, do, g, y) == st3(dy, None, do, g, y) == -9
    assert st3(dy, V(4, 2), do, g, y) == st3(do, dg, do, g, y) == st3(dy, V(2, 2), do, g, y) == -8
    assert st3(dy, V(5, 2, dtype=F32), do, g, y) == -2
    assert st3(dy, V(5, 1), do, g, y) == -5
    assert st3(dy, dg, do, g, y, rng=BASE + 0x5000000) == -8               # dgate over the state
    assert st3(dy, dg, do, g, y, p=1.0) == -12
    assert st3(dy, dg, do, None, y) == -1


def H(slot, B=2, S=3, h=4, hd=64, order="bshd", dtype=BF16, off=0, strides=None):
    from modulation_bit_exact_gb300 import _Heads
    st = strides or ((S * h * hd, h * hd, hd) if order == "bshd" else (h * S * hd, hd, S * hd))
    return _Heads(BASE + slot * 0x1000000 + off, B, S, h, hd, *st, dtype)


def test_rope_refusals(mbx):
    L = mbx.lib()

    def st(qo, ko, q, k, pos=None, fr=None, axes=(16, 24, 24), il=1, inv=0, n=None):
        pos = pos or V(8, 3, 3, dtype=I32)
        fr = fr or V(9, 1, sum(axes) // 2, dtype=F64)
        ax = (ctypes.c_int32 * len(axes))(*axes)
        args = [ref(qo), ref(ko), ref(q), ref(k), ref(pos), ref(fr), ax, len(axes) if n is None else n, il, inv]
        a = L.mbx_check_rope_axes(*args)
        assert a == L.mbx_rope_axes(*args, None)
        return a

    qo, ko, q, k = H(0), H(1, h=2), H(2), H(3, h=2)
    assert st(qo, ko, q, k) == st(qo, None, q, None) == -9
    assert st(q, k, q, k) == -9                                            # in place
    assert st(qo, ko, H(2, order="bhsd"), k) == -9
    assert st(qo, ko, q, k, pos=V(8, 6, 3, dtype=F32)) == -9               # a row for each token of the batch
    assert st(qo, ko, q, k, axes=(8, 8, 8)) == -9                          # a part of the head
    assert st(qo, None, q, k) == st(qo, ko, q, None) == st(None, ko, q, k) == -1
    assert st(qo, ko, q, k, pos=V(8, 3, 3, dtype=F64)) == st(qo, ko, q, k, fr=V(9, 1, 32, dtype=F32)) == -2
    assert st(H(0, dtype=F32), ko, q, k) == st(qo, ko, q, H(3, h=2, dtype=F32)) == -2
    assert st(H(0, S=0), H(1, S=0), H(2, S=0), H(3, S=0)) == -3
    assert st(H(0, hd=512), None, H(2, hd=512), None) == -4
    assert st(qo, ko, q, k, pos=V(8, 4, 3, dtype=I32)) == st(qo, ko, q, k, pos=V(8, 3, 2, dtype=I32)) == -5
    assert st(qo, ko, q, k, fr=V(9, 1, 31, dtype=F64)) == st(H(0, h=3), ko, q, k) == -5
    assert st(qo, H(1, h=2, S=4), q, H(3, h=2, S=4)) == -5
    assert st(H(0, strides=(0, 256, 64)), ko, q, k) == -6                  # an output over itself
    assert st(H(0, strides=(768, 255, 64)), ko, q, k) == -6
    assert st(qo, ko, H(2, strides=(768, 256, -64)), k) == -6
    assert st(H(0, off=1), ko, q, k) == -7
    assert st(qo, ko, q, k, pos=V(8, 3, 3, dtype=I32, off=2)) == -7
    assert st(H(2, off=128), ko, q, k) == st(qo, H(2, h=2), q, k) == st(qo, H(0, h=2), q, k) == -8
    assert st(qo, ko, q, k, pos=V(0, 3, 3, dtype=I32)) == -8
    assert st(qo, ko, H(2, strides=(2 ** 62, 256, 64)), k) == -10
    for axes in ((15, 24, 24), (0, 32, 32), (32, 32, 32), (16, 16, 16, 8, 8)):
        assert st(qo, ko, q, k, axes=axes) == -12
    assert st(qo, ko, q, k, n=0) == st(qo, ko, q, k, il=2) == st(qo, ko, q, k, inv=-1) == -12


def test_rope_in_place_inside_a_merged_buffer(mbx):
    """Q and K slices of one merged buffer, token-major or head-major, share an
    address range but no element; slices that do share one are refused."""
    L = mbx.lib()
    B, S, hd = 2, 3, 64
    ax = (ctypes.c_int32 * 1)(64)
    pos, fr = V(8, 3, 1, dtype=I32), V(9, 1, 32, dtype=F64)

    def st(q, k):
        return L.mbx_check_rope_axes(ref(q), ref(k), ref(q), ref(k), ref(pos), ref(fr), ax, 1, 1, 0)

    tok = (S * 8 * hd, 8 * hd, hd)                                         # [B, S, 4 + 2 + 2, hd]
    assert st(H(0, strides=tok), H(0, h=2, strides=tok, off=4 * hd * 2)) == -9
    assert st(H(0, strides=tok), H(0, h=2, strides=tok, off=3 * hd * 2)) == -8
    assert st(H(0, h=6, strides=tok, off=4 * hd * 2), H(0, h=4, strides=tok)) == -8  # wraps into the next token's
    hm = (3 * 4 * S * hd, hd, S * hd)                                      # [B, 3, 4, S, hd]
    assert st(H(0, strides=hm), H(0, strides=hm, off=4 * S * hd * 2)) == -9
    assert st(H(0, strides=hm), H(0, strides=hm, off=3 * S * hd * 2)) == -8
    hd3 = (S * 4 * 3 * hd, 4 * 3 * hd, 3 * hd)                             # [B, S, 4, 3, hd]
    assert st(H(0, strides=hd3), H(0, strides=hd3, off=hd * 2)) == -9
    assert st(H(0, strides=hd3), H(0, strides=hd3, off=hd * 2 - 2)) == -8
    assert st(H(0, strides=hd3, off=hd * 4), H(0, strides=hd3, off=hd * 6 - 2)) == -8  # wraps into the next head's
    odd = (S * (4 * 3 * hd + 8), 4 * 3 * hd + 8, 3 * hd)                   # tokens no whole heads apart
    assert st(H(0, strides=odd), H(0, strides=odd, off=hd * 2)) == -8
    one = (S * 8 * hd, 8 * hd, hd)
    assert st(H(0, B=1, strides=one), H(0, B=1, h=2, strides=one, off=4 * hd * 2)) == -9


def test_host_tensors_and_bad_states_are_refused(mbx):
    x = torch.randn(4, 64)
    rng = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: mbx.layer_norm(x), lambda: mbx.dropout(x, 0.5, rng),
                 lambda: mbx.layer_norm_backward(x, x), lambda: mbx.ln_modulate_backward(x, x, x[:1]),
                 lambda: mbx.dropout_gate_add(x, x[:1], x, 0.5, rng),
                 lambda: mbx.dropout_gate_add_backward(x, x[:1], x, 0.5, rng),
                 lambda: mbx.rope_axes(x.view(1, 4, 2, 32), None, torch.zeros(4, 1, dtype=torch.int32),
                                       mbx.rope_axis_freqs((32,), device="cpu"), (32,))):
        with pytest.raises(mbx.MbxError) as e:
            call()
        assert e.value.status == -9
    for bad in (torch.zeros(2), torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=torch.int64)[::2]):
        with pytest.raises(mbx.MbxError) as e:
            mbx.dropout(x, 0.5, bad)
        assert e.value.status == -12
    with pytest.raises(mbx.MbxError) as e:
        mbx.rope_axes(x, None, rng, rng, (2,))
    assert e.value.status == -5
    q = x.view(1, 4, 2, 32)
    fr = mbx.rope_axis_freqs((32,), device="cpu")
    pos = torch.zeros(4, 1, dtype=torch.int32)
    for axes in ((), (8,) * 5, (-2,), (2 ** 40,)):
        with pytest.raises(mbx.MbxError) as e:
            mbx.rope_axes(q, None, pos, fr, axes)
        assert e.value.status == -12
    with pytest.raises(mbx.MbxError) as e:
        mbx.rope_axes(q.transpose(2, 3), None, pos, fr, (32,))
    assert e.value.status == -6


def test_binding_follows_the_flat_row_rule(mbx):
    """The native binding's views are those of _rows_cols: what that gives a stride of -1 is refused."""
    buf = torch.zeros(6, 72)
    ok = (torch.zeros(2, 3, 8), buf[:, :64], torch.zeros(8), torch.zeros(2, 1, 8), torch.zeros(3, 4, 10)[:, :, :8],
          torch.zeros(4, 1, 6, 8)[:, :, ::2][:, :, :1])
    bad = (torch.zeros(4, 8).t(), torch.zeros(2, 5, 16)[:, :4, :], torch.zeros(3, 4, 8).transpose(0, 1))
    for t in ok:
        assert mbx._rows_cols(t)[2] >= 0
        with pytest.raises(mbx.MbxError) as e:
            mbx.layer_norm(t)
        assert e.value.status == -9                                        # only the device check refuses
    for t in bad:
        assert mbx._rows_cols(t)[2] == -1
        with pytest.raises(mbx.MbxError) as e:
            mbx.layer_norm(t)
        assert e.value.status == -6


def test_binding_arguments(mbx):
    x, rng = torch.zeros(4, 8), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: mbx.layer_norm(None), lambda: mbx.layer_norm(x, 3), lambda: mbx.layer_norm(x, eps="a"),
                 lambda: mbx.dropout(x, None, rng), lambda: mbx.dropout(x, 0.5, None),
                 lambda: mbx.ln_modulate_backward(x, x, None), lambda: mbx.rope_axes(x, None, x, x, 3),
                 lambda: mbx._native().layer_norm(x)):
        with pytest.raises((TypeError, mbx.MbxError)):
            call()
    with pytest.raises(OverflowError):
        mbx.dropout(x, 0.5, rng, offset=2 ** 63)
    with pytest.raises(mbx.MbxError) as e:
        mbx.layer_norm(torch.zeros(0, 8))
    assert e.value.status == -1                                            # no data, as everywhere


def test_workspace_query_refusals(mbx):
    n = ctypes.c_int64(-1)
    f = lambda *a: mbx.lib().mbx_param_grad_workspace(*a, ctypes.byref(n))
    assert f(8, 64, 8, BF16) == 0 and n.value == 0                         # per token: none
    assert f(8, 64, 3, BF16) == -5 and f(0, 64, 1, BF16) == -3 and f(8, 8193, 1, BF16) == -4
    assert f(8, 64, 1, I32) == -2 and f(2 ** 32, 64, 1, F32) == -12
    assert mbx.lib().mbx_param_grad_workspace(8, 64, 1, BF16, None) == -1


def test_philox_reference_known_answers():
    """The test vectors published with the generator (Salmon et al., SC 2011)."""
    z, f = 0, 0xFFFFFFFF
    for ctr, key, want in [
            ((z, z, z, z), (z, z), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((f, f, f, f), (f, f), (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))]:
        got = tr.philox(*[np.array([c]) for c in ctr], *key)
        assert tuple(int(g[0]) for g in got) == want


def test_references_match_differences():
    """The 64-bit gradient formulas against central differences of the 64-bit
    forward formulas (h = 1e-6 on unit-scale values: error about h^2 plus 2^-53/h)."""
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, f, do = n(6, 40), 1 + 0.1 * n(2, 40), n(6, 40)
    eps, h = 1e-6, 1e-6

    def loss(x, f, b):
        xh, _, _ = tr.ln_stats(x, eps)
        return ((xh.reshape(2, 3, 40) * f[:, None] + b[:, None]).reshape(6, 40) * do).sum()

    (dx, _), (df, _), (db, _) = tr.ln_backward(do, x, f, eps)
    b = n(2, 40)
    for grad, k in ((dx, 0), (df, 1), (db, 2)):
        args = [x, f, b]
        v = n(*args[k].shape)
        lo, hi = list(args), list(args)
        lo[k], hi[k] = args[k] - h * v, args[k] + h * v
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        assert abs(num - (grad * v).sum()) < 1e-7 * (grad * v).abs().sum()
