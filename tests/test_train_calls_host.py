"""Host-side properties of the Python calls and the build: nothing here reaches a device."""
import pytest
import torch


@pytest.fixture(scope="module")
def mbx():
    from modulation_bit_exact_gb300 import _build
    _build.build()
    import modulation_bit_exact_gb300 as m
    m.lib()
    return m


def refused(mbx, call):
    with pytest.raises(mbx.MbxError) as e:
        call()
    return e.value.status


def test_a_single_row_that_is_not_contiguous_is_refused(mbx):
    """One row has no row stride to be wrong, but its elements have to lie side by side: each operand,
    through the native calls and through ctypes."""
    bf, f64 = torch.bfloat16, torch.float64
    x, row, far = torch.zeros(4, 64), torch.zeros(64), torch.zeros(128)[::2]
    one, far1 = torch.zeros(1, 64), torch.zeros(1, 128)[:, ::2]
    rng = torch.zeros(2, dtype=torch.int64)
    assert mbx._rows_cols(far) == (1, 64, -1)
    for call in (lambda w, b: mbx.layer_norm(x, w, b), lambda w, b: mbx.layer_norm_backward(x, x, w, dbias=b)):
        assert refused(mbx, lambda: call(row, torch.zeros(64))) == -9      # only the device check refuses
        assert refused(mbx, lambda: call(far, row)) == refused(mbx, lambda: call(row, far)) == -6
    for call in (lambda t, o: mbx.layer_norm(t, out=o), lambda t, o: mbx.dropout(t, 0.5, rng, out=o),
                 lambda t, o: mbx.layer_norm_backward(t, one, dx=o), lambda t, o: mbx.layer_norm_backward(one, t, dx=o),
                 lambda t, o: mbx.ln_modulate_backward(one, one, t, dscale=o),
                 lambda t, o: mbx.dropout_gate_add(one, t, one, 0.5, rng, out=o),
                 lambda t, o: mbx.dropout_gate_add_backward(one, one, t, 0.5, rng, dgate=o)):
        assert refused(mbx, lambda: call(one, torch.zeros(1, 64))) == -9
        assert refused(mbx, lambda: call(far1, None)) == refused(mbx, lambda: call(one, torch.zeros(1, 128)[:, ::2])) == -6
    b = lambda t: t.to(bf) if t.is_contiguous() else torch.zeros(*t.shape[:-1], 128, dtype=bf)[..., ::2]
    for t, want in ((one, -9), (far1, -6)):
        assert refused(mbx, lambda: mbx.ln_modulate(b(t), b(one), b(one))) == want
        assert refused(mbx, lambda: mbx.ln_modulate(b(x), b(one), b(t))) == want
        assert refused(mbx, lambda: mbx.rmsnorm_scale(b(x), b(t), b(one))) == want
        assert refused(mbx, lambda: mbx.residual_gate_add(b(one), b(one), b(one), out=b(t))) == want
        assert mbx.check_layer_norm(torch.zeros_like(x), x, t) == want
    q, pos, fr = torch.zeros(1, 1, 2, 64), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(32, dtype=f64)
    assert refused(mbx, lambda: mbx.rope_axes(q, None, pos, fr, (32, 32))) == -9
    assert refused(mbx, lambda: mbx.rope_axes(q, None, torch.zeros(1, 4, dtype=torch.int32)[:, ::2], fr, (32, 32))) == -6
    assert refused(mbx, lambda: mbx.rope_axes(q, None, pos, torch.zeros(64, dtype=f64)[::2], (32, 32))) == -6
    fp8 = torch.zeros(1, 128, dtype=torch.uint8)[:, ::2]
    assert refused(mbx, lambda: mbx.ln_modulate_fp8(b(one), b(one), b(one), torch.ones(1), out_fp8=fp8)) == -6


def test_another_torch_rebuilds_the_binding(mbx, monkeypatch):
    """Also one that was installed in the place of the old one, under the same paths."""
    from modulation_bit_exact_gb300 import _build
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        raise RuntimeError("stop")

    monkeypatch.setattr(_build.subprocess, "run", run)
    _build.build()                                                         # everything is in place
    assert not ran
    for name, value in (("__version__", "0.0.1"), ("version.git_version", "0" * 40)):
        with monkeypatch.context() as m:
            m.setattr("torch." + name, value)
            with pytest.raises(RuntimeError, match="stop"):
                _build.build()
        assert ran and all(_build.BINDING_SRC in c for c in ran)
        ran.clear()


def test_gradient_of_a_bias_alone(mbx):
    """layer_norm takes a bias without a weight; so does its backward call."""
    from .test_train_host import F32, I32, V, WS, ref
    L = mbx.lib()

    def st(dx, dw, db, do, x, ws=WS, n=1 << 30):
        args = [ref(v) for v in (dx, dw, db, do, x, None, None)]
        a = L.mbx_check_layer_norm_backward(*args, 1e-6, ws, n)
        assert a == L.mbx_layer_norm_backward(*args, 1e-6, ws, n, None)
        return a

    dx, db, do, x = V(0), V(2, 1), V(3), V(4)
    assert st(dx, None, db, do, x) == st(dx, None, V(2, 1, dtype=F32), do, x) == -9  # host checks pass
    assert st(dx, V(1, 1), db, do, x) == st(dx, V(1, 1), None, do, x) == -1          # no weight to have a gradient
    assert st(dx, None, V(2, 1, dtype=I32), do, x) == -2
    assert st(V(0, dtype=F32), None, db, V(3, dtype=F32), V(4, dtype=F32)) == -2
    assert st(dx, None, V(2, 2), do, x) == st(dx, None, V(2, 1, 32), do, x) == -5
    assert st(dx, None, V(0, 1), do, x) == st(dx, None, V(4, 1), do, x) == -8
    args = [ref(v) for v in (dx, None, V(2, 4), do, x, None, None)]
    assert L.mbx_check_ln_modulate_backward(*args, 1e-6, WS, 1 << 30) == -1          # AdaLN has a scale
    t = torch.zeros(4, 64)
    assert refused(mbx, lambda: mbx.layer_norm_backward(t, t, dbias=torch.zeros(64))) == -9
