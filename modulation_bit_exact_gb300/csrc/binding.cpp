// binding.cpp -- the training path's calls from Python without ctypes.
//
// A call on a few rows is bound by the host.  Marshalling its tensors through
// ctypes costs more than everything else: affine LayerNorm of [77, 1024] took
// 12.2 us a call on the GB300's host, of which 2.9 us ran on the GPU; through
// this module it takes 5.7 to 6.1 us (torch's negation of the same: 6.7 to 7.1).
//
// Each function takes its arguments by position (the defaults and the
// documentation are in __init__.py), turns the tensors into views of mbx.h
// under the flat-row rule, allocates the outputs that it is not given and the
// workspace, calls the C ABI on the current stream, and raises MbxError on a
// negative status.  No arithmetic, and no state but the error class.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "mbx.h"

namespace {

PyObject* g_error = nullptr;  // MbxError(status, message)

PyObject* raise_status(int status, const char* message) {
    PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", status, message) : nullptr;
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_SetString(PyExc_RuntimeError, message);
    }
    return nullptr;
}
PyObject* raise_status(int status) { return raise_status(status, mbx_status_string(status)); }

// An argument that is not a tensor: reported by the caller, which returns null.
struct BadArgument {};

const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
        throw BadArgument();
    }
    return THPVariable_Unpack(o);
}
at::Tensor tensor_or_none(PyObject* o) { return o == Py_None ? at::Tensor() : tensor(o); }

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw BadArgument();
    return v;
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw BadArgument();
    return v;
}

int dtype_code(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return MBX_BF16;
        case at::kFloat: return MBX_F32;
        case at::kInt: return MBX_I32;
        case at::kDouble: return MBX_F64;
        default: return 0;
    }
}

// A tensor as [rows, cols] (the rule of _rows_cols in __init__.py): the last
// dimension contiguous, the outer ones flat over the rows; a tensor that breaks
// it gets a negative row stride, which the library rejects.
template <class V>
V view(const at::Tensor& t) {
    V v{t.numel() ? t.data_ptr() : nullptr, 1, 1, 1, dtype_code(t)};
    const int64_t dims = t.dim();
    if (dims == 0) return v;
    const auto size = t.sizes();
    const auto stride = t.strides();
    v.cols = size[dims - 1];
    v.rows = v.cols ? t.numel() / v.cols : 0;
    v.row_stride = v.cols;
    if (v.cols > 1 && stride[dims - 1] != 1) {
        v.row_stride = -1;
        return v;
    }
    int64_t expect = -1;  // the stride that the next dimension out must have
    for (int64_t d = dims - 2; d >= 0; --d) {
        if (size[d] == 1) continue;
        if (expect < 0) v.row_stride = stride[d];
        else if (stride[d] != expect) {
            v.row_stride = -1;
            return v;
        }
        expect = stride[d] * size[d];
    }
    return v;
}

// An optional operand: its view, or a null pointer.
template <class V>
struct Opt {
    V v;
    bool has;
    explicit Opt(const at::Tensor& t) : v(t.defined() ? view<V>(t) : V{}), has(t.defined()) {}
    const V* ptr() const { return has ? &v : nullptr; }
};
using In = Opt<mbx_cview>;
using Out = Opt<mbx_view>;

void* stream_of(const at::Tensor& t) {
    // host tensors are refused by the library
    return t.is_cuda() ? c10::cuda::getCurrentCUDAStream(t.get_device()).stream() : nullptr;
}

// An uninitialised tensor of t's shape and dtype with flat rows.
at::Tensor like(const at::Tensor& t) {
    return t.is_contiguous() ? at::empty_like(t) : at::empty(t.sizes(), t.options());
}
void default_like(at::Tensor& out, const at::Tensor& t) {
    if (!out.defined()) out = like(t);
}

// The workspace of the gradient of `params` summed over x's rows (none where
// there are no params, and for a call that will be refused).
struct Workspace {
    at::Tensor t;
    int64_t bytes = 0;
    float* ptr = nullptr;
    Workspace(const at::Tensor& x, const at::Tensor& params) {
        if (!params.defined() || !x.is_cuda() || x.numel() == 0 || x.dim() == 0 || params.numel() == 0) return;
        const int64_t cols = x.size(-1);
        int64_t n = 0;
        if (mbx_param_grad_workspace(x.numel() / cols, cols, params.numel() / cols, dtype_code(x), &n) != MBX_OK) return;
        if (n == 0) return;
        t = at::empty({n / 4}, x.options().dtype(at::kFloat));
        bytes = n;
        ptr = static_cast<float*>(t.data_ptr());
    }
};

// The generator's state, or null when it is not a pair of int64.
const int64_t* rng_state(const at::Tensor& rng) {
    if (rng.scalar_type() != at::kLong || rng.numel() != 2 || !rng.is_contiguous()) return nullptr;
    return static_cast<const int64_t*>(rng.data_ptr());
}
constexpr const char* kBadRng = "MBX_E_ARG: rng must be a contiguous int64 tensor (seed, counter)";

PyObject* wrap(const at::Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
PyObject* wrap2(const at::Tensor& a, const at::Tensor& b) {
    PyObject* x = wrap(a);
    PyObject* y = x ? wrap(b) : nullptr;
    PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}
PyObject* wrap3(const at::Tensor& a, const at::Tensor& b, const at::Tensor& c) {
    PyObject* x = wrap(a);
    PyObject* y = x ? wrap(b) : nullptr;
    PyObject* z = y ? wrap(c) : nullptr;
    PyObject* r = z ? PyTuple_Pack(3, x, y, z) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return r;
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// The library call runs without the interpreter lock: a launch may wait for
// room in the stream's queue.
template <class F>
int call(F&& f) {
    int st;
    Py_BEGIN_ALLOW_THREADS st = f();
    Py_END_ALLOW_THREADS return st;
}

// Every entry: no C++ exception leaves it.
template <PyObject* (*F)(PyObject* const*)>
PyObject* guarded(PyObject* const* a) {
    HANDLE_TH_ERRORS
    try {
        return F(a);
    } catch (const BadArgument&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
template <Py_ssize_t N, PyObject* (*F)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return count_is(n, N) ? guarded<F>(a) : nullptr;
}

// ---------------------------------------------------------------- the calls

// x, weight, bias, eps, out
PyObject* layer_norm(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0]);
    const In w(tensor_or_none(a[1])), b(tensor_or_none(a[2]));
    const float eps = (float)number(a[3]);
    at::Tensor out = tensor_or_none(a[4]);
    default_like(out, x);
    const Out o(out);
    const In xv(x);
    void* s = stream_of(x);
    if (int st = call([&] { return mbx_layer_norm(o.ptr(), xv.ptr(), w.ptr(), b.ptr(), eps, s); })) return raise_status(st);
    return wrap(out);
}

// dout, x, factor, eps, dresidual, dx, dfactor, dshift
template <bool MODULATE>
PyObject* ln_backward(PyObject* const* a) {
    const at::Tensor &dout = tensor(a[0]), &x = tensor(a[1]);
    const at::Tensor factor = tensor_or_none(a[2]);
    const float eps = (float)number(a[3]);
    const In res(tensor_or_none(a[4]));
    at::Tensor dx = tensor_or_none(a[5]), df = tensor_or_none(a[6]), ds = tensor_or_none(a[7]);
    default_like(dx, x);
    if (factor.defined()) {
        default_like(df, factor);
        default_like(ds, factor);
    }
    const Workspace ws(x, ds);
    const Out o(dx), of(df), os(ds);
    const In d(dout), xv(x), f(factor);
    void* s = stream_of(x);
    auto* fn = MODULATE ? mbx_ln_modulate_backward : mbx_layer_norm_backward;
    if (int st = call([&] {
            return fn(o.ptr(), of.ptr(), os.ptr(), d.ptr(), xv.ptr(), f.ptr(), res.ptr(), eps, ws.ptr, ws.bytes, s);
        }))
        return raise_status(st);
    return wrap3(dx, df, ds);
}

// x, p, rng, offset, out
PyObject* dropout(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0]);
    const double p = number(a[1]);
    const int64_t* rng = rng_state(tensor(a[2]));
    const int64_t offset = integer(a[3]);
    if (!rng) return raise_status(MBX_E_ARG, kBadRng);
    at::Tensor out = tensor_or_none(a[4]);
    default_like(out, x);
    const Out o(out);
    const In xv(x);
    void* s = stream_of(x);
    if (int st = call([&] { return mbx_dropout(o.ptr(), xv.ptr(), p, rng, offset, s); })) return raise_status(st);
    return wrap(out);
}

// x, gate, y, p, rng, offset, out
PyObject* dropout_gate_add(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0]), &gate = tensor(a[1]), &y = tensor(a[2]);
    const double p = number(a[3]);
    const int64_t* rng = rng_state(tensor(a[4]));
    const int64_t offset = integer(a[5]);
    if (!rng) return raise_status(MBX_E_ARG, kBadRng);
    at::Tensor out = tensor_or_none(a[6]);
    default_like(out, x);
    const Out o(out);
    const In xv(x), g(gate), yv(y);
    void* s = stream_of(x);
    if (int st = call([&] { return mbx_dropout_gate_add(o.ptr(), xv.ptr(), g.ptr(), yv.ptr(), p, rng, offset, s); }))
        return raise_status(st);
    return wrap(out);
}

// dout, gate, y, p, rng, offset, dy, dgate
PyObject* dropout_gate_add_backward(PyObject* const* a) {
    const at::Tensor &dout = tensor(a[0]), &gate = tensor(a[1]), &y = tensor(a[2]);
    const double p = number(a[3]);
    const int64_t* rng = rng_state(tensor(a[4]));
    const int64_t offset = integer(a[5]);
    if (!rng) return raise_status(MBX_E_ARG, kBadRng);
    at::Tensor dy = tensor_or_none(a[6]), dgate = tensor_or_none(a[7]);
    default_like(dy, y);
    default_like(dgate, gate);
    const Workspace ws(y, gate);
    const Out o(dy), og(dgate);
    const In d(dout), g(gate), yv(y);
    void* s = stream_of(y);
    if (int st = call([&] {
            return mbx_dropout_gate_add_backward(o.ptr(), og.ptr(), d.ptr(), g.ptr(), yv.ptr(), p, rng, offset, ws.ptr,
                                                 ws.bytes, s);
        }))
        return raise_status(st);
    return wrap2(dy, dgate);
}

// A [batch, tokens, heads, head_dim] (or [tokens, heads, head_dim]) tensor;
// strides of any order, the last dimension contiguous.  0, or the status that
// its shape or strides call for.
template <class H>
int heads(H& h, const at::Tensor& t) {
    const int64_t n = t.dim();
    if (n != 3 && n != 4) return MBX_E_SHAPE;
    const auto z = t.sizes();
    const auto s = t.strides();
    if (z[n - 1] > 1 && s[n - 1] != 1) return MBX_E_STRIDE;
    h = H{t.numel() ? t.data_ptr() : nullptr, n == 4 ? z[0] : 1, z[n - 3], z[n - 2], z[n - 1],
          n == 4 ? s[0] : 0,                  s[n - 3],          s[n - 2], dtype_code(t)};
    return MBX_OK;
}

// q, k, positions, freqs, axes, interleaved, inverse, q_out, k_out
PyObject* rope_axes(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0]);
    const at::Tensor k = tensor_or_none(a[1]);
    const In pos(tensor(a[2])), freqs(tensor(a[3]));
    std::vector<int32_t> axes;
    PyObject* seq = PySequence_Fast(a[4], "axes: expected a sequence of integers");
    if (!seq) return nullptr;
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(seq); ++i) {
        const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
        if (v == -1 && PyErr_Occurred()) {
            Py_DECREF(seq);
            return nullptr;
        }
        axes.push_back(v < 0 || v > 1 << 20 ? 0 : (int32_t)v);  // out of range: refused
    }
    Py_DECREF(seq);
    if (axes.empty() || axes.size() > 4) return raise_status(MBX_E_ARG);
    const int interleaved = PyObject_IsTrue(a[5]), inverse = PyObject_IsTrue(a[6]);
    if (interleaved < 0 || inverse < 0) return nullptr;
    at::Tensor qo = tensor_or_none(a[7]), ko = tensor_or_none(a[8]);
    if (!qo.defined()) qo = at::empty_like(q);
    if (!ko.defined() && k.defined()) ko = at::empty_like(k);
    mbx_heads_cview qv, kv;
    mbx_heads_view qov, kov;
    int st = heads(qv, q);
    if (!st) st = heads(qov, qo);
    if (!st && k.defined()) st = heads(kv, k);
    if (!st && ko.defined()) st = heads(kov, ko);
    if (st) return raise_status(st);
    void* s = stream_of(q);
    st = call([&] {
        return mbx_rope_axes(&qov, ko.defined() ? &kov : nullptr, &qv, k.defined() ? &kv : nullptr, pos.ptr(),
                             freqs.ptr(), axes.data(), (int)axes.size(), interleaved, inverse, s);
    });
    if (st) return raise_status(st);
    return wrap2(qo, ko);
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

template <Py_ssize_t N, PyObject* (*F)(PyObject* const*)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(entry<N, F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<5, layer_norm>("layer_norm"),
    method<8, ln_backward<false>>("layer_norm_backward"),
    method<8, ln_backward<true>>("ln_modulate_backward"),
    method<5, dropout>("dropout"),
    method<7, dropout_gate_add>("dropout_gate_add"),
    method<8, dropout_gate_add_backward>("dropout_gate_add_backward"),
    method<9, rope_axes>("rope_axes"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
