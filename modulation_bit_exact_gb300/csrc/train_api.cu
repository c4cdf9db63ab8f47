// train_api.cu -- the C ABI of the training path: validation and dispatch of
// mbx_layer_norm and its gradients, mbx_ln_modulate_backward, the dropout
// entry points and mbx_rope_axes.  The order of the checks is that of
// mbx_api.cu: pure host checks first, then the device checks, then the launch.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "mbx.h"
#include "kernels/train.h"
#include "views.h"

namespace {

// Activations are bfloat16 or binary32, one type a call; parameters have the
// activations' type, or binary32 with bfloat16 activations.
bool act_dtype(int32_t d) { return d == MBX_BF16 || d == MBX_F32; }
bool param_dtype(int32_t p, int32_t act) { return p == act || p == MBX_F32; }

// A set of views with the checks of one call.  add() in the order in which the
// entry point names its operands.
struct Operands {
    V v[10];
    int n = 0;
    const V& add(const V& x) {
        v[n] = x;
        return v[n++];
    }
    int null_check() const {
        for (int i = 0; i < n; ++i)
            if (!v[i].data) return MBX_E_NULL;
        return MBX_OK;
    }
    int basic_checks() const {
        for (int i = 0; i < n; ++i) MBX_TRY(basic_any(v[i]));
        return MBX_OK;
    }
};

int check_same_shape(const V& a, const V& x) { return a.rows == x.rows && a.cols == x.cols ? MBX_OK : MBX_E_SHAPE; }

int check_eps(float eps) { return eps >= 0.0f && std::isfinite(eps) ? MBX_OK : MBX_E_ARG; }

bool vec_row(const V& v) { return aligned16(v); }

// The workspace of a call that needs `need` bytes of it, overlapping none of
// the n views.
int check_workspace(const float* ws, int64_t bytes, int64_t need, const V* views, int n) {
    if (!ws) return MBX_E_NULL;
    if (bytes < need) return MBX_E_BOUNDS;
    if (reinterpret_cast<uintptr_t>(ws) % 16) return MBX_E_ALIGN;
    const V w{ws, 1, need / 4, need / 4, MBX_F32};
    MBX_TRY(extent_ok(w));
    for (int i = 0; i < n; ++i)
        if (overlaps(w, views[i])) return MBX_E_ALIAS;
    return MBX_OK;
}

// Rows, columns and counts that the kernels' index arithmetic takes.
int check_extent(const V& x) {
    if (x.cols > kMaxHidden) return MBX_E_DIM_TOO_LARGE;
    if (x.rows >= (int64_t)1 << 32) return MBX_E_ARG;  // a row is one 32-bit word of the dropout counter
    return MBX_OK;
}

int64_t workspace_need(int64_t rows, int64_t mod_rows, int64_t cols, int32_t dtype) {
    if (rows == mod_rows) return 0;
    if (mbx::sm_count() < 1) return -1;
    return mbx::grad_workspace_bytes(rows, mod_rows, (int)cols, (int)esize(dtype));
}

// ---------------------------------------------------------------- LayerNorm

int check_layer_norm(const mbx_view* out, const mbx_cview* x, const mbx_cview* weight, const mbx_cview* bias,
                     float eps, bool dev) {
    if (!out || !x) return MBX_E_NULL;
    Operands o;
    const V ov = o.add(of(out)), xv = o.add(of(x));
    if (weight) o.add(of(weight));
    if (bias) o.add(of(bias));
    MBX_TRY(o.null_check());
    if (!act_dtype(xv.dtype) || ov.dtype != xv.dtype) return MBX_E_DTYPE;
    for (int i = 2; i < o.n; ++i)
        if (!param_dtype(o.v[i].dtype, xv.dtype) || o.v[i].dtype != o.v[2].dtype) return MBX_E_DTYPE;
    MBX_TRY(o.basic_checks());
    MBX_TRY(check_extent(xv));
    MBX_TRY(check_same_shape(ov, xv));
    for (int i = 2; i < o.n; ++i) MBX_TRY(check_weight(o.v[i], xv));
    MBX_TRY(check_eps(eps));
    for (int i = 1; i < o.n; ++i)
        if (overlaps(ov, o.v[i])) return MBX_E_ALIAS;
    return dev ? views_on_device(o.v, o.n) : MBX_OK;
}

// dx, then the operands it is computed from, then the two parameter gradients
// (either may be null).  `factor` has mod_rows rows (LayerNorm: one, or none, where
// dshift, the gradient of a bias alone, has a type of its own).
int check_ln_backward(const mbx_view* dx, const mbx_view* dfactor, const mbx_view* dshift, const mbx_cview* dout,
                      const mbx_cview* x, const mbx_cview* factor, const mbx_cview* dres, bool one_row, float eps,
                      const float* ws, int64_t ws_bytes, bool dev) {
    if (!dx || !dout || !x) return MBX_E_NULL;
    if (!factor && (!one_row || dfactor)) return MBX_E_NULL;
    Operands o;
    const V dxv = o.add(of(dx)), dov = o.add(of(dout)), xv = o.add(of(x));
    const int i_f = factor ? o.n : -1;
    if (factor) o.add(of(factor));
    const int i_r = dres ? o.n : -1;
    if (dres) o.add(of(dres));
    const int i_out = o.n;
    if (dfactor) o.add(of(dfactor));
    if (dshift) o.add(of(dshift));
    MBX_TRY(o.null_check());
    if (!act_dtype(xv.dtype) || dov.dtype != xv.dtype || dxv.dtype != xv.dtype) return MBX_E_DTYPE;
    if (dres && o.v[i_r].dtype != xv.dtype) return MBX_E_DTYPE;
    if (factor && !param_dtype(o.v[i_f].dtype, xv.dtype)) return MBX_E_DTYPE;
    for (int i = i_out; i < o.n; ++i)
        if (factor ? o.v[i].dtype != o.v[i_f].dtype : !param_dtype(o.v[i].dtype, xv.dtype)) return MBX_E_DTYPE;
    MBX_TRY(o.basic_checks());
    MBX_TRY(check_extent(xv));
    MBX_TRY(check_same_shape(dxv, xv));
    MBX_TRY(check_same_shape(dov, xv));
    if (dres) MBX_TRY(check_same_shape(o.v[i_r], xv));
    if (factor) MBX_TRY(one_row ? check_weight(o.v[i_f], xv) : check_mod(o.v[i_f], xv));
    for (int i = i_out; i < o.n; ++i)
        MBX_TRY(factor ? check_same_shape(o.v[i], o.v[i_f]) : check_weight(o.v[i], xv));
    MBX_TRY(check_eps(eps));
    // dx may be exactly the residual stream's gradient; nothing else overlaps an output
    for (int i = 1; i < o.n; ++i)
        if (overlaps(dxv, o.v[i]) && !(i == i_r && same_view(dxv, o.v[i]))) return MBX_E_ALIAS;
    for (int k = i_out; k < o.n; ++k)
        for (int i = 1; i < o.n; ++i)
            if (i != k && overlaps(o.v[k], o.v[i])) return MBX_E_ALIAS;
    if (dfactor || dshift) {
        const int64_t m = factor ? o.v[i_f].rows : 1;
        // without a device the size is unknown: the device check refuses the call
        const int64_t need = workspace_need(xv.rows, m, xv.cols, xv.dtype);
        if (need > 0) {
            MBX_TRY(check_workspace(ws, ws_bytes, need, o.v, o.n));
            o.add(V{ws, 1, need / 4, need / 4, MBX_F32});
        }
    }
    return dev ? views_on_device(o.v, o.n) : MBX_OK;
}

int ln_backward(const mbx_view* dx, const mbx_view* dfactor, const mbx_view* dshift, const mbx_cview* dout,
                const mbx_cview* x, const mbx_cview* factor, const mbx_cview* dres, float factor_add, float eps,
                float* ws, void* stream) {
    mbx::LnBwdParams p = {};
    p.dx = dx->data;
    p.dx_stride = dx->row_stride;
    p.dout = dout->data;
    p.dout_stride = dout->row_stride;
    p.x = x->data;
    p.x_stride = x->row_stride;
    p.rows = x->rows;
    p.D = (int)x->cols;
    p.eps = eps;
    p.factor_add = factor_add;
    p.neg_zero = -0.0f;
    p.mod_rows = 1;
    const int ce = x->dtype == MBX_F32 ? 4 : 8;
    bool vec = p.D % ce == 0 && vec_row(of(dx)) && vec_row(of(dout)) && vec_row(of(x));
    if (factor) {
        p.factor = factor->data;
        p.factor_stride = factor->row_stride;
        p.p_f32 = factor->dtype == MBX_F32;
        p.mod_rows = factor->rows;
        vec = vec && vec_row(of(factor));
    }
    if (dfactor) {
        p.dfactor = dfactor->data;
        p.dfactor_stride = dfactor->row_stride;
        vec = vec && vec_row(of(dfactor));
    }
    if (dshift) {
        p.dshift = dshift->data;
        p.dshift_stride = dshift->row_stride;
        p.p_f32 = dshift->dtype == MBX_F32;
        vec = vec && vec_row(of(dshift));
    }
    if (dres) {
        p.dres = dres->data;
        p.dres_stride = dres->row_stride;
        vec = vec && vec_row(of(dres));
    }
    p.seq = p.rows / p.mod_rows;
    p.ws = ws;
    return cuda_status(mbx::launch_ln_backward(p, x->dtype == MBX_F32, vec, (cudaStream_t)stream));
}

// ---------------------------------------------------------------- dropout

// p, and the generator's state as a view (16 bytes).
int check_dropout_args(double p, const int64_t* rng, V* state) {
    if (!(p >= 0.0 && p < 1.0)) return MBX_E_ARG;
    if (!rng) return MBX_E_NULL;
    if (reinterpret_cast<uintptr_t>(rng) % 8) return MBX_E_ALIGN;
    *state = V{rng, 1, 4, 4, MBX_F32};
    return extent_ok(*state);
}

// x null: plain dropout of y.
int check_dropout(const mbx_view* out, const mbx_cview* x, const mbx_cview* gate, const mbx_cview* y, bool gated,
                  double prob, const int64_t* rng, bool dev) {
    if (!out || !y || (gated && (!x || !gate))) return MBX_E_NULL;
    Operands o;
    const V ov = o.add(of(out)), yv = o.add(of(y));
    if (gated) {
        o.add(of(x));
        o.add(of(gate));
    }
    MBX_TRY(o.null_check());
    if (!act_dtype(yv.dtype) || ov.dtype != yv.dtype) return MBX_E_DTYPE;
    if (gated && (o.v[2].dtype != yv.dtype || !param_dtype(o.v[3].dtype, yv.dtype))) return MBX_E_DTYPE;
    MBX_TRY(o.basic_checks());
    MBX_TRY(check_extent(yv));
    MBX_TRY(check_same_shape(ov, yv));
    if (gated) {
        MBX_TRY(check_same_shape(o.v[2], yv));
        MBX_TRY(check_mod(o.v[3], yv));
    }
    // out may be exactly the residual (plain dropout: exactly the input)
    const int in_place = gated ? 2 : 1;
    for (int i = 1; i < o.n; ++i)
        if (overlaps(ov, o.v[i]) && !(i == in_place && same_view(ov, o.v[i]))) return MBX_E_ALIAS;
    V state;
    MBX_TRY(check_dropout_args(prob, rng, &state));
    if (overlaps(ov, state)) return MBX_E_ALIAS;
    o.add(state);
    return dev ? views_on_device(o.v, o.n) : MBX_OK;
}

int check_dropout_backward(const mbx_view* dy, const mbx_view* dgate, const mbx_cview* dout, const mbx_cview* gate,
                           const mbx_cview* y, double prob, const int64_t* rng, const float* ws, int64_t ws_bytes,
                           bool dev) {
    if (!dy || !dout || !gate || !y) return MBX_E_NULL;
    Operands o;
    const V dyv = o.add(of(dy)), dov = o.add(of(dout)), g = o.add(of(gate)), yv = o.add(of(y));
    if (dgate) o.add(of(dgate));
    MBX_TRY(o.null_check());
    if (!act_dtype(yv.dtype) || dyv.dtype != yv.dtype || dov.dtype != yv.dtype) return MBX_E_DTYPE;
    if (!param_dtype(g.dtype, yv.dtype) || (dgate && o.v[4].dtype != g.dtype)) return MBX_E_DTYPE;
    MBX_TRY(o.basic_checks());
    MBX_TRY(check_extent(yv));
    MBX_TRY(check_same_shape(dyv, yv));
    MBX_TRY(check_same_shape(dov, yv));
    MBX_TRY(check_mod(g, yv));
    if (dgate) MBX_TRY(check_same_shape(o.v[4], g));
    V state;
    MBX_TRY(check_dropout_args(prob, rng, &state));
    o.add(state);
    for (int i = 1; i < o.n; ++i) {
        if (overlaps(dyv, o.v[i])) return MBX_E_ALIAS;
        if (dgate && i != 4 && overlaps(o.v[4], o.v[i])) return MBX_E_ALIAS;
    }
    if (dgate) {
        const int64_t need = workspace_need(yv.rows, g.rows, yv.cols, yv.dtype);
        if (need > 0) {
            MBX_TRY(check_workspace(ws, ws_bytes, need, o.v, o.n));
            o.add(V{ws, 1, need / 4, need / 4, MBX_F32});
        }
    }
    return dev ? views_on_device(o.v, o.n) : MBX_OK;
}

mbx::DropParams drop_params(const mbx_view* out, const mbx_cview* x, const mbx_cview* gate, const mbx_cview* y,
                            double prob, const int64_t* rng, int64_t offset, bool* vec) {
    mbx::DropParams p = {};
    p.out = out->data;
    p.out_stride = out->row_stride;
    const int ce = out->dtype == MBX_F32 ? 4 : 8;
    *vec = out->cols % ce == 0 && vec_row(of(out)) && vec_row(of(x));
    p.x = x->data;
    p.x_stride = x->row_stride;
    p.rows = out->rows;
    p.D = (int)out->cols;
    p.mod_rows = 1;
    if (gate) {
        p.y = y->data;
        p.y_stride = y->row_stride;
        p.gate = gate->data;
        p.gate_stride = gate->row_stride;
        p.p_f32 = gate->dtype == MBX_F32;
        p.mod_rows = gate->rows;
        *vec = *vec && vec_row(of(y)) && vec_row(of(gate));
    }
    p.seq = p.rows / p.mod_rows;
    p.rng = rng;
    p.offset = offset;
    p.threshold = (uint32_t)(prob * 4294967296.0);  // p < 1: below 2^32
    p.inv_keep = (float)(1.0 / (1.0 - prob));
    return p;
}

// ---------------------------------------------------------------- rotary positions

// A heads view in one form.  Strides of dimensions of size 1 address nothing
// and are taken as 0.
struct H4 {
    const void* data;
    int64_t b, t, h, hd, sb, st, sh;
    int32_t dtype;
    int64_t es() const { return esize(dtype); }
    int64_t head_span() const { return (h - 1) * sh + hd; }
    int64_t token_span() const { return (t - 1) * st + head_span(); }
    int64_t span() const { return (b - 1) * sb + token_span(); }
};

template <class W>
H4 of4(const W* w) {
    return H4{w->data,
              w->batch,
              w->tokens,
              w->heads,
              w->head_dim,
              w->batch > 1 ? w->batch_stride : 0,
              w->tokens > 1 ? w->token_stride : 0,
              w->heads > 1 ? w->head_stride : 0,
              w->dtype};
}

int basic4(const H4& v) {
    if (!v.data) return MBX_E_NULL;
    if (!act_dtype(v.dtype)) return MBX_E_DTYPE;
    if (v.b <= 0 || v.t <= 0 || v.h <= 0 || v.hd <= 0) return MBX_E_EMPTY;
    if (v.hd > 256) return MBX_E_DIM_TOO_LARGE;
    if (v.h > (int64_t)1 << 20 || v.b > (int64_t)1 << 40 || v.t > (int64_t)1 << 40) return MBX_E_ARG;
    if (v.sb < 0 || v.st < 0 || v.sh < 0) return MBX_E_STRIDE;
    if (reinterpret_cast<uintptr_t>(v.data) % v.es()) return MBX_E_ALIGN;
    int64_t a = 0, bb = 0, c = 0, n = 0, bytes = 0;
    uintptr_t end = 0;
    if (__builtin_mul_overflow(v.b - 1, v.sb, &a) || __builtin_mul_overflow(v.t - 1, v.st, &bb) ||
        __builtin_mul_overflow(v.h - 1, v.sh, &c) || __builtin_add_overflow(a, bb, &n) ||
        __builtin_add_overflow(n, c, &n) || __builtin_add_overflow(n, v.hd, &n) ||
        __builtin_mul_overflow(n, v.es(), &bytes) ||
        __builtin_add_overflow(reinterpret_cast<uintptr_t>(v.data), (uintptr_t)bytes, &end))
        return MBX_E_BOUNDS;
    return MBX_OK;
}

// No two elements of an output share an address: sorted by stride, each
// dimension's stride covers the span of those below it.
int injective4(const H4& v) {
    int64_t n[3] = {v.h, v.t, v.b}, s[3] = {v.sh, v.st, v.sb};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                const int64_t a = n[i], c = s[i];
                n[i] = n[j];
                s[i] = s[j];
                n[j] = a;
                s[j] = c;
            }
    int64_t span = v.hd;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < span) return MBX_E_STRIDE;
        span += (n[i] - 1) * s[i];
    }
    return MBX_OK;
}

bool same4(const H4& a, const H4& b) {
    return a.data == b.data && a.b == b.b && a.t == b.t && a.h == b.h && a.hd == b.hd && a.sb == b.sb &&
           a.st == b.st && a.sh == b.sh;
}

// Whether two views share no element: their address ranges are apart, or they
// repeat with one period (the batch's, the token's or the head's stride) and lie
// in disjoint parts of it, as Q and K inside a merged QKV buffer do.
bool disjoint4(const H4& a, const H4& b) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.data), b0 = reinterpret_cast<uintptr_t>(b.data);
    if (a0 + a.span() * a.es() <= b0 || b0 + b.span() * b.es() <= a0) return true;
    if (a.dtype != b.dtype || (b0 > a0 ? b0 - a0 : a0 - b0) % a.es()) return false;
    const bool a_first = a0 <= b0;
    const H4 &lo = a_first ? a : b, &hi = a_first ? b : a;
    const int64_t delta = (int64_t)((a_first ? b0 - a0 : a0 - b0) / a.es());
    auto apart = [&](int64_t period, int64_t span_lo, int64_t span_hi) {
        return period > 0 && delta >= span_lo && delta + span_hi <= period;
    };
    if (a.b > 1 && b.b > 1 && a.sb == b.sb && apart(a.sb, lo.token_span(), hi.token_span())) return true;
    // a dimension of n entries, stride s, whose entries lie whole periods apart
    auto whole = [](int64_t na, int64_t nb, int64_t sa, int64_t sb, int64_t period) {
        return (na == 1 && nb == 1) || (sa == sb && period > 0 && sa % period == 0);
    };
    if (a.t > 1 && b.t > 1 && a.st == b.st && whole(a.b, b.b, a.sb, b.sb, a.st) &&
        apart(a.st, lo.head_span(), hi.head_span()))
        return true;
    return a.h > 1 && b.h > 1 && a.sh == b.sh && whole(a.b, b.b, a.sb, b.sb, a.sh) &&
           whole(a.t, b.t, a.st, b.st, a.sh) && apart(a.sh, a.hd, b.hd);
}

// The power of two up to 16 bytes that every head's start is a multiple of.
int align4(const H4& v) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(v.data) | (uint64_t)((v.sb | v.st | v.sh) * v.es()) | 16;
    return (int)(bits & (~bits + 1));
}

V flat4(const H4& v) { return V{v.data, 1, v.span(), v.span(), v.dtype}; }

int check_rope(const mbx_heads_view* q_out, const mbx_heads_view* k_out, const mbx_heads_cview* q,
               const mbx_heads_cview* k, const mbx_cview* positions, const mbx_cview* freqs, const int32_t* axes,
               int n_axes, bool dev) {
    if (!q_out || !q || !positions || !freqs || !axes) return MBX_E_NULL;
    if ((k == nullptr) != (k_out == nullptr)) return MBX_E_NULL;
    if (!positions->data || !freqs->data) return MBX_E_NULL;
    const H4 in[2] = {of4(q), k ? of4(k) : H4{}}, out[2] = {of4(q_out), k ? of4(k_out) : H4{}};
    const int nt = k ? 2 : 1;
    for (int i = 0; i < nt; ++i) {
        if (in[i].dtype != in[0].dtype || out[i].dtype != in[0].dtype) return MBX_E_DTYPE;
        MBX_TRY(basic4(out[i]));
        MBX_TRY(basic4(in[i]));
    }
    const V pv = of(positions), fv = of(freqs);
    if (pv.dtype != MBX_I32 && pv.dtype != MBX_F32) return MBX_E_DTYPE;
    if (fv.dtype != MBX_F64) return MBX_E_DTYPE;
    for (const V* v : {&pv, &fv}) {
        if (v->rows <= 0 || v->cols <= 0) return MBX_E_EMPTY;
        if (!stride_ok(*v)) return MBX_E_STRIDE;
        if (reinterpret_cast<uintptr_t>(v->data) % esize(v->dtype)) return MBX_E_ALIGN;
        MBX_TRY(extent_ok(*v));
    }
    for (int i = 0; i < nt; ++i) {
        const H4& a = in[i];
        if (a.b != in[0].b || a.t != in[0].t || a.hd != in[0].hd) return MBX_E_SHAPE;
        if (out[i].b != a.b || out[i].t != a.t || out[i].h != a.h || out[i].hd != a.hd) return MBX_E_SHAPE;
        MBX_TRY(injective4(out[i]));
    }
    int64_t tokens = 0;
    if (__builtin_mul_overflow(in[0].b, in[0].t, &tokens) || tokens > 0x7fffffff) return MBX_E_ARG;
    if (n_axes < 1 || n_axes > 4) return MBX_E_ARG;
    int64_t rot = 0;
    for (int i = 0; i < n_axes; ++i) {
        if (axes[i] < 2 || axes[i] % 2) return MBX_E_ARG;
        rot += axes[i];
    }
    if (rot > in[0].hd) return MBX_E_ARG;
    if (pv.cols != n_axes || (pv.rows != in[0].t && pv.rows != tokens)) return MBX_E_SHAPE;
    if (fv.rows != 1 || fv.cols != rot / 2) return MBX_E_SHAPE;
    // an output may be exactly its own input; nothing else overlaps an output
    for (int i = 0; i < nt; ++i) {
        for (int j = 0; j < nt; ++j) {
            if (!(i == j && same4(out[i], in[j])) && !disjoint4(out[i], in[j])) return MBX_E_ALIAS;
            if (i != j && !disjoint4(out[i], out[j])) return MBX_E_ALIAS;
        }
        if (overlaps(flat4(out[i]), pv) || overlaps(flat4(out[i]), fv)) return MBX_E_ALIAS;
    }
    if (dev) {
        const V all[6] = {pv, fv, flat4(out[0]), flat4(in[0]), flat4(out[nt - 1]), flat4(in[nt - 1])};
        MBX_TRY(views_on_device(all, k ? 6 : 4));
    }
    return MBX_OK;
}

}  // namespace

namespace mbx {

int sm_count() {
    static std::atomic<int> sms[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 0;
    }
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace mbx

// ---------------------------------------------------------------- C ABI

extern "C" {

MBX_API int mbx_check_layer_norm(const mbx_view* out, const mbx_cview* x, const mbx_cview* weight,
                                 const mbx_cview* bias, float eps) {
    return check_layer_norm(out, x, weight, bias, eps, true);
}

MBX_API int mbx_layer_norm(const mbx_view* out, const mbx_cview* x, const mbx_cview* weight, const mbx_cview* bias,
                           float eps, void* stream) {
    MBX_TRY(check_layer_norm(out, x, weight, bias, eps, true));
    mbx::LnFwdParams p = {};
    p.out = out->data;
    p.out_stride = out->row_stride;
    p.x = x->data;
    p.x_stride = x->row_stride;
    p.rows = x->rows;
    p.D = (int)x->cols;
    p.eps = eps;
    const int ce = x->dtype == MBX_F32 ? 4 : 8;
    bool vec = p.D % ce == 0 && vec_row(of(out)) && vec_row(of(x));
    if (weight) {
        p.weight = weight->data;
        p.p_f32 = weight->dtype == MBX_F32;
        vec = vec && vec_row(of(weight));
    }
    if (bias) {
        p.bias = bias->data;
        p.p_f32 = bias->dtype == MBX_F32;
        vec = vec && vec_row(of(bias));
    }
    return cuda_status(mbx::launch_layer_norm(p, x->dtype == MBX_F32, vec, (cudaStream_t)stream));
}

MBX_API int mbx_param_grad_workspace(int64_t rows, int64_t cols, int64_t mod_rows, int dtype, int64_t* bytes) {
    if (!bytes) return MBX_E_NULL;
    if (!act_dtype(dtype)) return MBX_E_DTYPE;
    if (rows <= 0 || cols <= 0 || mod_rows <= 0) return MBX_E_EMPTY;
    if (cols > kMaxHidden) return MBX_E_DIM_TOO_LARGE;
    if (rows >= (int64_t)1 << 32) return MBX_E_ARG;
    if (rows % mod_rows) return MBX_E_SHAPE;
    const int64_t need = workspace_need(rows, mod_rows, cols, dtype);
    if (need < 0) return MBX_E_DEVICE;
    *bytes = need;
    return MBX_OK;
}

MBX_API int mbx_check_layer_norm_backward(const mbx_view* dx, const mbx_view* dweight, const mbx_view* dbias,
                                          const mbx_cview* dout, const mbx_cview* x, const mbx_cview* weight,
                                          const mbx_cview* dresidual, float eps, const float* workspace,
                                          int64_t workspace_bytes) {
    return check_ln_backward(dx, dweight, dbias, dout, x, weight, dresidual, true, eps, workspace, workspace_bytes,
                             true);
}

MBX_API int mbx_layer_norm_backward(const mbx_view* dx, const mbx_view* dweight, const mbx_view* dbias,
                                    const mbx_cview* dout, const mbx_cview* x, const mbx_cview* weight,
                                    const mbx_cview* dresidual, float eps, float* workspace, int64_t workspace_bytes,
                                    void* stream) {
    MBX_TRY(check_ln_backward(dx, dweight, dbias, dout, x, weight, dresidual, true, eps, workspace, workspace_bytes,
                              true));
    return ln_backward(dx, dweight, dbias, dout, x, weight, dresidual, 0.0f, eps, workspace, stream);
}

MBX_API int mbx_check_ln_modulate_backward(const mbx_view* dx, const mbx_view* dscale, const mbx_view* dshift,
                                           const mbx_cview* dout, const mbx_cview* x, const mbx_cview* scale,
                                           const mbx_cview* dresidual, float eps, const float* workspace,
                                           int64_t workspace_bytes) {
    return check_ln_backward(dx, dscale, dshift, dout, x, scale, dresidual, false, eps, workspace, workspace_bytes,
                             true);
}

MBX_API int mbx_ln_modulate_backward(const mbx_view* dx, const mbx_view* dscale, const mbx_view* dshift,
                                     const mbx_cview* dout, const mbx_cview* x, const mbx_cview* scale,
                                     const mbx_cview* dresidual, float eps, float* workspace, int64_t workspace_bytes,
                                     void* stream) {
    MBX_TRY(check_ln_backward(dx, dscale, dshift, dout, x, scale, dresidual, false, eps, workspace, workspace_bytes,
                              true));
    return ln_backward(dx, dscale, dshift, dout, x, scale, dresidual, 1.0f, eps, workspace, stream);
}

MBX_API int mbx_check_dropout(const mbx_view* out, const mbx_cview* x, double p, const int64_t* rng, int64_t offset) {
    (void)offset;
    return check_dropout(out, nullptr, nullptr, x, false, p, rng, true);
}

MBX_API int mbx_dropout(const mbx_view* out, const mbx_cview* x, double p, const int64_t* rng, int64_t offset,
                        void* stream) {
    MBX_TRY(mbx_check_dropout(out, x, p, rng, offset));
    bool vec;
    const mbx::DropParams d = drop_params(out, x, nullptr, nullptr, p, rng, offset, &vec);
    return cuda_status(mbx::launch_dropout(d, x->dtype == MBX_F32, vec, (cudaStream_t)stream));
}

MBX_API int mbx_check_dropout_gate_add(const mbx_view* out, const mbx_cview* x, const mbx_cview* gate,
                                       const mbx_cview* y, double p, const int64_t* rng, int64_t offset) {
    (void)offset;
    return check_dropout(out, x, gate, y, true, p, rng, true);
}

MBX_API int mbx_dropout_gate_add(const mbx_view* out, const mbx_cview* x, const mbx_cview* gate, const mbx_cview* y,
                                 double p, const int64_t* rng, int64_t offset, void* stream) {
    MBX_TRY(mbx_check_dropout_gate_add(out, x, gate, y, p, rng, offset));
    bool vec;
    const mbx::DropParams d = drop_params(out, x, gate, y, p, rng, offset, &vec);
    return cuda_status(mbx::launch_dropout(d, x->dtype == MBX_F32, vec, (cudaStream_t)stream));
}

MBX_API int mbx_check_dropout_gate_add_backward(const mbx_view* dy, const mbx_view* dgate, const mbx_cview* dout,
                                                const mbx_cview* gate, const mbx_cview* y, double p,
                                                const int64_t* rng, int64_t offset, const float* workspace,
                                                int64_t workspace_bytes) {
    (void)offset;
    return check_dropout_backward(dy, dgate, dout, gate, y, p, rng, workspace, workspace_bytes, true);
}

MBX_API int mbx_dropout_gate_add_backward(const mbx_view* dy, const mbx_view* dgate, const mbx_cview* dout,
                                          const mbx_cview* gate, const mbx_cview* y, double p, const int64_t* rng,
                                          int64_t offset, float* workspace, int64_t workspace_bytes, void* stream) {
    MBX_TRY(check_dropout_backward(dy, dgate, dout, gate, y, p, rng, workspace, workspace_bytes, true));
    bool vec;
    mbx::DropParams d = drop_params(dy, dout, gate, y, p, rng, offset, &vec);
    if (dgate) {
        d.dgate = dgate->data;
        d.dgate_stride = dgate->row_stride;
        vec = vec && vec_row(of(dgate));
    }
    d.ws = workspace;
    return cuda_status(mbx::launch_dropout_backward(d, dout->dtype == MBX_F32, vec, (cudaStream_t)stream));
}

MBX_API int mbx_check_rope_axes(const mbx_heads_view* q_out, const mbx_heads_view* k_out, const mbx_heads_cview* q,
                                const mbx_heads_cview* k, const mbx_cview* positions, const mbx_cview* freqs,
                                const int32_t* axes, int n_axes, int interleaved, int inverse) {
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return MBX_E_ARG;
    return check_rope(q_out, k_out, q, k, positions, freqs, axes, n_axes, true);
}

MBX_API int mbx_rope_axes(const mbx_heads_view* q_out, const mbx_heads_view* k_out, const mbx_heads_cview* q,
                          const mbx_heads_cview* k, const mbx_cview* positions, const mbx_cview* freqs,
                          const int32_t* axes, int n_axes, int interleaved, int inverse, void* stream) {
    MBX_TRY(mbx_check_rope_axes(q_out, k_out, q, k, positions, freqs, axes, n_axes, interleaved, inverse));
    mbx::RopeParams p = {};
    const int nt = k ? 2 : 1;
    int align = 16;
    for (int i = 0; i < nt; ++i) {
        const H4 in = of4(i ? k : q), out = of4(i ? k_out : q_out);
        mbx::RopeTensor& t = i ? p.k : p.q;
        t = mbx::RopeTensor{in.data, const_cast<void*>(out.data), in.sb, in.st, in.sh, out.sb, out.st, out.sh,
                            (int)in.h};
        for (int a : {align4(in), align4(out)}) align = a < align ? a : align;
    }
    p.batch = q->batch;
    p.tokens = q->tokens;
    p.hd = (int)q->head_dim;
    int end = 0;
    for (int i = 0; i < n_axes; ++i) p.axis_end[i] = end += axes[i] / 2;
    p.axes = n_axes;
    p.pairs = end;
    p.pos = positions->data;
    p.pos_stride = positions->row_stride;
    p.pos_f32 = positions->dtype == MBX_F32;
    p.pos_batched = positions->rows != p.tokens;
    p.freqs = static_cast<const double*>(freqs->data);
    p.inverse = inverse != 0;
    return cuda_status(mbx::launch_rope_axes(p, q->dtype == MBX_F32, interleaved != 0, align, (cudaStream_t)stream));
}

}  // extern "C"
