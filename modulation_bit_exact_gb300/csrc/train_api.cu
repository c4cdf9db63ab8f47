// train_api.cu -- the C ABI of the training path: validation and dispatch of
// mbx_layer_norm and its gradients, mbx_ln_modulate_backward, the dropout
// entry points and mbx_rope_axes.  The order of the checks is that of
// mbx_api.cu: pure host checks first, then the device checks, then the launch.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "heads.h"
#include "kernels/train.h"
#include "mbx.h"

namespace {

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

bool vec_row(const V& v) { return aligned16(v); }

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
    MBX_TRY(check_turn_views(pv, fv));
    for (int i = 0; i < nt; ++i) {
        const H4& a = in[i];
        if (a.b != in[0].b || a.t != in[0].t || a.hd != in[0].hd) return MBX_E_SHAPE;
        if (out[i].b != a.b || out[i].t != a.t || out[i].h != a.h || out[i].hd != a.hd) return MBX_E_SHAPE;
        MBX_TRY(injective4(out[i]));
    }
    MBX_TRY(check_turn(in[0], pv, fv, axes, n_axes));
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
