// qknorm_api.cu -- the C ABI of the norm and rotation of Q and K heads and of its
// gradients: validation and dispatch.  The order of the checks is that of
// mbx_api.cu: pure host checks first, then the device checks, then the launch.
#include <cuda_runtime.h>

#include "heads.h"
#include "kernels/train.h"
#include "mbx.h"

namespace {

// The operands of one call; index 0 is Q's, 1 is K's.
struct Call {
    const mbx_heads_view* out[2];
    const mbx_heads_cview* dout[2];  // null in the forward call
    const mbx_heads_cview* x[2];
    const mbx_cview* w[2];
    const mbx_view* dw[2];
    const mbx_cview *positions, *freqs;
    const int32_t* axes;
    int n_axes, interleaved;
    float eps;
    const float* ws;
    int64_t ws_bytes;
    bool backward;
};

int64_t workspace_need(int64_t batch, int64_t tokens, int64_t head_dim) {
    if (mbx::sm_count() < 1) return -1;
    return mbx::qk_norm_grad_parts(batch, tokens) * 2 * head_dim * (int64_t)sizeof(float);
}

int check(const Call& c) {
    if (!c.out[0] || !c.x[0] || (c.backward && !c.dout[0])) return MBX_E_NULL;
    const int nt = c.x[1] ? 2 : 1;
    if ((c.out[1] != nullptr) != (nt == 2) || (c.backward && (c.dout[1] != nullptr) != (nt == 2))) return MBX_E_NULL;
    if (!c.positions || !c.freqs || !c.axes || !c.positions->data || !c.freqs->data) return MBX_E_NULL;
    if ((c.interleaved != 0 && c.interleaved != 1)) return MBX_E_ARG;
    for (int i = 0; i < 2; ++i)
        if ((c.w[i] && i >= nt) || (c.dw[i] && !c.w[i])) return MBX_E_NULL;

    const int no = c.backward ? 3 : 2;  // views of heads of a tensor: out, x, dout
    H4 h[2][3] = {};
    for (int i = 0; i < nt; ++i) {
        h[i][0] = of4(c.out[i]);
        h[i][1] = of4(c.x[i]);
        if (c.backward) h[i][2] = of4(c.dout[i]);
        for (int j = 0; j < no; ++j) {
            if (h[i][j].data && h[i][j].dtype != h[0][1].dtype) return MBX_E_DTYPE;
            MBX_TRY(basic4(h[i][j]));
        }
    }
    const H4& x = h[0][1];
    V pw[4];  // weights, then their gradients
    const V* w_of[2] = {};
    int np = 0, n_in = 0;
    for (int i = 0; i < nt; ++i)
        if (c.w[i]) w_of[i] = &(pw[np++] = of(c.w[i]));
    n_in = np;
    for (int i = 0; i < nt; ++i)
        if (c.dw[i]) pw[np++] = of(c.dw[i]);
    for (int i = 0; i < np; ++i) {
        if (!pw[i].data) return MBX_E_NULL;
        if (!param_dtype(pw[i].dtype, x.dtype) || pw[i].dtype != pw[0].dtype) return MBX_E_DTYPE;
        MBX_TRY(basic_any(pw[i]));
    }
    const V pv = of(c.positions), fv = of(c.freqs);
    MBX_TRY(check_turn_views(pv, fv));

    for (int i = 0; i < nt; ++i) {
        const H4& a = h[i][1];
        if (a.b != x.b || a.t != x.t || a.hd != x.hd) return MBX_E_SHAPE;
        for (int j = 0; j < no; ++j)
            if (h[i][j].b != a.b || h[i][j].t != a.t || h[i][j].h != a.h || h[i][j].hd != a.hd) return MBX_E_SHAPE;
        MBX_TRY(injective4(h[i][0]));
    }
    for (int i = 0; i < np; ++i)
        if (pw[i].rows != 1 || pw[i].cols != x.hd) return MBX_E_SHAPE;
    MBX_TRY(check_turn(x, pv, fv, c.axes, c.n_axes));
    MBX_TRY(check_eps(c.eps));

    // An output may be exactly its own input (forward x, backward dout); no output
    // overlaps anything else.
    V small[6];  // the parameters, positions and frequencies
    int ns = 0;
    for (int i = 0; i < np; ++i) small[ns++] = pw[i];
    small[ns++] = pv;
    small[ns++] = fv;
    const int own = c.backward ? 2 : 1;
    for (int i = 0; i < nt; ++i) {
        for (int k = 0; k < nt; ++k) {
            for (int j = 1; j < no; ++j)
                if (!(i == k && j == own && same4(h[i][0], h[k][j])) && !disjoint4(h[i][0], h[k][j])) return MBX_E_ALIAS;
            if (i != k && !disjoint4(h[i][0], h[k][0])) return MBX_E_ALIAS;
        }
        for (int k = 0; k < ns; ++k)
            if (overlaps(flat4(h[i][0]), small[k])) return MBX_E_ALIAS;
    }
    for (int g = n_in; g < np; ++g) {
        for (int k = 0; k < ns; ++k)
            if (k != g && overlaps(pw[g], small[k])) return MBX_E_ALIAS;
        for (int i = 0; i < nt; ++i)
            for (int j = 1; j < no; ++j)
                if (overlaps(pw[g], flat4(h[i][j]))) return MBX_E_ALIAS;
    }

    V all[14];
    int n = 0;
    for (int i = 0; i < ns; ++i) all[n++] = small[i];
    for (int i = 0; i < nt; ++i)
        for (int j = 0; j < no; ++j) all[n++] = flat4(h[i][j]);
    if (np > n_in) {
        // without a device the size is unknown: the device check refuses the call
        const int64_t need = workspace_need(x.b, x.t, x.hd);
        if (need > 0) {
            MBX_TRY(check_workspace(c.ws, c.ws_bytes, need, all, n));
            all[n++] = V{c.ws, 1, need / 4, need / 4, MBX_F32};
        }
    }
    return views_on_device(all, n);
}

mbx::QkNormParams params(const Call& c, int* align) {
    mbx::QkNormParams p = {};
    mbx::RopeParams& r = p.rope;
    *align = 16;
    for (int i = 0; i < 2 && c.x[i]; ++i) {
        const H4 in = of4(c.x[i]), out = of4(c.out[i]);
        (i ? r.k : r.q) = mbx::RopeTensor{in.data, const_cast<void*>(out.data), in.sb, in.st, in.sh, out.sb, out.st, out.sh,
                                          (int)in.h};
        for (int a : {align4(in), align4(out)}) *align = a < *align ? a : *align;
        if (c.backward) {
            const H4 d = of4(c.dout[i]);
            p.dout[i] = mbx::GradIn{d.data, d.sb, d.st, d.sh};
            if (align4(d) < *align) *align = align4(d);
        }
        if (c.w[i]) {
            p.w[i] = c.w[i]->data;
            p.w_f32 = c.w[i]->dtype == MBX_F32;
        }
    }
    r.batch = c.x[0]->batch;
    r.tokens = c.x[0]->tokens;
    r.hd = (int)c.x[0]->head_dim;
    int end = 0;
    for (int i = 0; i < c.n_axes; ++i) r.axis_end[i] = end += c.axes[i] / 2;
    r.axes = c.n_axes;
    r.pairs = end;
    r.pos = c.positions->data;
    r.pos_stride = c.positions->row_stride;
    r.pos_f32 = c.positions->dtype == MBX_F32;
    r.pos_batched = c.positions->rows != r.tokens;
    r.freqs = static_cast<const double*>(c.freqs->data);
    r.inverse = c.backward;
    p.eps = c.eps;
    p.inv_hd = 1.0f / (float)r.hd;
    return p;
}

}  // namespace

extern "C" {

MBX_API int mbx_check_qk_norm_rope(const mbx_heads_view* q_out, const mbx_heads_view* k_out, const mbx_heads_cview* q,
                                   const mbx_heads_cview* k, const mbx_cview* wq, const mbx_cview* wk,
                                   const mbx_cview* positions, const mbx_cview* freqs, const int32_t* axes, int n_axes,
                                   int interleaved, float eps) {
    return check(Call{{q_out, k_out}, {}, {q, k}, {wq, wk}, {}, positions, freqs, axes, n_axes, interleaved, eps, nullptr, 0,
                      false});
}

MBX_API int mbx_qk_norm_rope(const mbx_heads_view* q_out, const mbx_heads_view* k_out, const mbx_heads_cview* q,
                             const mbx_heads_cview* k, const mbx_cview* wq, const mbx_cview* wk, const mbx_cview* positions,
                             const mbx_cview* freqs, const int32_t* axes, int n_axes, int interleaved, float eps,
                             void* stream) {
    const Call c{{q_out, k_out}, {}, {q, k}, {wq, wk}, {}, positions, freqs, axes, n_axes, interleaved, eps, nullptr, 0, false};
    MBX_TRY(check(c));
    int align;
    const mbx::QkNormParams p = params(c, &align);
    return cuda_status(mbx::launch_qk_norm_rope(p, q->dtype == MBX_F32, interleaved != 0, align, (cudaStream_t)stream));
}

MBX_API int mbx_qk_norm_grad_workspace(int64_t batch, int64_t tokens, int64_t head_dim, int64_t* bytes) {
    if (!bytes) return MBX_E_NULL;
    if (batch <= 0 || tokens <= 0 || head_dim <= 0) return MBX_E_EMPTY;
    if (head_dim > 256) return MBX_E_DIM_TOO_LARGE;
    int64_t total = 0;
    if (__builtin_mul_overflow(batch, tokens, &total) || total > 0x7fffffff) return MBX_E_ARG;
    const int64_t need = workspace_need(batch, tokens, head_dim);
    if (need < 0) return MBX_E_DEVICE;
    *bytes = need;
    return MBX_OK;
}

MBX_API int mbx_check_qk_norm_rope_backward(const mbx_heads_view* dq, const mbx_heads_view* dk, const mbx_view* dwq,
                                            const mbx_view* dwk, const mbx_heads_cview* dq_out,
                                            const mbx_heads_cview* dk_out, const mbx_heads_cview* q,
                                            const mbx_heads_cview* k, const mbx_cview* wq, const mbx_cview* wk,
                                            const mbx_cview* positions, const mbx_cview* freqs, const int32_t* axes,
                                            int n_axes, int interleaved, float eps, const float* workspace,
                                            int64_t workspace_bytes) {
    return check(Call{{dq, dk}, {dq_out, dk_out}, {q, k}, {wq, wk}, {dwq, dwk}, positions, freqs, axes, n_axes, interleaved,
                      eps, workspace, workspace_bytes, true});
}

MBX_API int mbx_qk_norm_rope_backward(const mbx_heads_view* dq, const mbx_heads_view* dk, const mbx_view* dwq,
                                      const mbx_view* dwk, const mbx_heads_cview* dq_out, const mbx_heads_cview* dk_out,
                                      const mbx_heads_cview* q, const mbx_heads_cview* k, const mbx_cview* wq,
                                      const mbx_cview* wk, const mbx_cview* positions, const mbx_cview* freqs,
                                      const int32_t* axes, int n_axes, int interleaved, float eps, float* workspace,
                                      int64_t workspace_bytes, void* stream) {
    const Call c{{dq, dk},    {dq_out, dk_out}, {q, k},    {wq, wk}, {dwq, dwk}, positions, freqs, axes, n_axes,
                 interleaved, eps,              workspace, workspace_bytes, true};
    MBX_TRY(check(c));
    int align;
    mbx::QkNormParams p = params(c, &align);
    mbx::ColSumParams s = {};
    if (dwq || dwk) {
        p.ws = workspace;
        s.ws = workspace;
        s.segments = 1;
        s.D = p.rope.hd;
        s.nacc = 2;
        s.p_f32 = p.w_f32;
        if (dwq) s.out[0] = dwq->data;
        if (dwk) s.out[1] = dwk->data;
    }
    return cuda_status(mbx::launch_qk_norm_rope_backward(p, q->dtype == MBX_F32, interleaved != 0, align, s,
                                                         (cudaStream_t)stream));
}

}  // extern "C"
