// linear_api.cu -- the C ABI of the products with NVFP4 weights: validation and
// dispatch.  The order of the checks is that of mbx_api.cu: pure host checks
// first, then the device checks, then the launch.
#include <cuda_runtime.h>

#include "heads.h"
#include "kernels/linear.h"
#include "mbx.h"

namespace {

constexpr int64_t kMaxRows = 256, kMaxOutputs = (int64_t)1 << 24;

int64_t workspace_need(int64_t rows, int64_t outputs, int64_t cols) {
    if (mbx::sm_count() < 1) return -1;
    return mbx::linear_nvfp4_workspace_bytes((int)rows, outputs, (int)cols);
}

int check(const mbx_view* out, const mbx_cview* x, const mbx_cview* w4, const mbx_cview* w_sf, const float* fp4_scale,
          const mbx_cview* bias, int silu, const float* ws, int64_t ws_bytes) {
    if (!out || !x || !w4 || !w_sf || !fp4_scale) return MBX_E_NULL;
    const V o = of(out), xv = of(x), w = of(w4), sf = of(w_sf), b = bias ? of(bias) : V{};
    if (!o.data || !xv.data || !w.data || !sf.data || (bias && !b.data)) return MBX_E_NULL;
    if (!act_dtype(xv.dtype) || !param_dtype(o.dtype, xv.dtype)) return MBX_E_DTYPE;
    if (bias && !act_dtype(b.dtype)) return MBX_E_DTYPE;
    if (w.dtype != MBX_E2M1X2 || sf.dtype != MBX_E4M3) return MBX_E_DTYPE;
    MBX_TRY(basic_any(o));
    MBX_TRY(basic_any(xv));
    if (bias) MBX_TRY(basic_any(b));
    for (const V* v : {&w, &sf}) {
        if (v->rows <= 0 || v->cols <= 0) return MBX_E_EMPTY;
        if (!stride_ok(*v) || (v == &sf && v->rows > 1 && v->stride != v->cols)) return MBX_E_STRIDE;
        MBX_TRY(extent_ok(*v));
    }
    if (reinterpret_cast<uintptr_t>(fp4_scale) % 4) return MBX_E_ALIGN;
    if (xv.cols > kMaxHidden) return MBX_E_DIM_TOO_LARGE;
    if (xv.cols % 16 || w.cols != xv.cols / 2) return MBX_E_SHAPE;
    if (sf.rows != (w.rows + 127) / 128 * 128 || sf.cols != (xv.cols / 16 + 3) / 4 * 4) return MBX_E_SHAPE;
    if (o.rows != xv.rows || o.cols != w.rows) return MBX_E_SHAPE;
    if (bias && (b.rows != 1 || b.cols != w.rows)) return MBX_E_SHAPE;
    if (xv.rows > kMaxRows || w.rows > kMaxOutputs || (silu != 0 && silu != 1)) return MBX_E_ARG;
    const V gs{fp4_scale, 1, 1, 1, MBX_F32};
    V all[7] = {o, xv, w, sf, gs, b};
    int n = bias ? 6 : 5;
    for (int i = 1; i < n; ++i)
        if (overlaps(o, all[i])) return MBX_E_ALIAS;
    // without a device the size is unknown: the device check refuses the call
    const int64_t need = workspace_need(xv.rows, w.rows, xv.cols);
    if (need > 0) {
        MBX_TRY(check_workspace(ws, ws_bytes, need, all, n));
        all[n++] = V{ws, 1, need / 4, need / 4, MBX_F32};
    }
    return views_on_device(all, n);
}

}  // namespace

extern "C" {

MBX_API int mbx_check_linear_nvfp4(const mbx_view* out, const mbx_cview* x, const mbx_cview* w4, const mbx_cview* w_sf,
                                   const float* fp4_scale, const mbx_cview* bias, int silu,
                                   const float* workspace, int64_t workspace_bytes) {
    return check(out, x, w4, w_sf, fp4_scale, bias, silu, workspace, workspace_bytes);
}

MBX_API int mbx_linear_nvfp4_workspace(int64_t rows, int64_t outputs, int64_t cols, int64_t* bytes) {
    if (!bytes) return MBX_E_NULL;
    if (rows <= 0 || outputs <= 0 || cols <= 0) return MBX_E_EMPTY;
    if (cols > kMaxHidden) return MBX_E_DIM_TOO_LARGE;
    if (cols % 16) return MBX_E_SHAPE;
    if (rows > kMaxRows || outputs > kMaxOutputs) return MBX_E_ARG;
    const int64_t need = workspace_need(rows, outputs, cols);
    if (need < 0) return MBX_E_DEVICE;
    *bytes = need;
    return MBX_OK;
}

MBX_API int mbx_linear_nvfp4(const mbx_view* out, const mbx_cview* x, const mbx_cview* w4, const mbx_cview* w_sf,
                             const float* fp4_scale, const mbx_cview* bias, int silu, float* workspace,
                             int64_t workspace_bytes, void* stream) {
    MBX_TRY(check(out, x, w4, w_sf, fp4_scale, bias, silu, workspace, workspace_bytes));
    mbx::LinearParams p = {};
    p.out = out->data;
    p.out_stride = out->row_stride;
    p.x = x->data;
    p.x_stride = x->row_stride;
    p.rows = (int)x->rows;
    p.K = (int)x->cols;
    p.N = w4->rows;
    p.w4 = static_cast<const uint8_t*>(w4->data);
    p.w_stride = w4->rows > 1 ? w4->row_stride : w4->cols;
    p.sf = static_cast<const uint8_t*>(w_sf->data);
    p.sf_col_tiles = (int)(w_sf->cols / 4);
    p.gs = fp4_scale;
    if (bias) {
        p.bias = bias->data;
        p.bias_f32 = bias->dtype == MBX_F32;
    }
    p.silu = silu != 0;
    p.ws = workspace;
    return cuda_status(mbx::launch_linear_nvfp4(p, x->dtype == MBX_F32, out->dtype == MBX_F32, (cudaStream_t)stream));
}

}  // extern "C"
