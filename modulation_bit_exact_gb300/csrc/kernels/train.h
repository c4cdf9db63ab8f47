// train.h -- internal interface between the C ABI (train_api.cu) and the
// kernels of the training path: LayerNorm and its gradients, dropout in the
// gated residual, the sums that make the gradients of shared parameters, and
// rotary positions on several axes.  Not installed; not part of the ABI.
#pragma once

#include <atomic>

#include "launch.h"

namespace mbx {

int sm_count();  // SMs of the current device; 0 if the runtime cannot tell

// Threads that own one row of D elements, `per` elements each: 8 or 16 lanes of a
// warp for the short rows, else whole warps.
inline int row_threads(int D, int per = 16) {
    return D <= 8 * per ? 8 : D <= 16 * per ? 16 : (D + 32 * per - 1) / (32 * per) * 32;
}

// Shared memory of one staged row (rowring.cuh): its elements, and for rows that
// are not 16-byte aligned a head and room for the shift.
inline int staged_row_bytes(int tpr, int esize, bool vec, int per = 16) {
    return per * esize * tpr + (vec ? 0 : 32);
}

// Threads of an SM: the row kernels take up to 96 registers a thread, those
// that also hold the sums of their columns up to 128.  Row groups of several
// warps use the named barriers 1 to 15, so there are at most ten of them.
constexpr int kRingThreads = 640, kGradThreads = 512;

// How a kernel that streams rows through shared memory fills an SM: blocks of
// `groups` row groups, `ctas_per_sm` blocks, and for every group a ring of
// `stages` stages of `rows` rows of row_bytes (and extra_bytes); fixed_bytes are
// the block's own.
struct RingShape {
    int tpr, groups, stages, ctas_per_sm;
    int row_bytes, extra_bytes, sums_bytes, fixed_bytes, group_bytes, smem;
};
RingShape ring_shape(int tpr, int row_bytes, int rows, int extra_bytes, int fixed_per_thread,
                     int threads_per_sm, int blocks_per_sm);  // stages < 1: does not fit

// Raises a kernel's shared-memory limit once for each device.
struct SmemOptIn {
    std::atomic<int> allowed[64] = {};
    cudaError_t allow(const void* kernel, const RingShape& sh);
};

// How the rows of each modulation row (a segment of `seq` rows) are split for
// the parameter gradients: `parts` parts of `rows_per_part` rows, one block a
// part, whose partial sums a second kernel joins; one part needs neither.
struct GradPlan {
    int64_t parts, rows_per_part;
};
GradPlan grad_plan(int64_t rows, int64_t mod_rows, int D, int esize);
int64_t grad_workspace_bytes(int64_t rows, int64_t mod_rows, int D, int esize);

struct LnFwdParams {
    void* out;
    int64_t out_stride;
    const void* x;
    int64_t x_stride;
    const void* weight;  // [D] or null (1)
    const void* bias;    // [D] or null (0)
    bool p_f32;          // weight and bias are binary32
    int64_t rows;
    int D;
    float eps;
};

// Gradients of out = LN(x) * f + shift, where f = factor_add + factor:
// LayerNorm's weight (factor_add 0) or AdaLN's 1 + scale (factor_add 1).
struct LnBwdParams {
    void* dx;
    int64_t dx_stride;
    void* dfactor;  // [mod_rows, D] or null
    int64_t dfactor_stride;
    void* dshift;  // [mod_rows, D] or null
    int64_t dshift_stride;
    const void* dout;
    int64_t dout_stride;
    const void* x;
    int64_t x_stride;
    const void* factor;  // [mod_rows, D], or null: f = factor_add + 1
    int64_t factor_stride;
    float factor_add;
    const void* dres;  // added to dx, or null
    int64_t dres_stride;
    bool p_f32;  // factor, dfactor, dshift are binary32
    int64_t rows, mod_rows, seq;
    int D;
    float eps;
    float neg_zero;  // -0.0f
    float* ws;
    GradPlan plan;  // filled by the launcher
};

struct DropParams {
    void* out;  // forward: out; backward: dy
    int64_t out_stride;
    const void* x;  // forward: the residual, or null (plain dropout); backward: dout
    int64_t x_stride;
    const void* y;
    int64_t y_stride;
    const void* gate;  // [mod_rows, D], or null (plain dropout)
    int64_t gate_stride;
    void* dgate;
    int64_t dgate_stride;
    bool p_f32;  // gate and dgate are binary32
    const int64_t* rng;  // device: seed, counter
    int64_t offset;
    uint32_t threshold;  // an element is kept where its word >= threshold
    float inv_keep;      // 1 / (1 - p)
    int64_t rows, mod_rows, seq;
    int D;
    float* ws;
    GradPlan plan;  // filled by the launcher
};

// out[k][s][c] = sum over the parts of ws[s][part][k][c], k < nacc.
struct ColSumParams {
    const float* ws;
    int64_t parts, segments;
    int D, nacc;
    void* out[2];  // null: not written
    int64_t out_stride[2];
    bool p_f32;
};

struct RopeTensor {
    const void* in;
    void* out;
    int64_t ib, it, ih, ob, ot, oh;  // batch, token and head strides (elements)
    int heads;
};
struct RopeParams {
    RopeTensor q, k;  // k.heads = 0: none
    int64_t batch, tokens;
    int hd, pairs;  // pairs = rotated elements of a head / 2
    const void* pos;  // [tokens or batch*tokens, axes]
    int64_t pos_stride;
    bool pos_f32, pos_batched;
    const double* freqs;  // [pairs] radians per position
    int axis_end[4];      // pair j belongs to the first axis a with j < axis_end[a]
    int axes;
    bool inverse;
};

cudaError_t launch_layer_norm(const LnFwdParams& p, bool f32, bool vec, cudaStream_t s);
cudaError_t launch_ln_backward(const LnBwdParams& p, bool f32, bool vec, cudaStream_t s);
cudaError_t launch_dropout(const DropParams& p, bool f32, bool vec, cudaStream_t s);
cudaError_t launch_dropout_backward(const DropParams& p, bool f32, bool vec, cudaStream_t s);
cudaError_t launch_column_sums(const ColSumParams& p, cudaStream_t s);
cudaError_t launch_rope_axes(const RopeParams& p, bool f32, bool interleaved, int align, cudaStream_t s);

}  // namespace mbx
