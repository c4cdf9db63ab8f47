// layernorm.cu -- affine LayerNorm, and the gradients of LayerNorm with a
// factor and a shift: the affine weight and bias, or AdaLN's 1 + scale and
// shift with one row of each for a sample or for a token.
//
//   mean, var over the row (biased); rstd = 1/sqrt(var + eps);
//   xh = (x - mean) * rstd;  y = xh * f + b
//   gy = dy * f;  c1 = mean(gy);  c2 = mean(gy * xh)
//   dx = rstd * (gy - c1 - xh * c2)  (+ the residual stream's gradient)
//   df = sum over the factor's rows of dy * xh;  db = sum of dy
//
// All of it is binary32 with one rounding at each output.  The variance is the
// mean of the squared deviations of registers that hold the whole row (no
// E[x^2] - mean^2), so a row with a large mean loses nothing.
//
// The backward pass takes the statistics from x again instead of reading saved
// ones: x is in registers for xh anyway, sum(x) travels with sum(gy) and
// sum((x-mean)^2) with sum(gy*(x-mean)), so it costs one more row sum of two
// and no memory, and a forward pass need not save anything.
#include "rowgroup.cuh"

namespace mbx {

template <class T, int NCH, Access A>
__global__ void __launch_bounds__(512) layer_norm_kernel(LnFwdParams p, int tpr) {
    constexpr int CE = ChunkOf<T>::CE, E = NCH * CE;
    __shared__ float2 sums[512 / 32][2][kMaxWarpsPerRow];
    const int g = threadIdx.x / tpr, t = threadIdx.x % tpr, groups = blockDim.x / tpr;
    GroupSum gsum{&sums[g][0][0], t, tpr, g + 1, 0};
    const float inv_d = 1.0f / (float)p.D;
    grid_dep_wait();  // launched programmatically: the previous kernel has finished
    grid_dep_launch();

    float w[E], b[E];
    if (p.weight) load_params<T, NCH, A>(w, p.weight, 0, p.p_f32, p.D, t, tpr, 0.0f);
    else
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = 1.0f;
    if (p.bias) load_params<T, NCH, A>(b, p.bias, 0, p.p_f32, p.D, t, tpr, 0.0f);
    else
#pragma unroll
        for (int e = 0; e < E; ++e) b[e] = 0.0f;

    const T* x = static_cast<const T*>(p.x);
    T* out = static_cast<T*>(p.out);
    const int64_t step = (int64_t)gridDim.x * groups;
    RawRow<T, NCH, A> next;
    int64_t row = (int64_t)blockIdx.x * groups + g;
    if (row < p.rows) next.load(x + row * p.x_stride, p.D, t, tpr);
    for (; row < p.rows; row += step) {
        float v[E];
        next.widen(v);
        if (row + step < p.rows) next.load(x + (row + step) * p.x_stride, p.D, t, tpr);
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += v[e];
        const float mean = gsum(s, 0.0f).x * inv_d;
        float q = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            v[e] = col_of<T, A>(e, t, tpr) < p.D ? v[e] - mean : 0.0f;
            q = fmaf(v[e], v[e], q);
        }
        const float var = gsum(q, 0.0f).x * inv_d;
        const float rstd = 1.0f / sqrtf(var + p.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fmaf(v[e] * rstd, w[e], b[e]);
        store_row<T, NCH, A>(out + row * p.out_stride, v, p.D, t, tpr);
    }
}

// One row's gradient: v holds x and becomes xh, dy holds dy, dx is returned.
template <class T, int NCH, Access A>
__device__ __forceinline__ void ln_row_backward(float (&v)[NCH * ChunkOf<T>::CE], const float (&dy)[NCH * ChunkOf<T>::CE],
                                                const float (&f)[NCH * ChunkOf<T>::CE],
                                                float (&dx)[NCH * ChunkOf<T>::CE], const LnBwdParams& p, float inv_d,
                                                GroupSum& gsum) {
    constexpr int CE = ChunkOf<T>::CE, E = NCH * CE;
    float s = 0.0f, sg = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        s += v[e];
        dx[e] = dy[e] * f[e];  // gy
        sg += dx[e];
    }
    const float2 m = gsum(s, sg);
    const float mean = m.x * inv_d, c1 = m.y * inv_d;
    float q = 0.0f, qg = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        v[e] = col_of<T, A>(e, gsum.t, gsum.tpr) < p.D ? v[e] - mean : 0.0f;
        q = fmaf(v[e], v[e], q);
        qg = fmaf(dx[e], v[e], qg);
    }
    const float2 m2 = gsum(q, qg);
    const float rstd = 1.0f / sqrtf(m2.x * inv_d + p.eps);
    const float c2 = m2.y * inv_d * rstd;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        v[e] *= rstd;
        dx[e] = rstd * (fmaf(-v[e], c2, dx[e] - c1));
    }
}

template <class T, int NCH, Access A>
__device__ __forceinline__ void load_factor(float (&f)[NCH * ChunkOf<T>::CE], const LnBwdParams& p, int64_t mrow, int t,
                                            int tpr) {
    constexpr int E = NCH * ChunkOf<T>::CE;
    if (p.factor) {
        load_params<T, NCH, A>(f, p.factor, mrow * p.factor_stride, p.p_f32, p.D, t, tpr, 0.0f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] += p.factor_add;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = 1.0f + p.factor_add;
    }
}

// One modulation row for every row: nothing is summed, every output is a row.
template <class T, int NCH, Access A>
__global__ void __launch_bounds__(512) ln_backward_token_kernel(LnBwdParams p) {
    constexpr int CE = ChunkOf<T>::CE, E = NCH * CE;
    __shared__ float2 sums[512 / 32][2][kMaxWarpsPerRow];
    const int tpr = p.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr, groups = blockDim.x / tpr;
    GroupSum gsum{&sums[g][0][0], t, tpr, g + 1, 0};
    const float inv_d = 1.0f / (float)p.D;
    grid_dep_wait();
    grid_dep_launch();
    const int64_t step = (int64_t)gridDim.x * groups;
    for (int64_t row = (int64_t)blockIdx.x * groups + g; row < p.rows; row += step) {
        RawRow<T, NCH, A> rx, rd, rr;
        rx.load(static_cast<const T*>(p.x) + row * p.x_stride, p.D, t, tpr);
        rd.load(static_cast<const T*>(p.dout) + row * p.dout_stride, p.D, t, tpr);
        float v[E], dy[E], f[E], dx[E];
        load_factor<T, NCH, A>(f, p, row, t, tpr);
        if (p.dres) rr.load(static_cast<const T*>(p.dres) + row * p.dres_stride, p.D, t, tpr);
        rx.widen(v);
        rd.widen(dy);
        ln_row_backward<T, NCH, A>(v, dy, f, dx, p, inv_d, gsum);
        if (p.dres) {
            float r[E];
            rr.widen(r);
#pragma unroll
            for (int e = 0; e < E; ++e) dx[e] += r[e];
        }
        store_row<T, NCH, A>(static_cast<T*>(p.dx) + row * p.dx_stride, dx, p.D, t, tpr);
        if (p.dshift) store_params<T, NCH, A>(p.dshift, row * p.dshift_stride, p.p_f32, dy, p.D, t, tpr);
        if (p.dfactor) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= dy[e];
            store_params<T, NCH, A>(p.dfactor, row * p.dfactor_stride, p.p_f32, v, p.D, t, tpr);
        }
    }
}

// Modulation rows shared by seq rows: a block takes one part of a segment, its
// row groups the rows of the part in turn; every thread sums its own columns
// in binary32 registers, the groups are added in shared memory, and the part's
// sums go to the workspace (or out, when the segment is one part).
template <class T, int NCH, Access A>
__global__ void __launch_bounds__(512) ln_backward_kernel(LnBwdParams p) {
    constexpr int CE = ChunkOf<T>::CE, E = NCH * CE;
    __shared__ float2 sums[512 / 32][2][kMaxWarpsPerRow];
    extern __shared__ float acc_smem[];  // [2][E][block]
    const int tpr = p.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr, groups = blockDim.x / tpr;
    GroupSum gsum{&sums[g][0][0], t, tpr, g + 1, 0};
    const float inv_d = 1.0f / (float)p.D;
    grid_dep_wait();
    grid_dep_launch();
    const T* px = static_cast<const T*>(p.x);
    const T* pd = static_cast<const T*>(p.dout);
    const T* pr = static_cast<const T*>(p.dres);
    const int64_t units = p.mod_rows * p.plan.parts;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t seg = unit / p.plan.parts, part = unit - seg * p.plan.parts;
        const int64_t r0 = seg * p.seq + part * p.plan.rows_per_part;
        int64_t r1 = r0 + p.plan.rows_per_part;
        if (r1 > (seg + 1) * p.seq) r1 = (seg + 1) * p.seq;
        float f[E], adf[E], ads[E];
        load_factor<T, NCH, A>(f, p, seg, t, tpr);
#pragma unroll
        for (int e = 0; e < E; ++e) adf[e] = ads[e] = 0.0f;
        RawRow<T, NCH, A> rx, rd;
        int64_t row = r0 + g;
        if (row < r1) {
            rx.load(px + row * p.x_stride, p.D, t, tpr);
            rd.load(pd + row * p.dout_stride, p.D, t, tpr);
        }
        for (; row < r1; row += groups) {
            float v[E], dy[E], dx[E];
            rx.widen(v);
            rd.widen(dy);
            RawRow<T, NCH, A> rr;
            if (pr) rr.load(pr + row * p.dres_stride, p.D, t, tpr);
            if (row + groups < r1) {
                rx.load(px + (row + groups) * p.x_stride, p.D, t, tpr);
                rd.load(pd + (row + groups) * p.dout_stride, p.D, t, tpr);
            }
            ln_row_backward<T, NCH, A>(v, dy, f, dx, p, inv_d, gsum);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                adf[e] = fmaf(dy[e], v[e], adf[e]);
                ads[e] += dy[e];
            }
            if (pr) {
                float r[E];
                rr.widen(r);
#pragma unroll
                for (int e = 0; e < E; ++e) dx[e] += r[e];
            }
            store_row<T, NCH, A>(static_cast<T*>(p.dx) + row * p.dx_stride, dx, p.D, t, tpr);
        }
        if (p.dfactor == nullptr && p.dshift == nullptr) continue;
        if (groups > 1) {
            const int n = blockDim.x;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                acc_smem[e * n + threadIdx.x] = adf[e];
                acc_smem[(E + e) * n + threadIdx.x] = ads[e];
            }
            __syncthreads();
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    for (int k = 1; k < groups; ++k) {
                        adf[e] += acc_smem[e * n + k * tpr + t];
                        ads[e] += acc_smem[(E + e) * n + k * tpr + t];
                    }
            }
            __syncthreads();
        }
        if (g == 0) {
            if (p.plan.parts == 1) {
                if (p.dfactor)
                    store_params<T, NCH, A>(p.dfactor, seg * p.dfactor_stride, p.p_f32, adf, p.D, t, tpr);
                if (p.dshift) store_params<T, NCH, A>(p.dshift, seg * p.dshift_stride, p.p_f32, ads, p.D, t, tpr);
            } else {
                store_params<T, NCH, A>(p.ws, unit * 2 * p.D, true, adf, p.D, t, tpr);
                store_params<T, NCH, A>(p.ws, (unit * 2 + 1) * p.D, true, ads, p.D, t, tpr);
            }
        }
    }
}

// ---------------------------------------------------------------- launch

template <class T, int NCH>
static cudaError_t ln_fwd(const LnFwdParams& p, const RowShape& sh, bool vec, cudaStream_t s) {
    auto k = vec ? layer_norm_kernel<T, NCH, kVec> : layer_norm_kernel<T, NCH, kScalar>;
    const int grid = grid_for_rows(reinterpret_cast<const void*>(k), p.rows, sh.groups, sh.block());
    if (grid < 0) return cudaErrorUnknown;
    return launch_pdl(k, grid, sh.block(), 0, s, p, sh.tpr);
}

cudaError_t launch_layer_norm(const LnFwdParams& p, bool f32, bool vec, cudaStream_t s) {
    const RowShape sh = row_shape(p.D, f32 ? 4 : 2);
    if (f32) return sh.epl == 16 ? ln_fwd<float, 4>(p, sh, vec, s) : ln_fwd<float, 2>(p, sh, vec, s);
    return sh.epl == 16 ? ln_fwd<uint16_t, 2>(p, sh, vec, s) : ln_fwd<uint16_t, 1>(p, sh, vec, s);
}

template <class T, int NCH>
static cudaError_t ln_bwd(const LnBwdParams& p0, const RowShape& sh, bool vec, cudaStream_t s) {
    LnBwdParams p = p0;
    p.tpr = sh.tpr;
    if (p.seq == 1) {
        auto k = vec ? ln_backward_token_kernel<T, NCH, kVec> : ln_backward_token_kernel<T, NCH, kScalar>;
        const int grid = grid_for_rows(reinterpret_cast<const void*>(k), p.rows, sh.groups, sh.block());
        if (grid < 0) return cudaErrorUnknown;
        return launch_pdl(k, grid, sh.block(), 0, s, p);
    }
    p.plan = grad_plan(p.rows, p.mod_rows, sh);
    const int block = p.plan.groups * sh.tpr;
    const size_t smem = p.plan.groups > 1 ? (size_t)block * sh.epl * 2 * sizeof(float) : 0;
    const int64_t units = p.mod_rows * p.plan.parts;
    auto k = vec ? ln_backward_kernel<T, NCH, kVec> : ln_backward_kernel<T, NCH, kScalar>;
    cudaError_t e = launch_pdl(k, (unsigned)(units < (1 << 30) ? units : (1 << 30)), block, smem, s, p);
    if (e != cudaSuccess || p.plan.parts == 1 || (!p.dfactor && !p.dshift)) return e;
    ColSumParams c{p.ws, p.plan.parts, p.mod_rows, p.D, 2, {p.dfactor, p.dshift}, {p.dfactor_stride, p.dshift_stride}, p.p_f32};
    return launch_column_sums(c, s);
}

cudaError_t launch_ln_backward(const LnBwdParams& p, bool f32, bool vec, cudaStream_t s) {
    const RowShape sh = row_shape(p.D, f32 ? 4 : 2);
    return launch_all_or_none([&] {
        if (f32) return sh.epl == 16 ? ln_bwd<float, 4>(p, sh, vec, s) : ln_bwd<float, 2>(p, sh, vec, s);
        return sh.epl == 16 ? ln_bwd<uint16_t, 2>(p, sh, vec, s) : ln_bwd<uint16_t, 1>(p, sh, vec, s);
    });
}

}  // namespace mbx
