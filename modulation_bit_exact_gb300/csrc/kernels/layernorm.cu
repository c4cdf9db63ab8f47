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
#include "lnorm.cuh"

namespace mbx {

// R rows of a group at a time: their sums share the shuffles and the barrier.
template <class T, int NCH, Access A, int R>
__global__ void __launch_bounds__(kRingThreads) layer_norm_kernel(LnFwdParams p, RingShape sh) {
    constexpr int CE = ChunkOf<T>::CE, E = NCH * CE;
    extern __shared__ __align__(16) char smem[];
    const int tpr = sh.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const Lane L = make_lane<CE, A>(t, tpr, p.D);
    GroupSums sums = group_sums(smem, sh, g, t);
    char* ring = smem + sh.sums_bytes + g * sh.group_bytes;
    const float inv_d = 1.0f / (float)p.D;
    grid_dep_wait();  // launched programmatically: the previous kernel has finished
    grid_dep_launch();

    u64 w[E / 2], b[E / 2];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        u64 c[CE / 2];
#pragma unroll
        for (int i = 0; i < CE / 2; ++i) c[i] = f2(1.0f, 1.0f);
        if (p.weight) get_param_chunk<T, CE, A>(c, p.weight, 0, p.p_f32, j, L);
#pragma unroll
        for (int i = 0; i < CE / 2; ++i) w[j * (CE / 2) + i] = c[i], c[i] = 0;
        if (p.bias) get_param_chunk<T, CE, A>(c, p.bias, 0, p.p_f32, j, L);
#pragma unroll
        for (int i = 0; i < CE / 2; ++i) b[j * (CE / 2) + i] = c[i];
    }

    const T* x = static_cast<const T*>(p.x);
    T* out = static_cast<T*>(p.out);
    const int row_bytes = sh.row_bytes, stage_bytes = R * row_bytes;
    // batches of R consecutive rows, dealt to the groups of the whole grid
    const int64_t per_round = (int64_t)gridDim.x * sh.groups;
    const int64_t first = (int64_t)blockIdx.x * sh.groups + g;
    const int64_t rounds = ((p.rows + R - 1) / R + per_round - 1) / per_round;  // the same for every group
    int fill_stage = 0;
    auto fill = [&](int64_t round) {
        const int64_t r0 = (first + round * per_round) * R;
        char* dst = ring + fill_stage * stage_bytes;
        if (++fill_stage == sh.stages) fill_stage = 0;
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (r0 + k < p.rows) ring_fill<T, NCH, CE, A>(dst + k * row_bytes, x + (r0 + k) * p.x_stride, L);
        ring_commit();
    };
    for (int i = 0; i < sh.stages - 1; ++i) fill(i);
    int stage = 0;
    for (int64_t round = 0; round < rounds; ++round) {
        ring_turn(sh.stages, round, fill);
        const char* src = ring + stage * stage_bytes;
        if (++stage == sh.stages) stage = 0;
        const int64_t r0 = (first + round * per_round) * R;

        float mean[R], rstd[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            u64 s = 0;
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                if (!has_chunk<A>(j, L)) continue;
                u64 v[CE / 2];
                ring_read<T, CE, A>(v, src + k * row_bytes, j, L);
#pragma unroll
                for (int i = 0; i < CE / 2; ++i) s = add2(s, v[i]);
            }
            mean[k] = f2lo(s) + f2hi(s);
        }
        sums(mean);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            mean[k] *= inv_d;
            const u64 m = f2(mean[k], mean[k]);
            u64 q = 0;
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                if (!has_chunk<A>(j, L)) continue;
                u64 v[CE / 2];
                ring_read<T, CE, A>(v, src + k * row_bytes, j, L);
#pragma unroll
                for (int i = 0; i < CE / 2; ++i) {
                    const u64 c = mask_pair<CE, A>(sub2(v[i], m), j, i, L);
                    q = fma2(c, c, q);
                }
            }
            rstd[k] = f2lo(q) + f2hi(q);
        }
        sums(rstd);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            rstd[k] = 1.0f / sqrtf(rstd[k] * inv_d + p.eps);
            const u64 m = f2(mean[k], mean[k]), rs = f2(rstd[k], rstd[k]);
            if (r0 + k >= p.rows) continue;
            T* dst = out + (r0 + k) * p.out_stride;
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                if (!has_chunk<A>(j, L)) continue;
                u64 v[CE / 2];
                ring_read<T, CE, A>(v, src + k * row_bytes, j, L);
#pragma unroll
                for (int i = 0; i < CE / 2; ++i)
                    v[i] = fma2(mul2(sub2(v[i], m), rs), w[j * (CE / 2) + i], b[j * (CE / 2) + i]);
                put_chunk<T, CE, A>(dst, v, j, L);
            }
        }
    }
}

template <class T, int NCH, Access A, int R>
static cudaError_t ln_fwd(const LnFwdParams& p, int tpr, cudaStream_t s) {
    auto k = layer_norm_kernel<T, NCH, A, R>;
    const RingShape sh = ring_shape(tpr, kRowBytesPerThread<T, NCH, ChunkOf<T>::CE> * tpr, R, 0);
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.allow(reinterpret_cast<const void*>(k), sh)) return e;
    const int64_t batches = (p.rows + R - 1) / R, need = (batches + sh.groups - 1) / sh.groups;
    const int64_t most = (int64_t)sm_count() * sh.ctas_per_sm;
    return launch_pdl(k, (unsigned)(need < most ? need : most), sh.groups * tpr, sh.smem, s, p, sh);
}

template <class T, int NCH>
static cudaError_t ln_fwd_r(const LnFwdParams& p, bool vec, cudaStream_t s) {
    const int tpr = row_threads(p.D);
    // two rows a round while every SM has several
    const bool two = p.rows >= 8 * (int64_t)sm_count();
    if (!vec) return ln_fwd<T, NCH, kScalar, 1>(p, tpr, s);
    return two ? ln_fwd<T, NCH, kVec, 2>(p, tpr, s) : ln_fwd<T, NCH, kVec, 1>(p, tpr, s);
}

cudaError_t launch_layer_norm(const LnFwdParams& p, bool f32, bool vec, cudaStream_t s) {
    return f32 ? ln_fwd_r<float, 4>(p, vec, s) : ln_fwd_r<uint16_t, 2>(p, vec, s);
}

}  // namespace mbx
