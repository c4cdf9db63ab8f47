// layernorm_bwd.cu -- the gradients of LayerNorm with a factor and a shift:
// the affine weight and bias (layernorm.cu), or AdaLN's 1 + scale and shift
// with one row of each for a sample or for a token.
//
//   mean, rstd of the row, xh = (x - mean) * rstd (layernorm.cu)
//   gy = dy * f;  c1 = mean(gy);  c2 = mean(gy * xh)
//   dx = rstd * (gy - c1 - xh * c2)  (+ the residual stream's gradient)
//   df = sum over the factor's rows of dy * xh;  db = sum of dy
//
// The statistics come from x again, not from saved ones: x is here for xh
// anyway, sum(x) travels with sum(gy) and sum((x-mean)^2) with
// sum(gy*(x-mean)), so it costs one more row sum and no memory, and a forward
// pass need not save anything.
#include "lnorm.cuh"

namespace mbx {

// The two row sums of R staged rows: mean, rstd, and the two coefficients of
//   dx = rstd*gy + k1 + xh*k2,   k1 = -rstd*c1, k2 = -rstd*c2.
// factor(k, j, f) gives chunk j of row k's factor.
template <class T, int NCH, Access A, int R, class Factor>
__device__ __forceinline__ void ln_row_sums(float (&mean)[R], float (&rstd)[R], float (&k1)[R], float (&k2)[R],
                                            const char* sx, const char* sdy, int row_bytes, const Lane& L,
                                            const LnBwdParams& p, float inv_d, GroupSums& sums, Factor factor) {
    constexpr int CE = ChunkOf<T>::CE;
    float v[2 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        u64 s = 0, sg = 0;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (!has_chunk<A>(j, L)) continue;
            u64 x[CE / 2], dy[CE / 2], f[CE / 2];
            ring_read<T, CE, A>(x, sx + k * row_bytes, j, L);
            ring_read<T, CE, A>(dy, sdy + k * row_bytes, j, L);
            factor(k, j, f);
#pragma unroll
            for (int i = 0; i < CE / 2; ++i) {
                s = add2(s, x[i]);
                sg = fma2(dy[i], f[i], sg);
            }
        }
        v[2 * k] = f2lo(s) + f2hi(s);
        v[2 * k + 1] = f2lo(sg) + f2hi(sg);
    }
    sums(v);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        mean[k] = v[2 * k] * inv_d;
        k1[k] = v[2 * k + 1] * inv_d;
        const u64 m = f2(mean[k], mean[k]);
        u64 q = 0, qg = 0;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (!has_chunk<A>(j, L)) continue;
            u64 x[CE / 2], dy[CE / 2], f[CE / 2];
            ring_read<T, CE, A>(x, sx + k * row_bytes, j, L);
            ring_read<T, CE, A>(dy, sdy + k * row_bytes, j, L);
            factor(k, j, f);
#pragma unroll
            for (int i = 0; i < CE / 2; ++i) {
                const u64 c = mask_pair<CE, A>(sub2(x[i], m), j, i, L);
                q = fma2(c, c, q);
                qg = fma2(mul2(dy[i], f[i]), c, qg);
            }
        }
        v[2 * k] = f2lo(q) + f2hi(q);
        v[2 * k + 1] = f2lo(qg) + f2hi(qg);
    }
    sums(v);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        rstd[k] = 1.0f / sqrtf(v[2 * k] * inv_d + p.eps);
        k1[k] *= -rstd[k];
        k2[k] = -rstd[k] * (v[2 * k + 1] * inv_d * rstd[k]);
    }
}

// One modulation row for every row: nothing is summed, every output is a row,
// and the factor's row streams with x and dy.
template <class T, int NCH, Access A, bool RES>
__global__ void __launch_bounds__(kRingThreads) ln_backward_token_kernel(LnBwdParams p, RingShape sh) {
    constexpr int CE = ChunkOf<T>::CE;
    extern __shared__ __align__(16) char smem[];
    const int tpr = sh.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const Lane L = make_lane<CE, A>(t, tpr, p.D);
    GroupSums sums = group_sums(smem, sh, g, t);
    char* ring = smem + sh.sums_bytes + g * sh.group_bytes;
    const float inv_d = 1.0f / (float)p.D;
    grid_dep_wait();
    grid_dep_launch();
    const T* px = static_cast<const T*>(p.x);
    const T* pd = static_cast<const T*>(p.dout);
    const int row_bytes = sh.row_bytes, stage_bytes = (RES ? 3 : 2) * row_bytes + sh.extra_bytes;
    constexpr int kF = RES ? 3 : 2;  // the factor's row comes last
    const int64_t per_round = (int64_t)gridDim.x * sh.groups, first = (int64_t)blockIdx.x * sh.groups + g;
    const int64_t rounds = (p.rows + per_round - 1) / per_round;
    const u64 one = f2(p.factor_add, p.factor_add);
    int fill_stage = 0;
    auto fill = [&](int64_t round) {
        const int64_t r = first + round * per_round;
        char* dst = ring + fill_stage * stage_bytes;
        if (++fill_stage == sh.stages) fill_stage = 0;
        if (r < p.rows) {
            ring_fill<T, NCH, CE, A>(dst, px + r * p.x_stride, L);
            ring_fill<T, NCH, CE, A>(dst + row_bytes, pd + r * p.dout_stride, L);
            if constexpr (RES)
                ring_fill<T, NCH, CE, A>(dst + 2 * row_bytes, static_cast<const T*>(p.dres) + r * p.dres_stride, L);
            if (sizeof(T) == 4 || p.p_f32)
                ring_fill<float, NCH, CE, A>(dst + kF * row_bytes, static_cast<const float*>(p.factor) + r * p.factor_stride, L);
            else
                ring_fill<uint16_t, NCH, CE, A>(dst + kF * row_bytes, static_cast<const uint16_t*>(p.factor) + r * p.factor_stride, L);
        }
        ring_commit();
    };
    for (int i = 0; i < sh.stages - 1; ++i) fill(i);
    int stage = 0;
    for (int64_t round = 0; round < rounds; ++round) {
        ring_turn(sh.stages, round, fill);
        const char* src = ring + stage * stage_bytes;
        if (++stage == sh.stages) stage = 0;
        const int64_t r = first + round * per_round;
        auto factor = [&](int, int j, u64 (&f)[CE / 2]) {
            if (sizeof(T) == 4 || p.p_f32) ring_read<float, CE, A>(f, src + kF * row_bytes, j, L);
            else ring_read<uint16_t, CE, A>(f, src + kF * row_bytes, j, L);
#pragma unroll
            for (int i = 0; i < CE / 2; ++i) f[i] = add2(f[i], one);
        };
        float mean[1], rstd[1], k1[1], k2[1];
        ln_row_sums<T, NCH, A, 1>(mean, rstd, k1, k2, src, src + row_bytes, row_bytes, L, p, inv_d, sums, factor);
        if (r >= p.rows) continue;
        const u64 m = f2(mean[0], mean[0]), rs = f2(rstd[0], rstd[0]), a = f2(k1[0], k1[0]), b = f2(k2[0], k2[0]);
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (!has_chunk<A>(j, L)) continue;
            u64 x[CE / 2], dy[CE / 2], f[CE / 2], res[CE / 2];
            if constexpr (RES) ring_read<T, CE, A>(res, src + 2 * row_bytes, j, L);
            ring_read<T, CE, A>(x, src, j, L);
            ring_read<T, CE, A>(dy, src + row_bytes, j, L);
            factor(0, j, f);
#pragma unroll
            for (int i = 0; i < CE / 2; ++i) {
                x[i] = mul2(sub2(x[i], m), rs);
                f[i] = fma2(x[i], b, fma2(mul2(dy[i], f[i]), rs, a));
                if constexpr (RES) f[i] = add2(f[i], res[i]);
                x[i] = mul2(x[i], dy[i]);
            }
            put_chunk<T, CE, A>(static_cast<T*>(p.dx) + r * p.dx_stride, f, j, L);
            if (p.dfactor) put_param_chunk<T, CE, A>(p.dfactor, r * p.dfactor_stride, p.p_f32, x, j, L);
            if (p.dshift) put_param_chunk<T, CE, A>(p.dshift, r * p.dshift_stride, p.p_f32, dy, j, L);
        }
    }
}

// Modulation rows shared by seq rows: a block takes one part of a segment, its
// row groups batches of R rows of the part in turn; every thread sums its own
// columns in binary32 registers, the groups are added in shared memory, and
// the part's sums go to the workspace (or out, when the segment is one part).
template <class T, int NCH, Access A, int R, bool RES>
__global__ void __launch_bounds__(kRingThreads) ln_backward_kernel(LnBwdParams p, RingShape sh) {
    constexpr int CE = ChunkOf<T>::CE, E = NCH * CE;
    extern __shared__ __align__(16) char smem[];
    const int tpr = sh.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr, groups = sh.groups;
    const Lane L = make_lane<CE, A>(t, tpr, p.D);
    GroupSums sums = group_sums(smem, sh, g, t);
    char* ring = smem + sh.sums_bytes + g * sh.group_bytes;
    const float inv_d = 1.0f / (float)p.D;
    grid_dep_wait();
    grid_dep_launch();
    const T* px = static_cast<const T*>(p.x);
    const T* pd = static_cast<const T*>(p.dout);
    const int row_bytes = sh.row_bytes, stage_bytes = (RES ? 3 : 2) * R * row_bytes;
    const int64_t units = p.mod_rows * p.plan.parts;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t seg = unit / p.plan.parts, part = unit - seg * p.plan.parts;
        const int64_t r0 = seg * p.seq + part * p.plan.rows_per_part;
        int64_t r1 = r0 + p.plan.rows_per_part;
        if (r1 > (seg + 1) * p.seq) r1 = (seg + 1) * p.seq;
        const int64_t per_round = (int64_t)groups * R, rounds = (r1 - r0 + per_round - 1) / per_round;
        u64 f[E / 2], adf[E / 2], ads[E / 2];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            u64 c[CE / 2];
#pragma unroll
            for (int i = 0; i < CE / 2; ++i) c[i] = f2(1.0f, 1.0f);
            if (p.factor) get_param_chunk<T, CE, A>(c, p.factor, seg * p.factor_stride, p.p_f32, j, L);
#pragma unroll
            for (int i = 0; i < CE / 2; ++i) {
                f[j * (CE / 2) + i] = add2(c[i], f2(p.factor_add, p.factor_add));
                adf[j * (CE / 2) + i] = ads[j * (CE / 2) + i] = 0;
            }
        }
        int fill_stage = 0;
        auto fill = [&](int64_t round) {
            const int64_t r = r0 + round * per_round + g * R;
            char* dst = ring + fill_stage * stage_bytes;
            if (++fill_stage == sh.stages) fill_stage = 0;
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (r + k < r1) {
                    ring_fill<T, NCH, CE, A>(dst + k * row_bytes, px + (r + k) * p.x_stride, L);
                    ring_fill<T, NCH, CE, A>(dst + (R + k) * row_bytes, pd + (r + k) * p.dout_stride, L);
                    if constexpr (RES)
                        ring_fill<T, NCH, CE, A>(dst + (2 * R + k) * row_bytes,
                                                 static_cast<const T*>(p.dres) + (r + k) * p.dres_stride, L);
                }
            ring_commit();
        };
        auto factor = [&](int, int j, u64 (&c)[CE / 2]) {
#pragma unroll
            for (int i = 0; i < CE / 2; ++i) c[i] = f[j * (CE / 2) + i];
        };
        for (int i = 0; i < sh.stages - 1; ++i) fill(i);
        int stage = 0;
        for (int64_t round = 0; round < rounds; ++round) {
            ring_turn(sh.stages, round, fill);
            const char* src = ring + stage * stage_bytes;
            if (++stage == sh.stages) stage = 0;
            const int64_t r = r0 + round * per_round + g * R;
            float mean[R], rstd[R], k1[R], k2[R];
            ln_row_sums<T, NCH, A, R>(mean, rstd, k1, k2, src, src + R * row_bytes, row_bytes, L, p, inv_d, sums, factor);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (r + k >= r1) continue;
                const u64 m = f2(mean[k], mean[k]), rs = f2(rstd[k], rstd[k]), a = f2(k1[k], k1[k]), b = f2(k2[k], k2[k]);
#pragma unroll
                for (int j = 0; j < NCH; ++j) {
                    if (!has_chunk<A>(j, L)) continue;
                    u64 x[CE / 2], dy[CE / 2], dx[CE / 2], res[CE / 2];
                    if constexpr (RES) ring_read<T, CE, A>(res, src + (2 * R + k) * row_bytes, j, L);
                    ring_read<T, CE, A>(x, src + k * row_bytes, j, L);
                    ring_read<T, CE, A>(dy, src + (R + k) * row_bytes, j, L);
#pragma unroll
                    for (int i = 0; i < CE / 2; ++i) {
                        const int e = j * (CE / 2) + i;
                        const u64 xh = mask_pair<CE, A>(mul2(sub2(x[i], m), rs), j, i, L);
                        dx[i] = fma2(xh, b, fma2(mul2(dy[i], f[e]), rs, a));
                        if constexpr (RES) dx[i] = add2(dx[i], res[i]);
                        adf[e] = fma2(xh, dy[i], adf[e]);
                        ads[e] = add2(ads[e], dy[i]);
                    }
                    put_chunk<T, CE, A>(static_cast<T*>(p.dx) + (r + k) * p.dx_stride, dx, j, L);
                }
            }
        }
        if (p.dfactor == nullptr && p.dshift == nullptr) continue;
        if (groups > 1) {
            // every group's sums in shared memory (the ring is drained: every
            // thread waited for its last rows), added in group order
            u64* acc = reinterpret_cast<u64*>(smem + sh.sums_bytes);  // [E][block]
            const int n = groups * tpr;
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                acc[e * n + threadIdx.x] = adf[e];
                acc[(E / 2 + e) * n + threadIdx.x] = ads[e];
            }
            __syncthreads();
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    for (int k = 1; k < groups; ++k) {
                        adf[e] = add2(adf[e], acc[e * n + k * tpr + t]);
                        ads[e] = add2(ads[e], acc[(E / 2 + e) * n + k * tpr + t]);
                    }
            }
            __syncthreads();
        }
        if (g == 0) {
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                if (!has_chunk<A>(j, L)) continue;
                u64 c[2][CE / 2];
#pragma unroll
                for (int i = 0; i < CE / 2; ++i) {
                    c[0][i] = adf[j * (CE / 2) + i];
                    c[1][i] = ads[j * (CE / 2) + i];
                }
                if (p.plan.parts == 1) {
                    if (p.dfactor) put_param_chunk<T, CE, A>(p.dfactor, seg * p.dfactor_stride, p.p_f32, c[0], j, L);
                    if (p.dshift) put_param_chunk<T, CE, A>(p.dshift, seg * p.dshift_stride, p.p_f32, c[1], j, L);
                } else {
                    put_chunk<float, CE, A>(p.ws + unit * 2 * p.D, c[0], j, L);
                    put_chunk<float, CE, A>(p.ws + (unit * 2 + 1) * p.D, c[1], j, L);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- launch

template <class T, int NCH, Access A, bool RES>
static cudaError_t ln_bwd_token(const LnBwdParams& p, cudaStream_t s) {
    auto k = ln_backward_token_kernel<T, NCH, A, RES>;
    const int tpr = row_threads(p.D), elem = p.p_f32 ? 4 : 2;
    const RingShape sh = ring_shape(tpr, 16 * (int)sizeof(T) * tpr, RES ? 3 : 2, 16 * elem * tpr);
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.allow(reinterpret_cast<const void*>(k), sh)) return e;
    const int64_t need = (p.rows + sh.groups - 1) / sh.groups, most = (int64_t)sm_count() * sh.ctas_per_sm;
    return launch_pdl(k, (unsigned)(need < most ? need : most), sh.groups * tpr, sh.smem, s, p, sh);
}

template <class T, int NCH, Access A, int R, bool RES>
static cudaError_t ln_bwd_sum(const LnBwdParams& p, const RingShape& sh, cudaStream_t s) {
    auto k = ln_backward_kernel<T, NCH, A, R, RES>;
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.allow(reinterpret_cast<const void*>(k), sh)) return e;
    const int64_t units = p.mod_rows * p.plan.parts, most = 1 << 30;
    return launch_pdl(k, (unsigned)(units < most ? units : most), sh.groups * sh.tpr, sh.smem, s, p, sh);
}

template <class T, int NCH, Access A, bool RES>
static cudaError_t ln_bwd(const LnBwdParams& p0, cudaStream_t s) {
    LnBwdParams p = p0;
    if (p.seq == 1 && p.factor) return ln_bwd_token<T, NCH, A, RES>(p, s);
    p.plan = grad_plan(p.rows, p.mod_rows, p.D, (int)sizeof(T));
    const RingShape one = grad_shape(p.D, (int)sizeof(T), RES ? 3 : 2), two = grad_shape(p.D, (int)sizeof(T), RES ? 6 : 4);
    cudaError_t e;
    // two rows a round where two stages of them fit in as many blocks
    if constexpr (A == kVec) {
        if (two.stages >= 2 && two.ctas_per_sm == one.ctas_per_sm) e = ln_bwd_sum<T, NCH, A, 2, RES>(p, two, s);
        else e = ln_bwd_sum<T, NCH, A, 1, RES>(p, one, s);
    } else {
        e = ln_bwd_sum<T, NCH, A, 1, RES>(p, one, s);
    }
    if (e != cudaSuccess || p.plan.parts == 1 || (!p.dfactor && !p.dshift)) return e;
    ColSumParams c{p.ws, p.plan.parts, p.mod_rows, p.D, 2, {p.dfactor, p.dshift}, {p.dfactor_stride, p.dshift_stride}, p.p_f32};
    return launch_column_sums(c, s);
}

template <class T, int NCH>
static cudaError_t ln_bwd_any(const LnBwdParams& p, bool vec, cudaStream_t s) {
    if (vec) return p.dres ? ln_bwd<T, NCH, kVec, true>(p, s) : ln_bwd<T, NCH, kVec, false>(p, s);
    return p.dres ? ln_bwd<T, NCH, kScalar, true>(p, s) : ln_bwd<T, NCH, kScalar, false>(p, s);
}

cudaError_t launch_ln_backward(const LnBwdParams& p, bool f32, bool vec, cudaStream_t s) {
    return launch_all_or_none([&] {
        return f32 ? ln_bwd_any<float, 4>(p, vec, s) : ln_bwd_any<uint16_t, 2>(p, vec, s);
    });
}

}  // namespace mbx
