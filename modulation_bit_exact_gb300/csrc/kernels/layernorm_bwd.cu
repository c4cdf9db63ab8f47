// layernorm_bwd.cu -- the gradients of LayerNorm with a factor and a shift:
// the affine weight and bias (layernorm.cu), or AdaLN's 1 + scale and shift
// with one row of each for a sample or for a token.
//
//   mean, rstd of the row, xh = (x - mean) * rstd (layernorm.cu)
//   gy = dy * f;  c1 = mean(gy);  c2 = mean(gy * xh)
//   dx = rstd * (gy - c1 - xh * c2)  (+ the residual stream's gradient)
//   df = sum over the factor's rows of dy * xh;  db = sum of dy
//
// gy is a rounded product in every kernel here: it is formed as a fused
// multiply-add of a -0 that the compiler does not know, since ptxas would fuse a
// packed product with the sum it goes into, in one kernel and not in another.
//
// The statistics come from x again, not from saved ones: x is here for xh
// anyway, sum(x) travels with sum(gy) and sum((x-mean)^2) with
// sum(gy*(x-mean)), so it costs one more row sum and no memory, and a forward
// pass need not save anything.
//
// Bound by memory where rows are many: x and dy are read once and dx is written
// once (a token's factor and its two gradients once each).  [65536, 1024]
// bfloat16 into one row: 69 us, 5.8 TB/s; [32760, 5120] a row each: 347 us, 5.8
// TB/s of 6.77 that a copy reaches.  With few rows a segment it is bound by a
// row's two dependent sums and by the second kernel: [8704, 4096] into two rows,
// 55 us.
#include "lnorm.cuh"

namespace mbx {

// One row in registers, x as pairs; gy(e) gives pair e of dy * f, and next_pass()
// runs after each of the two sums.  On return x holds xh; the result are the
// coefficients of dx = rstd*gy + k1 + xh*k2,   k1 = -rstd*c1, k2 = -rstd*c2.
struct RowCoef {
    float rstd, k1, k2;
};
template <class T, int NCH, Access A, class Gy, class NextPass>
__device__ __forceinline__ RowCoef ln_row_stats(u64 (&x)[NCH * ChunkOf<T>::CE / 2], const Lane& L, float inv_d,
                                                float eps, GroupSums& sums, Gy gy, NextPass next_pass) {
    constexpr int CE = ChunkOf<T>::CE, H = CE / 2;
    constexpr bool kSum = kSumDeviations<T>;
    u64 s[2] = {0, 0}, sg[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < NCH * H; ++e) {
        s[e % 2] = add2(s[e % 2], x[e]);
        sg[e % 2] = add2(sg[e % 2], gy(e));
    }
    s[0] = add2(s[0], s[1]);
    sg[0] = add2(sg[0], sg[1]);
    float v[2] = {f2lo(s[0]) + f2hi(s[0]), f2lo(sg[0]) + f2hi(sg[0])};
    sums(v);
    next_pass();
    const float mean = v[0] * inv_d, c1 = v[1] * inv_d, rest = kSum ? 0.0f : mean_rest(v[0], L.D, inv_d);
    u64 q[2] = {0, 0}, qg[2] = {0, 0}, d = 0;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int e = j * H + i;
            x[e] = sub2(x[e], where_column<CE, A>(mean, j, i, L));
            if constexpr (!kSum) x[e] = sub2(x[e], where_column<CE, A>(rest, j, i, L));
            q[e % 2] = fma2(x[e], x[e], q[e % 2]);
            qg[e % 2] = fma2(gy(e), x[e], qg[e % 2]);
            if constexpr (kSum) d = add2(d, x[e]);
        }
    }
    q[0] = add2(q[0], q[1]);
    qg[0] = add2(qg[0], qg[1]);
    float w[kSum ? 4 : 2] = {f2lo(q[0]) + f2hi(q[0]), f2lo(qg[0]) + f2hi(qg[0])};
    if constexpr (kSum) w[2] = f2lo(d) + f2hi(d);
    sums(w);
    next_pass();
    float rstd, m = w[1] * inv_d;  // m: mean(gy * (x - mean))
    if constexpr (kSum) {
        const float delta = w[2] * inv_d;
        rstd = rstd_of(w[0] * inv_d, delta, eps);
        const u64 rs = f2(rstd, rstd), nd = f2(-delta * rstd, -delta * rstd);
#pragma unroll
        for (int e = 0; e < NCH * H; ++e) x[e] = fma2(x[e], rs, nd);
        m = fmaf(-delta, c1, m);
    } else {
        rstd = rsqrtf(w[0] * inv_d + eps);
        const u64 rs = f2(rstd, rstd);
#pragma unroll
        for (int e = 0; e < NCH * H; ++e) x[e] = mul2(x[e], rs);
    }
    return RowCoef{rstd, -rstd * c1, -rstd * (m * rstd)};
}

// One modulation row for every row: nothing is summed, every output is a row,
// and the factor's row streams with x and dy.
template <class T, int NCH, Access A, bool RES>
__global__ void __launch_bounds__(kRingThreads) ln_backward_token_kernel(LnBwdParams p, RingShape sh) {
    constexpr int CE = ChunkOf<T>::CE, H = CE / 2;
    constexpr int kF = RES ? 3 : 2;  // a stage: x, dy, the residual's gradient, the factor
    extern __shared__ __align__(16) char smem[];
    const int tpr = sh.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const Lane L = make_lane<CE>(t, tpr, p.D, g + 1);
    GroupSums sums = group_sums(smem, sh, g, t);
    char* ring = smem + sh.sums_bytes + sh.fixed_bytes + g * sh.group_bytes;
    const float inv_d = 1.0f / (float)p.D;
    const int64_t step = (int64_t)gridDim.x * sh.groups, first = (int64_t)blockIdx.x * sh.groups + g;
    if (first < p.rows) {
        prefetch_row<T, A>(static_cast<const T*>(p.x) + first * p.x_stride, p.D, t);
        prefetch_row<T, A>(static_cast<const T*>(p.dout) + first * p.dout_stride, p.D, t);
    }
    grid_dep_wait();
    grid_dep_launch();
    const int row_bytes = sh.row_bytes, stage_bytes = kF * row_bytes + sh.extra_bytes;
    const int64_t rounds = (p.rows + step - 1) / step;  // the same for every group
    const u64 one = f2(p.factor_add, p.factor_add), nz = f2(p.neg_zero, p.neg_zero);
    int64_t fill_row = first;
    for (int i = 0; i < sh.stages; ++i) {
        char* dst = ring + i * stage_bytes;
        for (int o = 0; o < kF; ++o) ring_clear<T, NCH, CE, A>(dst + o * row_bytes, L);
        if (sizeof(T) == 4 || p.p_f32) ring_clear<float, NCH, CE, A>(dst + kF * row_bytes, L);
        else ring_clear<uint16_t, NCH, CE, A>(dst + kF * row_bytes, L);
    }
    auto fill = [&](int st) {
        char* dst = ring + st * stage_bytes;
        if (fill_row < p.rows) {
            ring_fill<T, NCH, CE, A>(dst, static_cast<const T*>(p.x) + fill_row * p.x_stride, L);
            ring_fill<T, NCH, CE, A>(dst + row_bytes, static_cast<const T*>(p.dout) + fill_row * p.dout_stride, L);
            if constexpr (RES)
                ring_fill<T, NCH, CE, A>(dst + 2 * row_bytes, static_cast<const T*>(p.dres) + fill_row * p.dres_stride, L);
            const int64_t f0 = fill_row * p.factor_stride;
            if (sizeof(T) == 4 || p.p_f32)
                ring_fill<float, NCH, CE, A>(dst + kF * row_bytes, static_cast<const float*>(p.factor) + f0, L);
            else ring_fill<uint16_t, NCH, CE, A>(dst + kF * row_bytes, static_cast<const uint16_t*>(p.factor) + f0, L);
        } else if constexpr (A == kShift) {
            for (int o = 0; o <= kF; ++o) ring_clear<T, NCH, CE, A>(dst + o * row_bytes, L);
        }
        fill_row += step;
        ring_commit();
    };
    for (int i = 0; i < sh.stages; ++i) fill(i);
    int stage = 0;
    int64_t r = first;
    for (int64_t round = 0; round < rounds; ++round, r += step) {
        ring_wait(sh.stages);
        if constexpr (A == kShift) group_sync(L);
        const char* src = ring + stage * stage_bytes;
        u64 x[NCH * H], dy[NCH * H], gy[NCH * H];
        read_row<T, NCH, CE, A>(x, src, L);
        read_row<T, NCH, CE, A>(dy, src + row_bytes, L);
        if (sizeof(T) == 4 || p.p_f32) read_row<float, NCH, CE, A>(gy, src + kF * row_bytes, L);
        else read_row<uint16_t, NCH, CE, A>(gy, src + kF * row_bytes, L);
        uint4 res[RES ? NCH : 1];
        if constexpr (RES) read_pieces<T, NCH, A>(res, src + 2 * row_bytes, L);
        if constexpr (A == kVec) fill(stage);
#pragma unroll
        for (int e = 0; e < NCH * H; ++e) gy[e] = fma2(dy[e], add2(gy[e], one), nz);
        const RowCoef k = ln_row_stats<T, NCH, A>(x, L, inv_d, p.eps, sums, [&](int e) { return gy[e]; }, [] {});
        if (r < p.rows) {
            const u64 rs = f2(k.rstd, k.rstd), a = f2(k.k1, k.k1), b = f2(k.k2, k.k2);
            T* dx_row = static_cast<T*>(p.dx) + r * p.dx_stride;
            char* out = ring + stage * stage_bytes;  // kShift: x and dy have been read
            const int64_t f_row = r * p.dfactor_stride, s_row = r * p.dshift_stride;
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                u64 dx[H], xd[H], d[H];
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int e = j * H + i;
                    dx[i] = fma2(x[e], b, fma2(gy[e], rs, a));
                    if constexpr (RES) dx[i] = add2(dx[i], piece_pair<T>(res, e));
                    xd[i] = mul2(x[e], dy[e]);
                    d[i] = dy[e];
                }
                // three rows out for three in: streamed stores, 351.6 -> 341.3 us at
                // [32760, 5120] bfloat16 (binary32 [32760, 2048]: 255 -> 257)
                put_row_chunk<T, CE, A, true>(dx_row, out, dx, j, L);
                if constexpr (A == kVec) {
                    if (p.dfactor) put_param_row_chunk<T, CE, A, true>(p.dfactor, f_row, p.p_f32, nullptr, xd, j, L);
                    if (p.dshift) put_param_row_chunk<T, CE, A, true>(p.dshift, s_row, p.p_f32, nullptr, d, j, L);
                }
            }
            if constexpr (A == kShift) {
                flush_row(dx_row, out, L);
#pragma unroll 1
                for (int which = 0; which < 2; ++which) {  // the stage holds one row at a time
                    void* to = which ? p.dshift : p.dfactor;
                    if (!to) continue;
                    const int64_t off = which ? s_row : f_row;
#pragma unroll
                    for (int j = 0; j < NCH; ++j) {
                        u64 v[H];
#pragma unroll
                        for (int i = 0; i < H; ++i) v[i] = which ? dy[j * H + i] : mul2(x[j * H + i], dy[j * H + i]);
                        put_param_row_chunk<T, CE, A>(to, off, p.p_f32, out, v, j, L);
                    }
                    flush_param_row<T>(to, off, p.p_f32, out, L);
                }
            }
        } else if constexpr (A == kShift) {
            group_sync(L);  // every thread has read the stage
        }
        if constexpr (A == kShift) fill(stage);
        if (++stage == sh.stages) stage = 0;
    }
}

// Modulation rows shared by seq rows: a block takes one part of a segment, its
// row groups the rows of the part in turn; every thread sums its own columns
// in binary32 registers, the groups are added in shared memory, and the part's
// sums go to the workspace (or out, when the segment is one part).
//
// A row's two sums are latency, so an SM wants two rows in work at least.  LEAN:
// dy * f is formed anew in each pass and the residual's gradient read last, so
// that more threads fit on an SM than kGradThreads.
template <class T, int NCH, Access A, bool RES, int THREADS>
__global__ void __launch_bounds__(THREADS) ln_backward_kernel(LnBwdParams p, RingShape sh) {
    constexpr int CE = ChunkOf<T>::CE, H = CE / 2, P = NCH * H;
    constexpr bool LEAN = THREADS > kGradThreads;
    extern __shared__ __align__(16) char smem[];
    const int tpr = sh.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr, groups = sh.groups;
    const Lane L = make_lane<CE>(t, tpr, p.D, g + 1);
    GroupSums sums = group_sums(smem, sh, g, t);
    // the factor lives in shared memory, each thread's own copy, so that x, dy
    // and the two sums of every column fit in registers
    ulonglong2* fs = reinterpret_cast<ulonglong2*>(smem + sh.sums_bytes) + threadIdx.x;  // [P/2][block]
    char* ring = smem + sh.sums_bytes + sh.fixed_bytes + g * sh.group_bytes;
    const int block = groups * tpr;
    const float inv_d = 1.0f / (float)p.D;
    const int64_t units = p.mod_rows * p.plan.parts;
    {
        const int64_t seg = blockIdx.x / p.plan.parts, r = seg * p.seq + (blockIdx.x - seg * p.plan.parts) * p.plan.rows_per_part + g;
        if (r < p.rows) {
            prefetch_row<T, A>(static_cast<const T*>(p.x) + r * p.x_stride, p.D, t);
            prefetch_row<T, A>(static_cast<const T*>(p.dout) + r * p.dout_stride, p.D, t);
        }
    }
    grid_dep_wait();
    grid_dep_launch();
    const int row_bytes = sh.row_bytes, stage_bytes = (RES ? 3 : 2) * row_bytes;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t seg = unit / p.plan.parts, part = unit - seg * p.plan.parts;
        const int64_t r0 = seg * p.seq + part * p.plan.rows_per_part;
        const int64_t left = (seg + 1) * p.seq - r0;
        const int n_rows = (int)(left < p.plan.rows_per_part ? left : p.plan.rows_per_part);
        const int rounds = (n_rows + groups - 1) / groups;
        const T* nx = static_cast<const T*>(p.x) + (r0 + g) * p.x_stride;
        const T* nd = static_cast<const T*>(p.dout) + (r0 + g) * p.dout_stride;
        const T* nr = RES ? static_cast<const T*>(p.dres) + (r0 + g) * p.dres_stride : nullptr;
        T* dx_row = static_cast<T*>(p.dx) + (r0 + g) * p.dx_stride;
        for (int i = 0; i < sh.stages * (RES ? 3 : 2); ++i) ring_clear<T, NCH, CE, A>(ring + i * row_bytes, L);
        int fill_row = g;
        const int64_t x_step = groups * p.x_stride, d_step = groups * p.dout_stride,
                      r_step = groups * p.dres_stride, dx_step = groups * p.dx_stride;
        auto fill = [&](int st) {
            char* dst = ring + st * stage_bytes;
            if (fill_row < n_rows) {
                ring_fill<T, NCH, CE, A>(dst, nx, L);
                ring_fill<T, NCH, CE, A>(dst + row_bytes, nd, L);
                if constexpr (RES) ring_fill<T, NCH, CE, A>(dst + 2 * row_bytes, nr, L);
            } else if constexpr (A == kShift) {
                for (int o = 0; o < (RES ? 3 : 2); ++o) ring_clear<T, NCH, CE, A>(dst + o * row_bytes, L);
            }
            fill_row += groups;
            nx += x_step;
            nd += d_step;
            if constexpr (RES) nr += r_step;
            ring_commit();
        };
        for (int i = 0; i < sh.stages; ++i) fill(i);
        u64 adf[P], ads[P];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            u64 c[H];
#pragma unroll
            for (int i = 0; i < H; ++i) c[i] = f2(1.0f, 1.0f);
            if (p.factor) get_param_chunk<T, CE, A>(c, p.factor, seg * p.factor_stride, p.p_f32, j, L);
#pragma unroll
            for (int i = 0; i < H; i += 2) {
                const u64 one = f2(p.factor_add, p.factor_add);
                fs[(j * H + i) / 2 * block] = make_ulonglong2(add2(c[i], one), add2(c[i + 1], one));
                adf[j * H + i] = adf[j * H + i + 1] = ads[j * H + i] = ads[j * H + i + 1] = 0;
            }
        }
        const u64 nz = f2(p.neg_zero, p.neg_zero);
        constexpr bool kFillLast = A == kShift || (LEAN && RES);  // the stage is read, or written, to the end
        int stage = 0;
        for (int round = 0; round < rounds; ++round, dx_row += dx_step) {
            ring_wait(sh.stages);
            if constexpr (A == kShift) group_sync(L);
            const char* src = ring + stage * stage_bytes;
            u64 x[P], dy[P], gy[LEAN ? 1 : P];
            uint4 res[RES ? NCH : 1];
            read_row<T, NCH, CE, A>(x, src, L);
            read_row<T, NCH, CE, A>(dy, src + row_bytes, L);
            if constexpr (RES && !LEAN) read_pieces<T, NCH, A>(res, src + 2 * row_bytes, L);
            if constexpr (!kFillLast) fill(stage);
            auto times_factor = [&](int e) {
                const ulonglong2 f = fs[e / 2 * block];
                return fma2(dy[e], e % 2 ? f.y : f.x, nz);
            };
            if constexpr (!LEAN) {
#pragma unroll
                for (int e = 0; e < P; ++e) gy[e] = times_factor(e);
            }
            auto gy_at = [&](int e) {
                if constexpr (LEAN) return times_factor(e);
                else return gy[e];
            };
            const RowCoef c = ln_row_stats<T, NCH, A>(x, L, inv_d, p.eps, sums, gy_at, [] {
                if constexpr (LEAN) asm volatile("" ::: "memory");  // the factor is read again
            });
            if (round * groups + g < n_rows) {
                const u64 rs = f2(c.rstd, c.rstd), a = f2(c.k1, c.k1), b = f2(c.k2, c.k2);
                char* out = ring + stage * stage_bytes;  // kShift: x and dy have been read
                if constexpr (RES && LEAN) read_pieces<T, NCH, A>(res, src + 2 * row_bytes, L);
#pragma unroll
                for (int j = 0; j < NCH; ++j) {
                    u64 dx[H];
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const int e = j * H + i;
                        dx[i] = fma2(x[e], b, fma2(gy_at(e), rs, a));
                        if constexpr (RES) dx[i] = add2(dx[i], piece_pair<T>(res, e));
                        adf[e] = fma2(x[e], dy[e], adf[e]);
                        ads[e] = add2(ads[e], dy[e]);
                    }
                    put_row_chunk<T, CE, A>(dx_row, out, dx, j, L);
                }
                if constexpr (A == kShift) flush_row(dx_row, out, L);
            } else if constexpr (A == kShift) {
                group_sync(L);  // every thread has read the stage
            }
            if constexpr (kFillLast) fill(stage);
            if (++stage == sh.stages) stage = 0;
        }
        if (p.dfactor == nullptr && p.dshift == nullptr) continue;
        if (groups > 1) {
            // every group's sums in shared memory, in the place of the ring (drained:
            // every thread waited for its last rows), added in group order.  They take
            // 8 bytes for each element of a row; a stage's two rows or three hold 4
            // bytes at least in bfloat16, where there are two stages at least, and 8 in
            // binary32, where there may be one
            u64* acc = reinterpret_cast<u64*>(smem + sh.sums_bytes + sh.fixed_bytes);  // [2P][block]
            const int n = block;
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
#pragma unroll
            for (int e = 0; e < P; ++e) {
                acc[e * n + threadIdx.x] = adf[e];
                acc[(P + e) * n + threadIdx.x] = ads[e];
            }
            __syncthreads();
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < P; ++e)
                    for (int k = 1; k < groups; ++k) {
                        adf[e] = add2(adf[e], acc[e * n + k * tpr + t]);
                        ads[e] = add2(ads[e], acc[(P + e) * n + k * tpr + t]);
                    }
            }
            __syncthreads();
        }
        if (g == 0) {
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                if (j >= L.nv) continue;
                u64 c[2][H];
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    c[0][i] = adf[j * H + i];
                    c[1][i] = ads[j * H + i];
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
    const RingShape sh = ring_shape(tpr, staged_row_bytes(tpr, (int)sizeof(T), A == kVec), RES ? 3 : 2, staged_row_bytes(tpr, elem, A == kVec), 0, kRingThreads, 2);
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.allow(reinterpret_cast<const void*>(k), sh)) return e;
    const int64_t need = (p.rows + sh.groups - 1) / sh.groups, most = (int64_t)sm_count() * sh.ctas_per_sm;
    return launch_pdl(k, (unsigned)(need < most ? need : most), sh.groups * tpr, sh.smem, s, p, sh);
}

template <class T, int NCH, Access A, bool RES, int THREADS>
static cudaError_t ln_bwd_sums(const LnBwdParams& p, cudaStream_t s) {
    auto k = ln_backward_kernel<T, NCH, A, RES, THREADS>;
    constexpr int per = NCH * ChunkOf<T>::CE;
    const int tpr = row_threads(p.D, per);
    const RingShape sh = ring_shape(tpr, staged_row_bytes(tpr, (int)sizeof(T), A == kVec, per), RES ? 3 : 2, 0, 4 * per, THREADS, 1);
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.allow(reinterpret_cast<const void*>(k), sh)) return e;
    const int64_t units = p.mod_rows * p.plan.parts, most = 1 << 30;
    return launch_pdl(k, (unsigned)(units < most ? units : most), sh.groups * sh.tpr, sh.smem, s, p, sh);
}

template <class T, int NCH, Access A, bool RES>
static cudaError_t ln_bwd_rows(const LnBwdParams& p, cudaStream_t s) {
    // 8 elements a thread in place of 16 where half of eight lanes' 16 would hold no
    // column: us, 8 / 16, bfloat16 1M rows of 40 70 / 100, 600000 of 64 48 / 66;
    // binary32 98 / 124, 83 / 82.  The columns lie with the same lanes either way, so
    // a row's sums, and its bits, are those of ln_bwd_token().  Up to 128 columns 8
    // elements would take 16 lanes and another order, for little: bfloat16 312496 rows
    // of 128 46.7 / 46.1, 62496 16.3 / 17.1, 600000 of 72 80 / 69.  kShift the same (in
    // the registers of 512 threads), so that a row's bits do not depend on where it
    // starts.
    if (p.D <= 64) return ln_bwd_sums<T, NCH / 2, A, RES, A == kVec ? 1024 : kGradThreads>(p, s);
    if constexpr (sizeof(T) == 2 && A == kVec) {
        // The widths of which two rows fit in 640 threads but not in 512.  160M
        // elements, us, LEAN / not: D = 4608 224 / 277, 5120 212 / 253, with a
        // residual 250 / 297 and 241 / 273.  One row fits either way at D = 6144
        // and 8192 (221, 204 not LEAN), and two at 4096 (174).
        if (p.D > 4096 && p.D <= 5120) return ln_bwd_sums<T, NCH, A, RES, kRingThreads>(p, s);
    }
    return ln_bwd_sums<T, NCH, A, RES, kGradThreads>(p, s);
}

template <class T, int NCH, Access A, bool RES>
static cudaError_t ln_bwd(const LnBwdParams& p0, cudaStream_t s) {
    LnBwdParams p = p0;
    if (p.seq == 1 && p.factor) return ln_bwd_token<T, NCH, A, RES>(p, s);
    p.plan = grad_plan(p.rows, p.mod_rows, p.D, (int)sizeof(T));
    const cudaError_t e = ln_bwd_rows<T, NCH, A, RES>(p, s);
    if (e != cudaSuccess || p.plan.parts == 1 || (!p.dfactor && !p.dshift)) return e;
    ColSumParams c{p.ws, p.plan.parts, p.mod_rows, p.D, 2, {p.dfactor, p.dshift}, {p.dfactor_stride, p.dshift_stride}, p.p_f32};
    return launch_column_sums(c, s);
}

template <class T, int NCH>
static cudaError_t ln_bwd_any(const LnBwdParams& p, bool vec, cudaStream_t s) {
    if (vec) return p.dres ? ln_bwd<T, NCH, kVec, true>(p, s) : ln_bwd<T, NCH, kVec, false>(p, s);
    return p.dres ? ln_bwd<T, NCH, kShift, true>(p, s) : ln_bwd<T, NCH, kShift, false>(p, s);
}

cudaError_t launch_ln_backward(const LnBwdParams& p, bool f32, bool vec, cudaStream_t s) {
    return launch_all_or_none([&] {
        return f32 ? ln_bwd_any<float, 4>(p, vec, s) : ln_bwd_any<uint16_t, 2>(p, vec, s);
    });
}

}  // namespace mbx
