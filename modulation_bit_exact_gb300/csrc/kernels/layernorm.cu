// layernorm.cu -- affine LayerNorm.
//
//   mean, var over the row (biased); rstd = 1/sqrt(var + eps);
//   xh = (x - mean) * rstd;  y = xh * weight + bias
//
// binary32 with one rounding at the output.  The variance is the mean of the
// squared deviations of registers that hold the whole row (no E[x^2] - mean^2), and
// what the rounded mean is off by is taken out of the deviations (lnorm.cuh), so
// that a row far from zero loses nothing.
//
// Bound by memory: a row is read once and written once.  A row's two sums depend
// on each other, so what hides them is rows in flight: the ring of rowring.cuh,
// filled again as soon as a row is in registers, and two rows a round where an
// SM has few groups.  [32760, 5120] bfloat16: 108 us, 6.2 TB/s of 6.77 that a
// copy reaches; [77, 1024]: 2.9 us in a graph, a launch's latency.
#include "lnorm.cuh"

namespace mbx {

// R rows of a group at a time: their sums share the shuffles and the barrier.
template <class T, int NCH, Access A, int R>
__global__ void __launch_bounds__(kRingThreads) layer_norm_kernel(LnFwdParams p, RingShape sh) {
    constexpr int CE = ChunkOf<T>::CE, P = NCH * CE / 2;
    extern __shared__ __align__(16) char smem[];
    const int tpr = sh.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const Lane L = make_lane<CE>(t, tpr, p.D, g + 1);
    GroupSums sums = group_sums(smem, sh, g, t);
    char* ring = smem + sh.sums_bytes + sh.fixed_bytes + g * sh.group_bytes;
    const float inv_d = 1.0f / (float)p.D;
    // batches of R consecutive rows, dealt to the groups of the whole grid
    const int64_t step = (int64_t)gridDim.x * sh.groups * R;
    const int64_t rounds = (p.rows + step - 1) / step;  // the same for every group
    int64_t r = ((int64_t)blockIdx.x * sh.groups + g) * R, fill_row = r;
#pragma unroll
    for (int k = 0; k < R; ++k)
        if (r + k < p.rows) prefetch_row<T, A>(static_cast<const T*>(p.x) + (r + k) * p.x_stride, p.D, t);
    grid_dep_wait();  // launched programmatically: the previous kernel has finished
    grid_dep_launch();

    u64 w[P], b[P];
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

    const int row_bytes = sh.row_bytes, stage_bytes = R * row_bytes;
    auto fill = [&](int st) {
        char* dst = ring + st * stage_bytes;
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (fill_row + k < p.rows)
                ring_fill<T, NCH, CE, A>(dst + k * row_bytes, static_cast<const T*>(p.x) + (fill_row + k) * p.x_stride, L);
            else if constexpr (A == kShift) ring_clear<T, NCH, CE, A>(dst + k * row_bytes, L);
        fill_row += step;
        ring_commit();
    };
    for (int i = 0; i < sh.stages * R; ++i) ring_clear<T, NCH, CE, A>(ring + i * row_bytes, L);
    for (int i = 0; i < sh.stages; ++i) fill(i);
    int stage = 0;
    for (int64_t round = 0; round < rounds; ++round, r += step) {
        ring_wait(sh.stages);
        if constexpr (A == kShift) group_sync(L);
        u64 v[R][P];
        constexpr bool kSum = kSumDeviations<T>;
        float total[R], delta[R], second[kSum ? 2 * R : R];  // the squares' sums, the deviations'
#pragma unroll
        for (int k = 0; k < R; ++k) read_row<T, NCH, CE, A>(v[k], ring + stage * stage_bytes + k * row_bytes, L);
        if constexpr (A == kVec) fill(stage);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            u64 s = 0;
#pragma unroll
            for (int e = 0; e < P; ++e) s = add2(s, v[k][e]);
            total[k] = f2lo(s) + f2hi(s);
        }
        sums(total);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const float mean = total[k] * inv_d;
            delta[k] = mean_rest(total[k], p.D, inv_d);
            u64 q = 0, d = 0;
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
#pragma unroll
                for (int i = 0; i < CE / 2; ++i) {
                    u64& c = v[k][j * (CE / 2) + i];
                    c = sub2(c, where_column<CE, A>(mean, j, i, L));
                    q = fma2(c, c, q);
                    if constexpr (kSum) d = add2(d, c);
                }
            }
            second[k] = f2lo(q) + f2hi(q);
            if constexpr (kSum) second[R + k] = f2lo(d) + f2hi(d);
        }
        sums(second);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (r + k >= p.rows) continue;
            if constexpr (kSum) delta[k] = second[R + k] * inv_d;
            const float rs1 = rstd_of(second[k] * inv_d, delta[k], p.eps);
            const u64 rs = f2(rs1, rs1), nd = f2(-delta[k] * rs1, -delta[k] * rs1);
            T* dst = static_cast<T*>(p.out) + (r + k) * p.out_stride;
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                u64 c[CE / 2];
#pragma unroll
                for (int i = 0; i < CE / 2; ++i) {
                    const int e = j * (CE / 2) + i;
                    c[i] = fma2(fma2(v[k][e], rs, nd), w[e], b[e]);
                }
                put_row_chunk<T, CE, A>(dst, ring + stage * stage_bytes + k * row_bytes, c, j, L);
            }
            if constexpr (A == kShift) flush_row(dst, ring + stage * stage_bytes + k * row_bytes, L);
        }
        if constexpr (A == kShift) fill(stage);
        if (++stage == sh.stages) stage = 0;
    }
}

template <class T, int NCH, Access A, int R>
static cudaError_t ln_fwd(const LnFwdParams& p, int tpr, cudaStream_t s) {
    auto k = layer_norm_kernel<T, NCH, A, R>;
    const RingShape sh = ring_shape(tpr, staged_row_bytes(tpr, (int)sizeof(T), A == kVec, NCH * ChunkOf<T>::CE), R, 0, 0, kRingThreads, 2);
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.allow(reinterpret_cast<const void*>(k), sh)) return e;
    const int64_t batches = (p.rows + R - 1) / R, need = (batches + sh.groups - 1) / sh.groups;
    const int64_t most = (int64_t)sm_count() * sh.ctas_per_sm;
    return launch_pdl(k, (unsigned)(need < most ? need : most), sh.groups * tpr, sh.smem, s, p, sh);
}

template <class T, int NCH>
static cudaError_t ln_fwd_r(const LnFwdParams& p, bool vec, cudaStream_t s) {
    if constexpr (sizeof(T) == 2) {
        // 8 elements a thread in place of 16 where half of eight lanes would hold none:
        // bfloat16, us, 8 / 16, 125000 rows of 64 8.3 / 9.4, 625000 31 to 37 / 36, 1562496
        // 70 / 82, 1M rows of 40 47 / 55; binary32 gains nothing (625000 of 64 61 / 57).
        // kShift the same, so that a row's bits do not depend on where it starts.
        if (p.D <= 64) {
            const int tpr = row_threads(p.D, 8);
            return vec ? ln_fwd<T, NCH / 2, kVec, 1>(p, tpr, s) : ln_fwd<T, NCH / 2, kShift, 1>(p, tpr, s);
        }
    }
    const int tpr = row_threads(p.D);
    if (!vec) return ln_fwd<T, NCH, kShift, 1>(p, tpr, s);
    // Two rows a round where an SM has fewer than four row groups, so that a row's
    // sums are latency, and several rows for each.  bfloat16, us, two / one, 160M
    // elements: D = 1024 119 / 114, 2048 115 / 102, 2560 115 / 103, 3584 110 / 131,
    // 5120 104 / 116, 8192 112 / 128; 5120 columns of 304 rows 3.5 / 3.2, of 608
    // 4.1 / 4.2, of 1216 5.9 / 6.4.  binary32 rows arrive in twice the time: 40M
    // elements of 1024 55.5 / 55.5, of 2048 57.5 / 55.1, of 8192 54.7 / 55.3.
    if constexpr (sizeof(T) == 2)
        if (kRingThreads / tpr < 4 && p.rows >= 4 * (int64_t)sm_count()) return ln_fwd<T, NCH, kVec, 2>(p, tpr, s);
    return ln_fwd<T, NCH, kVec, 1>(p, tpr, s);
}

cudaError_t launch_layer_norm(const LnFwdParams& p, bool f32, bool vec, cudaStream_t s) {
    return f32 ? ln_fwd_r<float, 4>(p, vec, s) : ln_fwd_r<uint16_t, 2>(p, vec, s);
}

}  // namespace mbx
