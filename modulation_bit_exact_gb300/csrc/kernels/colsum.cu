// colsum.cu -- the second step of the parameter gradients: the parts' partial
// sums (binary32, [segments][parts][nacc][D]) joined in part order, and the
// split of rows into parts.
#include "rowgroup.cuh"

namespace mbx {

RingShape ring_shape(int tpr, int row_bytes, int rows, int extra_bytes, int fixed_per_thread, int threads_per_sm,
                     int blocks_per_sm) {
    RingShape s;
    s.tpr = tpr;
    s.row_bytes = row_bytes;
    s.extra_bytes = extra_bytes;
    s.groups = threads_per_sm / blocks_per_sm / tpr;
    if (s.groups < 1) s.groups = 1;
    while (s.groups * tpr % 32) --s.groups;  // whole warps
    s.sums_bytes = tpr > 32 ? s.groups * 2 * 4 * 16 * (int)sizeof(float) : 0;
    s.fixed_bytes = fixed_per_thread * s.groups * tpr;
    const int stage = (rows * row_bytes + extra_bytes) * s.groups;
    // as many blocks as the threads allow, if two stages fit for each
    for (s.ctas_per_sm = threads_per_sm / (s.groups * tpr);; --s.ctas_per_sm) {
        const int room = 228 * 1024 / s.ctas_per_sm - 1024 - s.sums_bytes - s.fixed_bytes;  // 1 KB of each block's is the system's
        s.stages = room / stage;
        if (s.stages >= 2 || s.ctas_per_sm == 1) break;
    }
    if (s.stages > 4) s.stages = 4;
    s.group_bytes = s.stages * (rows * row_bytes + extra_bytes);
    s.smem = s.sums_bytes + s.fixed_bytes + s.groups * s.group_bytes;
    return s;
}

cudaError_t SmemOptIn::allow(const void* kernel, const RingShape& sh) {
    if (sh.stages < 1) return cudaErrorInvalidConfiguration;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (allowed[dev].load(std::memory_order_acquire) >= sh.smem) return cudaSuccess;
    int most = 0;
    if (cudaError_t e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) return e;
    if (sh.smem > most) return cudaErrorInvalidConfiguration;
    // the limit itself: another thread may ask for more at the same time
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) return e;
    allowed[dev].store(most, std::memory_order_release);
    return cudaSuccess;
}

GradPlan grad_plan(int64_t rows, int64_t mod_rows, int D, int esize) {
    const int64_t seq = rows / mod_rows;
    // the shape of a block that streams aligned rows of two operands, 16 elements a
    // thread.  Some are launched with more row groups (layernorm_bwd.cu: up to 64
    // columns, and 4104 to 5120); their last round of a part may be half empty.
    const int tpr = row_threads(D);
    const RingShape sh = ring_shape(tpr, staged_row_bytes(tpr, esize, true), 2, 0, 64, kGradThreads, 1);
    const int64_t round = sh.groups;  // rows of a block's round
    const int64_t slots = (int64_t)sm_count() * sh.ctas_per_sm;
    // One part, which needs no second kernel, or as many as fill the device once,
    // twice, ...: the cost in half rounds (a round takes a block 1.1 to 1.3 us) of
    // the rounds, of each block's start and end (3.5 rounds), of the second kernel
    // (4.5) and of the parts' sums, written and read.  bfloat16 gradients of AdaLN,
    // us: 64 segments of 128 rows of 4096: one part 85, two 53, three (the device
    // once and a quarter) 71; 150 of 128: one 87, two 107; 4 of 256: one 162, 32 15.
    GradPlan g{1, seq};
    int64_t best = INT64_MAX;
    auto consider = [&](int64_t parts) {
        const int64_t per = ((seq + parts - 1) / parts + round - 1) / round;  // rounds of a part
        parts = (seq + per * round - 1) / (per * round);
        const int64_t cost = (mod_rows * parts + slots - 1) / slots * (2 * per + 7) +
                             (parts > 1 ? 9 + mod_rows * parts * D / 250000 : 0);
        if (cost < best) {
            best = cost;
            g = parts == 1 ? GradPlan{1, seq} : GradPlan{parts, per * round};
        }
    };
    consider(1);
    const int64_t fewest = (mod_rows + slots - 1) / slots;
    for (int64_t times = fewest; times < fewest + 4; ++times)
        if (times * slots / mod_rows > 1) consider(times * slots / mod_rows);
    return g;
}

int64_t grad_workspace_bytes(int64_t rows, int64_t mod_rows, int D, int esize) {
    if (rows == mod_rows) return 0;
    const GradPlan g = grad_plan(rows, mod_rows, D, esize);
    return g.parts == 1 ? 0 : mod_rows * g.parts * 2 * D * (int64_t)sizeof(float);
}

// A block of 256 threads: 256 / LANES threads side by side hold W columns each,
// LANES rows of such threads take every LANES-th part, with up to kColAtOnce loads
// of each in flight, and the lanes' sums are added in shared memory in a fixed
// order.  The parts' sums are 2 to 10 MB that the first kernel has just written,
// so they come from L2; latency bounds this kernel, not bandwidth: it adds 4.2 us
// to the first kernel's 49 for [8704, 4096] bfloat16 into two rows.  With 4 lanes
// for up to 40 parts, 64 segments of 10 rows of 4096 in 3 parts take 20 us, with 32
// lanes 48; 76 parts take 57 and 53.
constexpr int kColBlock = 256, kColAtOnce = 5, kFewParts = 40;

template <int W, int LANES>
__global__ void __launch_bounds__(kColBlock) column_sums_kernel(ColSumParams p) {
    constexpr int kThreads = kColBlock / LANES;
    __shared__ float part[LANES][kThreads * W];
    grid_dep_wait();
    grid_dep_launch();
    const int cols = p.nacc * p.D;
    const int c0 = (blockIdx.x * kThreads + threadIdx.x) * W;
    const int64_t seg = blockIdx.y;
    const float* w = p.ws + seg * p.parts * cols + c0;
    float s[W] = {};
    if (c0 < cols) {
        for (int64_t i = threadIdx.y; i < p.parts; i += kColAtOnce * LANES) {
            float v[kColAtOnce][W];
#pragma unroll
            for (int u = 0; u < kColAtOnce; ++u) {
                const int64_t k = i + u * LANES;
                if constexpr (W == 4) {
                    const float4 q = k < p.parts ? *reinterpret_cast<const float4*>(w + k * cols) : make_float4(0, 0, 0, 0);
                    v[u][0] = q.x, v[u][1] = q.y, v[u][2] = q.z, v[u][3] = q.w;
                } else {
                    v[u][0] = k < p.parts ? w[k * cols] : 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < kColAtOnce; ++u)
#pragma unroll
                for (int j = 0; j < W; ++j) s[j] += v[u][j];
        }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) part[threadIdx.y][threadIdx.x * W + i] = s[i];
    __syncthreads();
    for (int t = threadIdx.y * kThreads + threadIdx.x; t < kThreads * W; t += kColBlock) {
        const int c = blockIdx.x * kThreads * W + t;
        if (c >= cols) break;
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < LANES; ++i) a += part[i][t];
        const int k = c / p.D, d = c - k * p.D;
        if (!p.out[k]) continue;
        const int64_t o = seg * p.out_stride[k] + d;
        if (p.p_f32) store_elem(static_cast<float*>(p.out[k]) + o, a);
        else store_elem(static_cast<uint16_t*>(p.out[k]) + o, a);
    }
}

template <int W, int LANES>
static cudaError_t column_sums(const ColSumParams& p, cudaStream_t s) {
    constexpr int kThreads = kColBlock / LANES, tile = kThreads * W;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.nacc * p.D + tile - 1) / tile, (unsigned)p.segments);
    cfg.blockDim = dim3(kThreads, LANES);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, column_sums_kernel<W, LANES>, p);
    const cudaError_t last = cudaGetLastError();
    return e != cudaSuccess ? e : last;
}

cudaError_t launch_column_sums(const ColSumParams& p, cudaStream_t s) {
    // gridDim.y is the segment.  grad_plan() makes two parts of a segment at least, out
    // of at most three blocks an SM more than there are segments, so the segments that
    // come here are at most four times the SMs.
    if (p.segments > 65535) return cudaErrorInvalidConfiguration;
    if (t_dry_run) return cudaSuccess;
    const bool wide = p.nacc * p.D % 4 == 0;  // 16-byte loads (the workspace is 16-byte aligned)
    if (p.parts <= kFewParts) return wide ? column_sums<4, 4>(p, s) : column_sums<1, 4>(p, s);
    return wide ? column_sums<4, 32>(p, s) : column_sums<1, 32>(p, s);
}

}  // namespace mbx
