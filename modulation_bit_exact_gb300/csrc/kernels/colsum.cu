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

RingShape grad_shape(int D, int esize, int rows, bool vec) {
    const int tpr = row_threads(D);
    return ring_shape(tpr, staged_row_bytes(tpr, esize, vec), rows, 0, 64, kGradThreads, 1);
}

GradPlan grad_plan(int64_t rows, int64_t mod_rows, int D, int esize) {
    const int64_t seq = rows / mod_rows;
    const RingShape sh = grad_shape(D, esize, 2, true);
    const int64_t round = sh.groups;  // rows of a block's round
    GradPlan g;
    // Few rounds: one block, and no second kernel.  D = 1024, two segments, a
    // round takes 1.06 us of the block: at four rounds 8.4 us on the device
    // against 6.7 of two kernels, but 9.7 against 13.4 for a call on its own.
    if (seq <= 4 * sh.groups) {
        g.parts = 1;
        g.rows_per_part = seq;
        return g;
    }
    int64_t parts = ((int64_t)sm_count() * sh.ctas_per_sm + mod_rows - 1) / mod_rows;
    if (parts > (seq + round - 1) / round) parts = (seq + round - 1) / round;
    g.rows_per_part = ((seq + parts - 1) / parts + round - 1) / round * round;
    g.parts = (seq + g.rows_per_part - 1) / g.rows_per_part;
    return g;
}

int64_t grad_workspace_bytes(int64_t rows, int64_t mod_rows, int D, int esize) {
    if (rows == mod_rows) return 0;
    const GradPlan g = grad_plan(rows, mod_rows, D, esize);
    return g.parts == 1 ? 0 : mod_rows * g.parts * 2 * D * (int64_t)sizeof(float);
}

// A block adds 8*W columns: 8 threads side by side hold W columns each, 32
// rows of such threads take every 32nd part, with up to eight loads of each in
// flight, and the 32 sums are added in shared memory in a fixed order.  The
// parts' sums are 2 to 10 MB that the first kernel has just written, so they
// come from L2; latency bounds this kernel, not bandwidth.
constexpr int kColThreads = 8, kColLanes = 32;

template <int W>
__global__ void __launch_bounds__(kColThreads* kColLanes) column_sums_kernel(ColSumParams p) {
    __shared__ float part[kColLanes][kColThreads * W];
    grid_dep_wait();
    grid_dep_launch();
    const int cols = p.nacc * p.D;
    const int c0 = (blockIdx.x * kColThreads + threadIdx.x) * W;
    const int64_t seg = blockIdx.y;
    const float* w = p.ws + seg * p.parts * cols + c0;
    float s[W] = {};
    if (c0 < cols) {
#pragma unroll 8
        for (int64_t i = threadIdx.y; i < p.parts; i += kColLanes) {
            if constexpr (W == 4) {
                const float4 v = *reinterpret_cast<const float4*>(w + i * cols);
                s[0] += v.x;
                s[1] += v.y;
                s[2] += v.z;
                s[3] += v.w;
            } else {
                s[0] += w[i * cols];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) part[threadIdx.y][threadIdx.x * W + i] = s[i];
    __syncthreads();
    const int t = threadIdx.y * kColThreads + threadIdx.x, c = blockIdx.x * kColThreads * W + t;
    if (t >= kColThreads * W || c >= cols) return;
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < kColLanes; ++i) a += part[i][t];
    const int k = c / p.D, d = c - k * p.D;
    if (!p.out[k]) return;
    const int64_t o = seg * p.out_stride[k] + d;
    if (p.p_f32) store_elem(static_cast<float*>(p.out[k]) + o, a);
    else store_elem(static_cast<uint16_t*>(p.out[k]) + o, a);
}

cudaError_t launch_column_sums(const ColSumParams& p, cudaStream_t s) {
    if (t_dry_run) return cudaSuccess;
    const int cols = p.nacc * p.D;
    const bool wide = cols % 4 == 0;  // 16-byte loads (the workspace is 16-byte aligned)
    const int tile = kColThreads * (wide ? 4 : 1);
    cudaLaunchConfig_t cfg = {};
    // more than one part a segment: no more segments than blocks on the device
    cfg.gridDim = dim3((cols + tile - 1) / tile, (unsigned)p.segments);
    cfg.blockDim = dim3(kColThreads, kColLanes);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, wide ? column_sums_kernel<4> : column_sums_kernel<1>, p);
    const cudaError_t last = cudaGetLastError();
    return e != cudaSuccess ? e : last;
}

}  // namespace mbx
