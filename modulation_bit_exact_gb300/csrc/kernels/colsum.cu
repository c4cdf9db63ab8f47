// colsum.cu -- the second step of the parameter gradients: the parts' partial
// sums (binary32, [segments][parts][nacc][D]) joined in part order, and the
// split of rows into parts.
#include "rowgroup.cuh"

namespace mbx {

RingShape ring_shape(int tpr, int row_bytes, int rows, int extra_bytes, int fixed_per_thread, int threads_per_sm) {
    RingShape s;
    s.tpr = tpr;
    s.row_bytes = row_bytes;
    s.extra_bytes = extra_bytes;
    s.groups = 2 * tpr > threads_per_sm ? 1 : threads_per_sm / 2 / tpr;  // two blocks an SM
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

RingShape grad_shape(int D, int esize, int rows) {
    const int tpr = row_threads(D);
    return ring_shape(tpr, 16 * esize * tpr, rows, 0, 64, kGradThreads);
}

GradPlan grad_plan(int64_t rows, int64_t mod_rows, int D, int esize) {
    const int64_t seq = rows / mod_rows;
    const RingShape sh = grad_shape(D, esize, 2);
    const int64_t round = (int64_t)sh.groups * 2;  // whole rounds of a block, which takes one or two rows a group
    GradPlan g;
    if (seq <= 4 * sh.groups) {  // few rounds: one block, and no second kernel
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

constexpr int kColTile = 32, kColLanes = 32;

__global__ void __launch_bounds__(kColTile* kColLanes) column_sums_kernel(ColSumParams p) {
    __shared__ float part[kColLanes][kColTile];
    grid_dep_wait();
    grid_dep_launch();
    const int cols = p.nacc * p.D;
    const int c = blockIdx.x * kColTile + threadIdx.x;
    for (int64_t seg = blockIdx.y; seg < p.segments; seg += gridDim.y) {
        const float* w = p.ws + seg * p.parts * cols;
        float s = 0.0f;
        if (c < cols) {
#pragma unroll 8
            for (int64_t i = threadIdx.y; i < p.parts; i += kColLanes) s += w[i * cols + c];
        }
        part[threadIdx.y][threadIdx.x] = s;
        __syncthreads();
        if (threadIdx.y == 0 && c < cols) {
#pragma unroll
            for (int i = 1; i < kColLanes; ++i) s += part[i][threadIdx.x];
            const int k = c / p.D, d = c - k * p.D;
            if (p.out[k]) {
                const int64_t o = seg * p.out_stride[k] + d;
                if (p.p_f32) store_elem(static_cast<float*>(p.out[k]) + o, s);
                else store_elem(static_cast<uint16_t*>(p.out[k]) + o, s);
            }
        }
        __syncthreads();
    }
}

cudaError_t launch_column_sums(const ColSumParams& p, cudaStream_t s) {
    if (t_dry_run) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.nacc * p.D + kColTile - 1) / kColTile, (unsigned)(p.segments < 65535 ? p.segments : 65535));
    cfg.blockDim = dim3(kColTile, kColLanes);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, column_sums_kernel, p);
    const cudaError_t last = cudaGetLastError();
    return e != cudaSuccess ? e : last;
}

}  // namespace mbx
