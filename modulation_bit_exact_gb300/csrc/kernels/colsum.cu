// colsum.cu -- the second step of the parameter gradients: the parts' partial
// sums (binary32, [segments][parts][nacc][D]) joined in part order, and the
// split of rows into parts.
#include "rowgroup.cuh"

namespace mbx {

RowShape row_shape(int D, int esize) {
    const int ce = 16 / esize;
    RowShape s;
    s.epl = D <= 256 ? 8 : 16;
    const int lanes = (D + s.epl - 1) / s.epl;  // threads that own a full share
    s.tpr = (lanes + 31) / 32 * 32;
    (void)ce;
    s.groups = s.tpr >= 256 ? 1 : 256 / s.tpr;
    return s;
}

GradPlan grad_plan(int64_t rows, int64_t mod_rows, const RowShape& sh) {
    const int64_t seq = rows / mod_rows;
    GradPlan g;
    g.groups = seq >= 2 * sh.groups ? sh.groups : 1;
    const int64_t target = (int64_t)sm_count() * (sh.block() <= 320 ? 2 : 1);
    int64_t parts = (target + mod_rows - 1) / mod_rows;
    const int64_t most = (seq + 2 * g.groups - 1) / (2 * g.groups);  // two rows a group at least
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    g.rows_per_part = (seq + parts - 1) / parts;
    g.parts = (seq + g.rows_per_part - 1) / g.rows_per_part;
    return g;
}

int64_t grad_workspace_bytes(int64_t rows, int64_t mod_rows, int D, int esize) {
    if (rows == mod_rows) return 0;
    const GradPlan g = grad_plan(rows, mod_rows, row_shape(D, esize));
    return g.parts == 1 ? 0 : mod_rows * g.parts * 2 * D * (int64_t)sizeof(float);
}

constexpr int kColTile = 32, kColLanes = 8;

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
#pragma unroll 4
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
