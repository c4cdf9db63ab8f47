// linear_nvfp4.cu -- out = a(x) W^T / gs + bias for a few rows x and a weight in
// NVFP4: E2M1 values in pairs, one E4M3 scale for 16 of them in tiles of 128 rows
// x 4 blocks, and a global scale gs; a is the identity or SiLU.
//
// A warp makes kCols output columns of kRows rows: a lane takes a block of 16
// weights of each column and multiplies it with the rows' activations, which the
// thread block keeps in shared memory, a piece of K at a time.  binary32 sums: 16
// products of a block, times the block's scale, then over the lane's blocks and
// the lanes.  For weights that linear_tc.cu does not take (rows that start at no 8-byte
// boundary, scales at no 16-byte one: slices of larger buffers): bound by
// decoding, [1, 5120] x [30720, 5120] 176 us against 17.8 there.
#include "linear.cuh"

namespace mbx {

constexpr int kLinWarps = 8, kLinCols = 4, kLinRows = 4;
constexpr int kPieceBlocks = 64;  // blocks of 16 in a piece of K

template <class T, class O>
__global__ void __launch_bounds__(32 * kLinWarps) linear_nvfp4_kernel(LinearParams p, int wide) {
    __shared__ float act[kLinRows][16][kPieceBlocks];  // by place in the block, so that lanes read side by side
    const int lane = threadIdx.x % 32;
    const int64_t n0 = ((int64_t)blockIdx.x * kLinWarps + threadIdx.x / 32) * kLinCols;
    const int row0 = blockIdx.y * kLinRows, rows = min(p.rows - row0, kLinRows), blocks = p.K / 16;
    grid_dep_wait();
    grid_dep_launch();
    float sum[kLinCols][kLinRows] = {};
    for (int b0 = 0; b0 < blocks; b0 += kPieceBlocks) {
        const int nb = min(blocks - b0, kPieceBlocks);
        __syncthreads();
        for (int i = threadIdx.x; i < kLinRows * nb * 16; i += blockDim.x) {
            const int r = i / (nb * 16), k = i - r * nb * 16;
            float v = 0.0f;
            if (r < rows) v = load_elem(static_cast<const T*>(p.x) + (int64_t)(row0 + r) * p.x_stride + b0 * 16 + k);
            act[r][k % 16][k / 16] = p.silu ? silu(v) : v;
        }
        __syncthreads();
        for (int b = lane; b < nb; b += 32) {
#pragma unroll 1
            for (int c = 0; c < kLinCols; ++c) {
                const int64_t n = n0 + c;
                if (n >= p.N) break;
                const int blk = b0 + b;
                const uint8_t* w = p.w4 + n * p.w_stride + blk * 8;
                uint32_t q[2];
                if (wide) {
                    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(q[0]), "=r"(q[1]) : "l"(w));
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) q[i] = w[4 * i] | w[4 * i + 1] << 8 | w[4 * i + 2] << 16 | (uint32_t)w[4 * i + 3] << 24;
                }
                const float s = e4m3_value(p.sf[(n / 128 * p.sf_col_tiles + blk / 4) * 512 + n % 32 * 16 + n % 128 / 32 * 4 + blk % 4]);
                float part[kLinRows] = {};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float f[8];
                    e2m1x8(f, q[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int r = 0; r < kLinRows; ++r) part[r] = __fmaf_rn(f[j], act[r][8 * i + j][b], part[r]);
                }
#pragma unroll
                for (int cc = 0; cc < kLinCols; ++cc)
                    if (cc == c) {
#pragma unroll
                        for (int r = 0; r < kLinRows; ++r) sum[cc][r] = __fmaf_rn(s, part[r], sum[cc][r]);
                    }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < kLinCols; ++c)
#pragma unroll
        for (int r = 0; r < kLinRows; ++r) {
            float v = sum[c][r];
            for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
            const int64_t n = n0 + c;
            if (lane == 0 && n < p.N && r < rows) {
                v /= *p.gs;
                if (p.bias) v += p.bias_f32 ? load_elem(static_cast<const float*>(p.bias) + n)
                                            : load_elem(static_cast<const uint16_t*>(p.bias) + n);
                store_elem(static_cast<O*>(p.out) + (int64_t)(row0 + r) * p.out_stride + n, v);
            }
        }
}

template <class T, class O>
static cudaError_t linear_rows(const LinearParams& p, cudaStream_t s) {
    const int wide = reinterpret_cast<uintptr_t>(p.w4) % 8 == 0 && p.w_stride % 8 == 0;
    const dim3 grid((unsigned)((p.N + kLinWarps * kLinCols - 1) / (kLinWarps * kLinCols)), (p.rows + kLinRows - 1) / kLinRows);
    return launch_pdl_2d(linear_nvfp4_kernel<T, O>, grid, 32 * kLinWarps, 0, s, p, wide);
}

cudaError_t launch_linear_nvfp4(const LinearParams& p, bool x_f32, bool out_f32, cudaStream_t s) {
    if (linear_tc_takes(p)) return launch_linear_tc(p, x_f32, out_f32, s);
    return x_f32 ? linear_rows<float, float>(p, s) : out_f32 ? linear_rows<uint16_t, float>(p, s) : linear_rows<uint16_t, uint16_t>(p, s);
}

}  // namespace mbx
