// linear.cuh -- the launch, the activation and the decoding of NVFP4 shared by the products
// (linear_tc.cu, linear_nvfp4.cu).
#pragma once

#include "linear.h"
#include "rowgroup.cuh"

namespace mbx {

// launch_pdl of a grid of two dimensions.
template <class... KArgs, class... Args>
inline cudaError_t launch_pdl_2d(void (*k)(KArgs...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, const Args&... args) {
    if (t_dry_run) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
    const cudaError_t last = cudaGetLastError();
    return e != cudaSuccess ? e : last;
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// Eight E2M1 codes of a word, the lowest first.
__device__ __forceinline__ void e2m1x8(float (&f)[8], uint32_t w) {
    uint32_t h[4];
    asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\ncvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n.reg .f16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}"
            : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
            : "r"(h[i]));
}
__device__ __forceinline__ float e4m3_value(uint8_t v) {
    uint32_t h;
    float f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)v));
    asm("{\n.reg .f16 a, b;\nmov.b32 {a, b}, %1;\ncvt.f32.f16 %0, a;\n}" : "=f"(f) : "r"(h));
    return f;
}
// One E2M1 code: 0, 0.5, 1, 1.5, 2, 3, 4, 6, and with bit 3 their negatives.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t e = c >> 1 & 3u;
    const float m = e ? __uint_as_float((e + 126u) << 23 | (c & 1u) << 22) : (float)(c & 1u) * 0.5f;
    return c & 8u ? -m : m;
}

}  // namespace mbx
