// linear.h -- internal interface between the C ABI (linear_api.cu) and the
// products with NVFP4 weights.  Not installed; not part of the ABI.
#pragma once

#include "launch.h"

namespace mbx {

int sm_count();  // SMs of the current device; 0 if the runtime cannot tell

struct LinearParams {
    void* out;
    int64_t out_stride;
    const void* x;
    int64_t x_stride;
    int rows, K;
    int64_t N;
    const uint8_t* w4;  // [N, K/2] pairs of E2M1 codes
    int64_t w_stride;   // bytes
    const uint8_t* sf;  // E4M3 scales in tiles of 128 rows x 4 blocks
    int sf_col_tiles;   // tiles of a band of 128 rows
    const float* gs;    // device: the global scale
    const void* bias;   // [N] or null
    bool bias_f32, silu;
    float* ws;
};

int64_t linear_nvfp4_workspace_bytes(int rows, int64_t N, int K);

bool linear_tc_takes(const LinearParams& p);
cudaError_t launch_linear_tc(const LinearParams& p, bool x_f32, bool out_f32, cudaStream_t s);
cudaError_t launch_linear_nvfp4(const LinearParams& p, bool x_f32, bool out_f32, cudaStream_t s);

}  // namespace mbx
