// lnorm.cuh -- the launch shape shared by the LayerNorm kernels.
#pragma once

#include "rowring.cuh"

namespace mbx {

__device__ __forceinline__ GroupSums group_sums(char* smem, const RingShape& sh, int g, int t) {
    float* buf = reinterpret_cast<float*>(smem) + g * kSumFloats;
    if (sh.tpr > 32) {
        for (int i = t; i < kSumFloats; i += sh.tpr) buf[i] = 0.0f;
        named_bar(g + 1, sh.tpr);  // the warps that are not there add nothing
    }
    return GroupSums{buf, t, sh.tpr, g + 1, 0};
}

}  // namespace mbx
