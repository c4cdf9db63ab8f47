// lnorm.cuh -- what the LayerNorm kernels share.
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

// The mean m of a row is a rounded sum times a rounded 1/D, off by up to some 40
// roundings of mean|x|.  In a row far from zero that is much beside the deviations
// x - m: a constant row of 1000 in 104 columns gave -0.06 where 0 is right.  So with
// delta = mean(x - m),
//   var = mean((x - m)^2) - delta^2,   xh = (x - m - delta) * rstd,
// and what is left of the error is of second order.
//
// binary32 rows: the deviations are summed too, in the exchange that sums their
// squares (LayerNorm of [30000, 2048] 84.1 -> 85.3 us, its gradients of [19528, 2048]
// 106.8 -> 107.4).
//
// bfloat16 rows: delta is what the sum has left over D*m, for no sum; the gradients,
// short of registers, subtract it along with the mean (LayerNorm of [32760, 5120]
// 104.6 -> 108 us, gradients of [31248, 5120] 201 -> 212, with a residual 233 -> 240;
// subtracted later 215 and 279; with the deviations summed LayerNorm took 124, the
// gradients 238).  The sum is exact where no element is below D / 2^16 of the largest
// (an eighth at 8192 columns): all are whole multiples of one quantum, and so is every
// partial sum, below 2^24 of them.  Otherwise the row's standard deviation is at least
// 0.6 mean|x| / sqrt(D), and a chain of at most 29 roundings puts the mean off by less
// than 3e-4 of it.
template <class T>
constexpr bool kSumDeviations = sizeof(T) == 4;

// (sum - D*m) / D with m = sum * inv_d, the difference rounded once.
__device__ __forceinline__ float mean_rest(float sum, int D, float inv_d) {
    return fmaf(-(sum * inv_d), (float)D, sum) * inv_d;
}

// 1/sqrt(var + eps) of a row whose deviations have the mean square q and the mean
// delta.  The difference may round below 0.
__device__ __forceinline__ float rstd_of(float q, float delta, float eps) {
    const float var = fmaf(-delta, delta, q);
    return rsqrtf((var < 0.0f ? 0.0f : var) + eps);
}

}  // namespace mbx
