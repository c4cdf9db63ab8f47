// rowgroup.cuh -- element access shared by the training kernels.
#pragma once

#include "numerics.cuh"
#include "train.h"

namespace mbx {

template <class T>
struct ChunkOf;
template <>
struct ChunkOf<uint16_t> {  // bfloat16 bits
    static constexpr int CE = 8;
};
template <>
struct ChunkOf<float> {
    static constexpr int CE = 4;
};

__device__ __forceinline__ void widen_chunk(const uint4& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = lo_f(w_of(v, i));
        f[2 * i + 1] = hi_f(w_of(v, i));
    }
}
__device__ __forceinline__ void widen_chunk(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint4 narrow_chunk(const float (&f)[8]) {  // one rounding to bfloat16
    return make_uint4(pack_rn(f[0], f[1]), pack_rn(f[2], f[3]), pack_rn(f[4], f[5]), pack_rn(f[6], f[7]));
}
__device__ __forceinline__ uint4 narrow_chunk(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

__device__ __forceinline__ float load_elem(const uint16_t* p) { return __uint_as_float((uint32_t)ld_u16_rw(p) << 16); }
__device__ __forceinline__ float load_elem(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void store_elem(uint16_t* p, float v) { st_u16(p, (uint16_t)(pack_rn(v, 0.0f) & 0xffffu)); }
__device__ __forceinline__ void store_elem(float* p, float v) {
    asm volatile("st.global.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}

// How rows are moved (rowring.cuh): kVec by aligned 16-byte chunks; kShift where
// a width is no multiple of a chunk or a row starts at no 16-byte boundary.
enum Access { kShift = 0, kVec = 1 };

__device__ __forceinline__ void named_bar(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

constexpr int kMaxWarpsPerRow = 16;

}  // namespace mbx
