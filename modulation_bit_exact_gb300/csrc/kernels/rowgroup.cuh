// rowgroup.cuh -- the row machinery of the training kernels.
//
// A row group of `tpr` threads (whole warps) owns one row at a time; thread t
// holds E of its elements in registers as binary32, in chunks of one 16-byte
// access (CE elements: 8 bfloat16 or 4 binary32).  kVec: chunk j of thread t is
// chunk j*tpr + t of the row, so a warp's accesses are consecutive 16-byte
// pieces.  Otherwise (a width that is no multiple of CE, or a row that starts
// at no 16-byte boundary) accesses are single elements: kScalar gives element e
// of thread t column e*tpr + t, so a warp's accesses are consecutive; kQuad
// gives a thread four consecutive columns at a time, which share one call of
// the dropout generator.  Elements past the row's end are held as 0.
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

enum Access { kScalar = 0, kVec = 1, kQuad = 2 };

// Column of a thread's element e for thread t of a group of tpr threads.
template <class T, Access A>
__device__ __forceinline__ int col_of(int e, int t, int tpr) {
    constexpr int CE = ChunkOf<T>::CE;
    return A == kVec ? (e / CE * tpr + t) * CE + e % CE : A == kQuad ? (e / 4 * tpr + t) * 4 + e % 4 : e * tpr + t;
}

// A thread's chunks of a row as loaded (not yet widened), so that the next
// row can be in flight in half the registers.  The kernels may overwrite a
// row they have read (an exact in-place update), so loads are coherent.
template <class T, int NCH, Access A>
struct RawRow {
    float v[NCH * ChunkOf<T>::CE];
    __device__ __forceinline__ void load(const T* row, int D, int t, int tpr) {
#pragma unroll
        for (int e = 0; e < NCH * ChunkOf<T>::CE; ++e) {
            const int c = col_of<T, A>(e, t, tpr);
            v[e] = c < D ? load_elem(row + c) : 0.0f;
        }
    }
    __device__ __forceinline__ void widen(float (&f)[NCH * ChunkOf<T>::CE]) const {
#pragma unroll
        for (int e = 0; e < NCH * ChunkOf<T>::CE; ++e) f[e] = v[e];
    }
};
template <class T, int NCH>
struct RawRow<T, NCH, kVec> {
    uint4 v[NCH];
    __device__ __forceinline__ void load(const T* row, int D, int t, int tpr) {
        constexpr int CE = ChunkOf<T>::CE;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = j * tpr + t;
            v[j] = c * CE < D ? ld_stream_rw(row + (int64_t)c * CE) : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void widen(float (&f)[NCH * ChunkOf<T>::CE]) const {
        constexpr int CE = ChunkOf<T>::CE;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            float w[CE];
            widen_chunk(v[j], w);
#pragma unroll
            for (int i = 0; i < CE; ++i) f[j * CE + i] = w[i];
        }
    }
};
template <class T, int NCH, Access A>
__device__ __forceinline__ void store_row(T* row, const float (&f)[NCH * ChunkOf<T>::CE], int D, int t, int tpr) {
    constexpr int CE = ChunkOf<T>::CE;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        if constexpr (A == kVec) {
            const int c = j * tpr + t;
            float w[CE];
#pragma unroll
            for (int i = 0; i < CE; ++i) w[i] = f[j * CE + i];
            if (c * CE < D) st_v4(row + (int64_t)c * CE, narrow_chunk(w));
        } else {
#pragma unroll
            for (int i = 0; i < CE; ++i) {
                const int c = col_of<T, A>(j * CE + i, t, tpr);
                if (c < D) store_elem(row + c, f[j * CE + i]);
            }
        }
    }
}

// A parameter row (bfloat16 or binary32, whatever T is) at this thread's
// columns, as binary32; `fill` past the row's end.
template <class T, int NCH, Access A>
__device__ __forceinline__ void load_params(float (&f)[NCH * ChunkOf<T>::CE], const void* p, int64_t row_off,
                                            bool p_f32, int D, int t, int tpr, float fill) {
    constexpr int CE = ChunkOf<T>::CE;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        if constexpr (A == kVec) {
            const int c = (j * tpr + t) * CE;
            if (c < D) {
                if (p_f32) {
                    const float* q = static_cast<const float*>(p) + row_off + c;
#pragma unroll
                    for (int h = 0; h < CE / 4; ++h) {
                        float w[4];
                        widen_chunk(ld_shared_row(q + 4 * h), w);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[j * CE + 4 * h + i] = w[i];
                    }
                } else if constexpr (CE == 8) {  // binary32 rows never go with bfloat16 parameters
                    float w[8];
                    widen_chunk(ld_shared_row(static_cast<const uint16_t*>(p) + row_off + c), w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[j * 8 + i] = w[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < CE; ++i) f[j * CE + i] = fill;
            }
        } else {
#pragma unroll
            for (int i = 0; i < CE; ++i) {
                const int c = col_of<T, A>(j * CE + i, t, tpr);
                float v = fill;
                if (c < D)
                    v = p_f32 ? load_elem(static_cast<const float*>(p) + row_off + c)
                              : load_elem(static_cast<const uint16_t*>(p) + row_off + c);
                f[j * CE + i] = v;
            }
        }
    }
}

// A parameter row's gradient at this thread's columns, rounded once.
template <class T, int NCH, Access A>
__device__ __forceinline__ void store_params(void* p, int64_t row_off, bool p_f32, const float (&f)[NCH * ChunkOf<T>::CE],
                                             int D, int t, int tpr) {
    constexpr int CE = ChunkOf<T>::CE;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        if constexpr (A == kVec) {
            const int c = (j * tpr + t) * CE;
            if (c < D) {
                if (p_f32) {
                    float* q = static_cast<float*>(p) + row_off + c;
#pragma unroll
                    for (int h = 0; h < CE / 4; ++h) {
                        float w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = f[j * CE + 4 * h + i];
                        st_v4(q + 4 * h, narrow_chunk(w));
                    }
                } else if constexpr (CE == 8) {
                    float w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = f[j * 8 + i];
                    st_v4(static_cast<uint16_t*>(p) + row_off + c, narrow_chunk(w));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < CE; ++i) {
                const int c = col_of<T, A>(j * CE + i, t, tpr);
                if (c < D) {
                    if (p_f32) store_elem(static_cast<float*>(p) + row_off + c, f[j * CE + i]);
                    else store_elem(static_cast<uint16_t*>(p) + row_off + c, f[j * CE + i]);
                }
            }
        }
    }
}

__device__ __forceinline__ void named_bar(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

constexpr int kMaxWarpsPerRow = 16;

// Sums of two values over a row group, in every thread: shuffles inside each
// warp, then every thread adds the warps' values in warp order.  The published
// values alternate between two buffers: a buffer is written again two sums
// later, after the barrier of the sum in between, which every reader has
// passed.
struct GroupSum {
    float2* buf;  // [2][kMaxWarpsPerRow] of this group
    int t, tpr, bar_id, par;
    __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
        for (int s = 16; s >= 1; s /= 2) {
            a += __shfl_xor_sync(0xffffffffu, a, s);
            b += __shfl_xor_sync(0xffffffffu, b, s);
        }
        if (tpr == 32) return make_float2(a, b);
        float2* slot = buf + par * kMaxWarpsPerRow;
        par ^= 1;
        if (t % 32 == 0) slot[t / 32] = make_float2(a, b);
        named_bar(bar_id, tpr);
        const int warps = tpr / 32;
        float2 s = slot[0];
        for (int w = 1; w < warps; ++w) {
            s.x += slot[w].x;
            s.y += slot[w].y;
        }
        return s;
    }
};

}  // namespace mbx
