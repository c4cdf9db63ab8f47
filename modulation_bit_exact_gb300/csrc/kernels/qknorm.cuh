// qknorm.cuh -- how a warp holds heads, for the norm of Q and K heads with the
// rotation (qknorm.cu) and its gradients (qknorm_bwd.cu).
//
// A head is cut into units, one unit of a lane at a time: interleaved pairs lie
// side by side, so a unit is one access of W elements; pairs in halves (j, j+n)
// are the access at j and the one at j+n; elements past the pairs come two
// accesses a unit.  With W = 1 a unit is one pair, or two elements that pass.
// A group of G lanes (a power of two up to 32) has the head's units, unit
// lane + G*u in place u < U, so a row sum is a chain within the lane and a
// butterfly over the group.  W, G and U follow the head's size, its pairs and the
// type alone: where a head lies decides only whether an access is one load
// or one for each element, so its bits are the same at any address.
#pragma once

#include "rope.cuh"

namespace mbx {

// An access of W elements as 32-bit words, and as binary32 values.
template <class T, int W, bool VEC>
struct Access1 {
    static constexpr int NW = W * (int)sizeof(T) >= 4 ? W * (int)sizeof(T) / 4 : 1;
    uint32_t w[NW];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (!VEC || W == 1) {
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < W; ++i) w[i] = __float_as_uint(load_elem(p + i));
            } else {
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    w[i] = ld_u16_rw(p + 2 * i);
                    if constexpr (W > 1) w[i] |= (uint32_t)ld_u16_rw(p + 2 * i + 1) << 16;
                }
            }
        } else if constexpr (NW == 4) {
            const uint4 v = ld_stream_rw(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (!VEC || W == 1) {
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < W; ++i) store_elem(p + i, __uint_as_float(w[i]));
            } else {
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    st_u16(p + 2 * i, (uint16_t)w[i]);
                    if constexpr (W > 1) st_u16(p + 2 * i + 1, (uint16_t)(w[i] >> 16));
                }
            }
        } else if constexpr (NW == 4) {
            st_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
        } else {
            st_v2(p, w[0], w[1]);
        }
    }
    __device__ __forceinline__ void widen(float* f) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                f[2 * i] = lo_f(w[i]);
                if constexpr (W > 1) f[2 * i + 1] = hi_f(w[i]);
            }
        }
    }
    __device__ __forceinline__ void narrow(const float* f) {  // one rounding to T
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NW; ++i) w[i] = pack_rn(f[2 * i], W > 1 ? f[2 * i + 1] : 0.0f);
        }
    }
};

// A lane's units of a head.  Values in the order of the accesses: of the A*W
// values of a unit, pair i is (2i, 2i+1) in one access and (i, W+i) in two.
template <class T, bool INTERLEAVED, int W, int U, bool VEC>
struct HeadUnits {
    static constexpr bool kTwo = !INTERLEAVED || W == 1;  // two accesses a unit
    static constexpr int A = kTwo ? 2 : 1, E = A * W, P = E / 2;
    static constexpr int lo(int i) { return kTwo ? i : 2 * i; }
    static constexpr int hi(int i) { return kTwo ? W + i : 2 * i + 1; }
    int off0[U], off1[U];    // offsets within a head, < 0: none
    int pair0[U], turns[U];  // pairs pair0 .. pair0 + turns - 1 of the unit turn
    __device__ __forceinline__ HeadUnits(int lane, int G, int hd, int n) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int a = lane + G * u;
            if constexpr (!kTwo) {
                off0[u] = a * W < hd ? a * W : -1;
                off1[u] = -1;
                pair0[u] = a * P;
                turns[u] = min(max(n - pair0[u], 0), P);
            } else {
                const int nt = n / W;  // units that turn
                const bool t = a < nt;
                const int pass = 2 * n + 2 * (a - nt) * W;
                off0[u] = t ? (INTERLEAVED ? 2 * a : a * W) : (pass < hd ? pass : -1);
                off1[u] = t ? (INTERLEAVED ? 2 * a + 1 : n + a * W) : (pass + W < hd ? pass + W : -1);
                pair0[u] = a * W;
                turns[u] = t ? W : 0;
            }
        }
    }
    struct Raw {
        Access1<T, W, VEC> a[U][A];
    };
    __device__ __forceinline__ void load(Raw& r, const T* head) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (off0[u] >= 0) r.a[u][0].load(head + off0[u]);
            if constexpr (kTwo)
                if (off1[u] >= 0) r.a[u][1].load(head + off1[u]);
        }
    }
    // Values of the head's elements; 0 where the lane has none.
    __device__ __forceinline__ void values(float (&f)[U][E], const Raw& r) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r.a[u][0].widen(f[u]);
            if (off0[u] < 0) {
#pragma unroll
                for (int i = 0; i < W; ++i) f[u][i] = 0.0f;
            }
            if constexpr (kTwo) {
                r.a[u][1].widen(f[u] + W);
                if (off1[u] < 0) {
#pragma unroll
                    for (int i = 0; i < W; ++i) f[u][W + i] = 0.0f;
                }
            }
        }
    }
    __device__ __forceinline__ void store(T* head, const float (&f)[U][E]) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Access1<T, W, VEC> a;
            if (off0[u] >= 0) {
                a.narrow(f[u]);
                a.store(head + off0[u]);
            }
            if constexpr (kTwo)
                if (off1[u] >= 0) {
                    a.narrow(f[u] + W);
                    a.store(head + off1[u]);
                }
        }
    }
    // f = w's elements, 1 where w is null
    __device__ __forceinline__ void weight(float (&f)[U][E], const void* w, bool w_f32) const {
        auto one = [&](int e) {
            return !w ? 1.0f : w_f32 ? load_elem(static_cast<const float*>(w) + e) : load_elem(static_cast<const uint16_t*>(w) + e);
        };
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                f[u][i] = off0[u] >= 0 ? one(off0[u] + i) : 0.0f;
                if constexpr (kTwo) f[u][W + i] = off1[u] >= 0 ? one(off1[u] + i) : 0.0f;
            }
    }
    // This lane's cosines and sines out of those of the token's n pairs.
    __device__ __forceinline__ void angles(float (&c)[U][P], float (&s)[U][P], const float2* cs) const {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 v = i < turns[u] ? cs[pair0[u] + i] : make_float2(1.0f, 0.0f);
                c[u][i] = v.x;
                s[u][i] = v.y;
            }
    }
    // Turns the pairs of f: each result one product and one fused multiply-add.
    __device__ __forceinline__ void turn(float (&f)[U][E], const float (&c)[U][P], const float (&s)[U][P]) const {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float x0 = f[u][lo(i)], x1 = f[u][hi(i)];
                if (i < turns[u]) {
                    f[u][lo(i)] = __fmaf_rn(-x1, s[u][i], __fmul_rn(x0, c[u][i]));
                    f[u][hi(i)] = __fmaf_rn(x0, s[u][i], __fmul_rn(x1, c[u][i]));
                }
            }
    }
};

// Sum over the G lanes of a group, in every lane.
__device__ __forceinline__ float group_sum(float v, int G) {
    for (int m = 1; m < G; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// The widest access (in elements) that divides the head and, where pairs lie in
// halves, the number of pairs; 1 where only single elements do.
inline int unit_width(int hd, int n, bool f32, bool interleaved) {
    auto fits = [&](int w) { return hd % w == 0 && (interleaved || n % w == 0); };
    return f32 ? (fits(4) ? 4 : 1) : fits(8) ? 8 : fits(4) ? 4 : 1;
}
inline int head_units(int hd, int n, int w, bool interleaved) {
    if (interleaved && w > 1) return hd / w;
    return n / w + ((hd - 2 * n) / w + 1) / 2;
}

// Calls f(T, INTERLEAVED, W, U, VEC as types) for a head's shape; G is the group.
template <int V>
using Int = std::integral_constant<int, V>;
template <bool V>
using Bool = std::integral_constant<bool, V>;

template <class F>
cudaError_t for_head_shape(int hd, int n, bool f32, bool interleaved, int align, F&& f) {
    const int w = unit_width(hd, n, f32, interleaved), units = head_units(hd, n, w, interleaved);
    const bool vec = align >= w * (f32 ? 4 : 2);
    const int u = units <= 32 ? 1 : units <= 64 ? 2 : 4;  // hd <= 256: at most 128 units
    int g = 1;
    while (g * u < units) g *= 2;
    auto with_u = [&](auto t, auto inter, auto width, auto v) {
        if constexpr (decltype(width)::value == 8) return f(t, inter, width, Int<1>(), v, g);
        else if (u == 1) return f(t, inter, width, Int<1>(), v, g);
        else if (decltype(width)::value > 1 || u == 2) return f(t, inter, width, Int<2>(), v, g);
        else return f(t, inter, Int<1>(), Int<4>(), v, g);
    };
    auto with_w = [&](auto t, auto inter) {
        constexpr bool kF32 = sizeof(t) == 4;
        if constexpr (!kF32)
            if (w == 8) return vec ? with_u(t, inter, Int<8>(), Bool<true>()) : with_u(t, inter, Int<8>(), Bool<false>());
        if (w == 4) return vec ? with_u(t, inter, Int<4>(), Bool<true>()) : with_u(t, inter, Int<4>(), Bool<false>());
        return with_u(t, inter, Int<1>(), Bool<true>());
    };
    if (f32) return interleaved ? with_w(0.0f, Bool<true>()) : with_w(0.0f, Bool<false>());
    return interleaved ? with_w((uint16_t)0, Bool<true>()) : with_w((uint16_t)0, Bool<false>());
}

}  // namespace mbx
