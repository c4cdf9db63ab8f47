// qknorm.cuh -- how a warp holds heads, for the norm of Q and K heads with the
// rotation (qknorm.cu) and its gradients (qknorm_bwd.cu).
//
// A head is cut into units, one unit of a lane at a time: interleaved pairs lie
// side by side, so a unit is one access of W elements; pairs in halves (j, j+n)
// are the access at j and the one at j+n; of the elements past the pairs a unit has an
// access of their first half and one of their second, so that lanes side by side have
// accesses side by side.  With W = 1 a unit is one pair, or two elements that pass.
// A group of G lanes has the head's units, unit lane + G*u in place u < U, so a row
// sum is a chain within the lane and a tree over the group.  W, G and U follow the
// head's size, its pairs and the type alone: where a head lies decides only whether an
// access is one load or one for each element, so its bits are the same at any address.
#pragma once

#include <type_traits>

#include "rowgroup.cuh"

namespace mbx {

template <int V>
using Int = std::integral_constant<int, V>;
template <bool V>
using Bool = std::integral_constant<bool, V>;

// The angles.  Position * frequency / (2 pi) turns, modulo a turn, in fixed point.  Once
// in a block for each pair the turns of one position are formed, the product of the
// frequency's 53 bits with 192 bits of 1 / (2 pi), to 2^-128 of a turn; once for each token
// they are multiplied by the position and cut to 2^-64 of a turn, in integers: an angle
// loses 2^-128 of a turn for each unit of its position, and the little binary64 that this
// GPU has is not used (65536 tokens of one head of 128 each for Q and K, whose angles are
// most of the work: 121 us with binary64, 89 in integers, 37 with what else is shared now).
struct PairFreq {  // 24 bytes: lanes that read structures side by side meet two at a bank (of 32 eight, gradients +1.8%)
    uint64_t hi, lo;  // the turns of one position: whole() + hi * 2^-64 + lo * 2^-128
    uint64_t tagged;
    __device__ __forceinline__ uint64_t whole() const { return tagged >> 4; }  // below 2^52
    __device__ __forceinline__ bool bad() const { return tagged & 8; }        // 2^54 or more, or not finite
    __device__ __forceinline__ bool minus() const { return tagged & 4; }
    __device__ __forceinline__ int axis() const { return (int)tagged & 3; }
};
// (hi:lo) >> n, its low word; n below 64
__device__ __forceinline__ uint64_t shift_right(uint64_t hi, uint64_t lo, int n) { return hi << 1 << (63 - n) | lo >> n; }
__device__ __forceinline__ PairFreq pair_freq(const RopeParams& p, int j) {
    PairFreq q;
    int a = 0;
    while (a < p.axes - 1 && j >= p.axis_end[a]) ++a;
    const uint64_t fb = __double_as_longlong(p.freqs[j]);
    const int fe = (int)(fb >> 52 & 2047) - 1023;  // the frequency is 1.m * 2^fe
    const bool bad = fe > 53;
    const uint64_t m = fe < -1022 ? 0 : (fb & 0xfffffffffffffull) | 1ull << 52;
    // m / (2 pi) in units of 2^-192, four words
    typedef unsigned __int128 u128;
    const u128 t0 = (u128)m * 0x36d8a5664f10e410ull;
    const u128 t1 = (u128)m * 0x7f09d5f47d4d3770ull + (uint64_t)(t0 >> 64);
    const u128 t2 = (u128)m * 0x28be60db9391054aull + (uint64_t)(t1 >> 64);
    uint64_t w0 = (uint64_t)t0, w1 = (uint64_t)t1, w2 = (uint64_t)t2, w3 = (uint64_t)(t2 >> 64);
    // times 2^(fe - 52), in units of 2^-128
    const int sh = bad ? 63 : 64 + 52 - fe;
    if (sh & 64) w0 = w1, w1 = w2, w2 = w3, w3 = 0;
    if (sh & 128) w0 = w2, w1 = w3, w2 = w3 = 0;
    if (sh >= 256) w0 = w1 = w2 = w3 = 0;
    q.lo = shift_right(w1, w0, sh & 63);
    q.hi = shift_right(w2, w1, sh & 63);
    q.tagged = shift_right(w3, w2, sh & 63) << 4 | (bad ? 8 : 0) | ((int64_t)fb < 0 ? 4 : 0) | (unsigned)a;
    return q;
}
// A position's bits on an axis at a token (its index `tok` in the batch, `s` in its sequence).
__device__ __forceinline__ uint32_t position_bits(const RopeParams& p, unsigned tok, unsigned s, int axis) {
    uint32_t v;
    const uint32_t* at = static_cast<const uint32_t*>(p.pos) + (int64_t)(p.pos_batched ? tok : s) * p.pos_stride + axis;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(at));
    return v;
}
// cos and sin of the angle, to 1.73 * 2^-24.  The remainder, at most an eighth of a turn,
// goes through the Taylor series, whose first terms left out, t^11 / 11! and t^12 / 12!, are
// below 2^-29.
__device__ __forceinline__ float2 pair_angle(const RopeParams& p, const PairFreq& q, uint32_t pos) {
    uint64_t T;  // turns in units of 2^-64
    bool minus = q.minus() != ((int)pos < 0), bad = q.bad();
    if (!p.pos_f32) {
        const uint32_t n = (int)pos < 0 ? 0u - pos : pos;
        T = q.hi * n + __umulhi((uint32_t)(q.lo >> 32), n);
    } else {
        const int e = (int)(pos >> 23 & 255);  // the position is pm * 2^(e - 150)
        bad |= e == 255;
        const uint64_t pm = e ? (pos & 0x7fffffu) | 0x800000u : (pos & 0x7fffffu) << 1;
        // pm times the turns of one position in units of 2^-128, of which 64 bits from bit sh are wanted
        const uint64_t w0 = q.lo * pm, c0 = __umul64hi(q.lo, pm), w1 = q.hi * pm + c0;
        const uint64_t c1 = __umul64hi(q.hi, pm) + (w1 < c0), w2 = q.whole() * pm + c1;
        const uint64_t w3 = __umul64hi(q.whole(), pm) + (w2 < c1);
        const int sh = 214 - e;
        T = sh >= 192 ? w3 >> (sh - 192) : sh >= 128 ? shift_right(w3, w2, sh - 128) : sh >= 64 ? shift_right(w2, w1, sh - 64)
            : sh >= 0 ? shift_right(w1, w0, sh) : w0 << -sh;
    }
    if (minus != p.inverse) T = 0 - T;
    const uint32_t quadrant = (uint32_t)((T + (1ull << 61)) >> 62);
    const float t = (float)(int)((T - ((uint64_t)quadrant << 62)) >> 32) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float z = t * t;
    float c = __fmaf_rn(z, -2.7557319e-7f, 2.4801587e-5f), n = __fmaf_rn(z, 2.7557319e-6f, -1.9841270e-4f);
    c = __fmaf_rn(z, c, -1.3888889e-3f), n = __fmaf_rn(z, n, 8.3333333e-3f);
    c = __fmaf_rn(z, c, 4.1666667e-2f), n = __fmaf_rn(z, n, -1.6666667e-1f);
    c = __fmaf_rn(z, c, -0.5f), n = __fmaf_rn(t * z, n, t);
    c = __fmaf_rn(z, c, 1.0f);
    const float cc = quadrant & 1 ? -n : c, ss = quadrant & 1 ? c : n;
    if (bad) return make_float2(__uint_as_float(0x7fffffffu), __uint_as_float(0x7fffffffu));
    return quadrant & 2 ? make_float2(-cc, -ss) : make_float2(cc, ss);
}

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
        } else if constexpr (NW == 2) {
            asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
        } else {
            asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
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
        } else if constexpr (NW == 4) {  // streamed: 32760 x 80 heads of 128, 219 -> 208 us
            asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
        } else if constexpr (NW == 2) {
            asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(w[0]), "r"(w[1]) : "memory");
        } else {
            asm volatile("st.global.cs.u32 [%0], %1;" ::"l"(p), "r"(w[0]) : "memory");
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

// A lane's units of a head.  The P pairs of a unit are held as packed binary32: a
// Values' first[u][i] has the first elements of pairs 2i and 2i+1, second the
// second ones (the pairs of elements that pass are those of their accesses).  Words
// of elements that the lane does not have stay 0.
template <class T, bool INTERLEAVED, int W, int U, bool VEC>
struct HeadUnits {
    static constexpr bool kTwo = !INTERLEAVED || W == 1;  // two accesses a unit
    static constexpr int A = kTwo ? 2 : 1, E = A * W, P = E / 2, NP = (P + 1) / 2;
    int off0[U], off1[U];    // offsets within a head, < 0: none
    int pair0[U], turns[U];  // pairs pair0 .. pair0 + turns - 1 of the unit turn
    bool all_turn;           // of every lane that has elements: no element passes
    __device__ __forceinline__ HeadUnits(int lane, int G, int hd, int n) {
        all_turn = 2 * n == hd;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int a = lane + G * u;
            if constexpr (!kTwo) {
                off0[u] = a * W < hd ? a * W : -1;
                off1[u] = -1;
                pair0[u] = a * P;
                turns[u] = min(max(n - pair0[u], 0), P);
            } else {
                const int nt = n / W, np = ((hd - 2 * n) / W + 1) / 2;  // units that turn, that pass
                const bool t = a < nt, own = a < nt + np;
                const int pass = 2 * n + (a - nt) * W;
                off0[u] = t ? (INTERLEAVED ? 2 * a : a * W) : own ? pass : -1;
                off1[u] = t ? (INTERLEAVED ? 2 * a + 1 : n + a * W) : own && pass + np * W < hd ? pass + np * W : -1;
                pair0[u] = a * W;
                turns[u] = t ? W : 0;
            }
        }
    }
    struct Raw {
        Access1<T, W, VEC> a[U][A];
        __device__ __forceinline__ void clear() {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < A; ++k)
#pragma unroll
                    for (int i = 0; i < Access1<T, W, VEC>::NW; ++i) a[u][k].w[i] = 0;
        }
    };
    struct Values {
        u64 first[U][NP], second[U][NP];
    };
    // Heads on their way: where accesses are aligned each lane copies its own to its
    // place in shared memory, asynchronously, and reads them back itself, so nothing
    // but its own wait orders the two.  One slot has a head of every group of the warp.
    static constexpr bool kRing = VEC && W > 1;
    static constexpr int kAccessBytes = W * (int)sizeof(T), kSlotBytes = kRing ? U * A * 32 * kAccessBytes : 0;
    __device__ __forceinline__ void copy(uint32_t slot, const T* head) const {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < A; ++k) {
                const int off = k ? off1[u] : off0[u];
                const uint32_t to = slot + (u * A + k) * 32 * kAccessBytes;
                if (off >= 0) {
                    if constexpr (kAccessBytes == 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(head + off) : "memory");
                    else
                        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(head + off), "n"(kAccessBytes) : "memory");
                }
            }
    }
    __device__ __forceinline__ void read(Raw& r, uint32_t slot) const {  // into a Raw that was cleared once
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < A; ++k) {
                const uint32_t from = slot + (u * A + k) * 32 * kAccessBytes;
                uint32_t* w = r.a[u][k].w;
                if ((k ? off1[u] : off0[u]) >= 0) {
                    if constexpr (kAccessBytes == 16)
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from) : "memory");
                    else if constexpr (kAccessBytes == 8)
                        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(from) : "memory");
                    else
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(from) : "memory");
                }
            }
    }
    __device__ __forceinline__ void load(Raw& r, const T* head) const {  // the same
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (off0[u] >= 0) r.a[u][0].load(head + off0[u]);
            if constexpr (kTwo)
                if (off1[u] >= 0) r.a[u][1].load(head + off1[u]);
        }
    }
    static __device__ __forceinline__ Values pack(const float (&f)[U][E]) {
        Values v;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int j = 2 * i, k = 2 * i + 1 < P ? 2 * i + 1 : -1;
                const int s0 = kTwo ? 1 : 2, d = kTwo ? W : 1;  // pair j: elements s0*j and s0*j + d
                v.first[u][i] = f2(f[u][s0 * j], k < 0 ? 0.0f : f[u][s0 * k]);
                v.second[u][i] = f2(f[u][s0 * j + d], k < 0 ? 0.0f : f[u][s0 * k + d]);
            }
        return v;
    }
    static __device__ __forceinline__ void unpack(float (&f)[U][E], const Values& v) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int s0 = kTwo ? 1 : 2, d = kTwo ? W : 1;
                f[u][s0 * j] = j & 1 ? f2hi(v.first[u][j / 2]) : f2lo(v.first[u][j / 2]);
                f[u][s0 * j + d] = j & 1 ? f2hi(v.second[u][j / 2]) : f2lo(v.second[u][j / 2]);
            }
    }
    static __device__ __forceinline__ Values values(const Raw& r) {
        float f[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < A; ++k) r.a[u][k].widen(f[u] + k * W);
        return pack(f);
    }
    __device__ __forceinline__ void store(T* head, const Values& v) const {
        float f[U][E];
        unpack(f, v);
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
    // w's elements, 1 where w is null
    __device__ __forceinline__ Values weight(const void* w, bool w_f32) const {
        float f[U][E];
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
        return pack(f);
    }
    // What turns a token's pairs: of (x0, x1) the first result is x0*a + x1*b, the second
    // x0*c + x1*d.
    struct Turn {
        u64 a[U][NP], b[U][NP], c[U][NP], d[U][NP];
    };
    // The rotation by the cosines and sines of the token's n pairs, out of cs, of values
    // that are multiplied by w first.
    __device__ __forceinline__ Turn turn_of(const float2* cs, const Values& w) const {
        Turn t;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float2 x = 2 * i < turns[u] ? cs[pair0[u] + 2 * i] : make_float2(1.0f, 0.0f);
                const float2 y = 2 * i + 1 < turns[u] ? cs[pair0[u] + 2 * i + 1] : make_float2(1.0f, 0.0f);
                const u64 co = f2(x.x, y.x), si = f2(x.y, y.y);
                t.a[u][i] = mul2(w.first[u][i], co);
                t.b[u][i] = mul2(w.second[u][i], f2(-x.y, -y.y));
                t.c[u][i] = mul2(w.first[u][i], si);
                t.d[u][i] = mul2(w.second[u][i], co);
            }
        return t;
    }
    // The rotation alone, a = d and c = -b.
    struct Rotation {
        u64 a[U][NP], b[U][NP], c[U][NP];
    };
    __device__ __forceinline__ Rotation rotation(const float2* cs) const {
        Rotation t;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float2 x = 2 * i < turns[u] ? cs[pair0[u] + 2 * i] : make_float2(1.0f, 0.0f);
                const float2 y = 2 * i + 1 < turns[u] ? cs[pair0[u] + 2 * i + 1] : make_float2(1.0f, 0.0f);
                t.a[u][i] = f2(x.x, y.x);
                t.b[u][i] = f2(-x.y, -y.y);
                t.c[u][i] = f2(x.y, y.y);
            }
        return t;
    }
    static __device__ __forceinline__ u64 second_factor(const Turn& t, int u, int i) { return t.d[u][i]; }
    static __device__ __forceinline__ u64 second_factor(const Rotation& t, int u, int i) { return t.a[u][i]; }
    template <class R>
    __device__ __forceinline__ void turn(Values& v, const R& t) const {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const u64 x0 = v.first[u][i], x1 = v.second[u][i], y0 = mul2(x0, t.a[u][i]), y1 = mul2(x1, second_factor(t, u, i));
                v.first[u][i] = fma2(x1, t.b[u][i], y0);
                v.second[u][i] = fma2(x0, t.c[u][i], y1);
                if (!all_turn) {  // an infinite partner does not reach an element that passes
                    auto keep = [&](u64& now, u64 was) {
                        if (2 * i >= turns[u]) now = (now & 0xffffffff00000000ull) | (was & 0xffffffffull);
                        if (2 * i + 1 >= turns[u]) now = (now & 0xffffffffull) | (was & 0xffffffff00000000ull);
                    };
                    keep(v.first[u][i], y0);
                    keep(v.second[u][i], y1);
                }
            }
    }
};

// The sum of products of a lane's values, the packed halves apart: one chain of each,
// first elements and second ones in turn.
template <class V, int U, int NP>
__device__ __forceinline__ float dot(const u64 (&a0)[U][NP], const u64 (&a1)[U][NP], const V& b) {
    u64 s = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            s = fma2(a0[u][i], b.first[u][i], s);
            s = fma2(a1[u][i], b.second[u][i], s);
        }
    return f2lo(s) + f2hi(s);
}

// Sum over the lanes of a group of GT (GT 0: of G), in every lane.  Groups of a power
// of two meet in a butterfly; others fold their upper half onto the lower one until one
// lane has the sum, which the group then reads.
template <int GT>
__device__ __forceinline__ float group_sum(float v, int G) {
    if constexpr (GT > 0 && (GT & (GT - 1)) == 0) {
#pragma unroll
        for (int m = 1; m < GT; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        return v;
    } else {
        const int g = GT ? GT : G, lane = threadIdx.x % 32, at = lane % g;
        if (GT == 0 && (g & (g - 1)) == 0) {
            for (int m = 1; m < g; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
            return v;
        }
#pragma unroll
        for (int n = g; n > 1; n = (n + 1) / 2) {
            const float up = __shfl_down_sync(0xffffffffu, v, (n + 1) / 2);
            if (at < n / 2) v += up;
        }
        return __shfl_sync(0xffffffffu, v, lane - at);
    }
}

// Two sums at once: the lanes of a pair take one each, and exchange them at the end.
template <int GT>
__device__ __forceinline__ void group_sums(float& a, float& b, int G) {
    const int g = GT ? GT : G;
    if ((g & (g - 1)) != 0 || g < 4) {
        a = group_sum<GT>(a, G);
        b = group_sum<GT>(b, G);
        return;
    }
    const bool odd = threadIdx.x & 1;
    float v = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
    if constexpr (GT > 0) {
#pragma unroll
        for (int m = 2; m < GT; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    } else {
        for (int m = 2; m < g; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    }
    const float o = __shfl_xor_sync(0xffffffffu, v, 1);
    a = odd ? o : v;
    b = odd ? v : o;
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// How tokens and heads are dealt out.  Blocks of kQkWarps warps.  Q and K have blocks of
// their own; either `wpt` warps (a power of two) share a token, or, where a warp has room
// for the heads of several tokens, it takes `tpw` of them at a time.  Where it has room
// for those of Q and of K the forward call takes both (`together`: all blocks are q's),
// with the angles made once (65536 tokens of 1 + 1 heads of 128: 53 us apart, 37
// together; the gradients lose more by lanes of one warp that have different tensors:
// 1 + 1 heads 67 -> 57 us, but 16 + 16 of 256 144 -> 154).
constexpr int kQkWarps = 8, kQkBlocks = 2;  // two blocks an SM: with a third the 80 registers a thread spill
struct QkDeal {
    int blocks, tpw;  // of a tensor
};
struct QkShare {
    QkDeal q, k;
    int wpt;
    bool together;
    FastDiv by_tokens;
};
// For `most` blocks and `groups` heads side by side in a warp.
QkShare qk_share(const RopeParams& r, int64_t most, int groups, bool may_be_together);

__device__ __forceinline__ unsigned batch_of(unsigned tok, const FastDiv& d) { return (unsigned)((tok * d.m) >> d.shift); }

// What a warp works on: its tokens tok0 + tok, step by step of `stride`, its heads h0,
// h0 + step, ...  A lane's group has a token and a head of its own where a warp takes
// several tokens.
struct QkPlace {
    bool k;               // of K
    int block, blocks, tpw, slot, share, sub;
    unsigned tok, stride;  // of this lane
    int h0, h_first, step;
    bool part;            // the lane's group takes part
    template <bool TOGETHER>
    __device__ __forceinline__ QkPlace(const QkShare& sh, int heads_q, int heads_k, int G, int groups, Bool<TOGETHER>) {
        const bool together = TOGETHER && sh.together;
        const int warp = threadIdx.x / 32, group = threadIdx.x % 32 / G;
        // the blocks of K are spread evenly among those of Q (gradients of 2 x 4352 x
        // (24 + 24) heads of 128: 66 us with K's after Q's, 60 so)
        const unsigned all = sh.q.blocks + sh.k.blocks, k_before = blockIdx.x * sh.k.blocks / all;
        k = (blockIdx.x + 1) * sh.k.blocks / all > k_before;
        block = k ? k_before : blockIdx.x - k_before;
        blocks = k ? sh.k.blocks : sh.q.blocks;
        tpw = k ? sh.k.tpw : sh.q.tpw;
        slot = warp / sh.wpt;
        share = warp % sh.wpt;
        step = groups * sh.wpt;
        h_first = share * groups;
        if (together || tpw > 1) {  // group = (token, head)
            const int heads = together ? heads_q + heads_k : k ? heads_k : heads_q;
            sub = group / heads;
            h0 = group - sub * heads;
            part = sub < tpw;
            if (together && h0 >= heads_q) {
                k = true;
                h0 -= heads_q;
            }
        } else {
            sub = 0;
            h0 = h_first + group;
            part = group < groups;
        }
        if (!part) sub = 0;
        const int per_block = kQkWarps / sh.wpt * tpw;
        tok = block * per_block + slot * tpw + sub;
        stride = blocks * per_block;
    }
};

// The sines and cosines of the tokens that a warp, with the others that share them
// (this is `id` of `wpt`), walks: `tpw` tokens' pairs, [tpw][pairs].  Of a single token
// the next one's positions are fetched while this one's heads are worked on.
struct TokenAngles {
    static constexpr int kMost = 4;  // pairs of a lane: 128 of a head
    const RopeParams& r;
    const PairFreq* freqs;
    float2* cs;
    const FastDiv& by_tokens;
    int wpt, tpw, first, gap;
    unsigned total;
    uint32_t pos[kMost];
    __device__ __forceinline__ TokenAngles(const RopeParams& r_, const PairFreq* freqs_, float2* cs_, int id, int wpt_, int tpw_,
                                           unsigned total_, const FastDiv& d)
        : r(r_), freqs(freqs_), cs(cs_), by_tokens(d), wpt(wpt_), tpw(tpw_), first(id * 32 + threadIdx.x % 32), gap(32 * wpt_),
          total(total_) {}
    __device__ __forceinline__ void meet() const {
        if (wpt == 1) __syncwarp();
        else if (wpt == kQkWarps) __syncthreads();
        else named_bar(1 + threadIdx.x / 32 / wpt, wpt * 32);
    }
    __device__ __forceinline__ uint32_t position(unsigned tok, int j) const {
        return position_bits(r, tok, tok - batch_of(tok, by_tokens) * (unsigned)r.tokens, freqs[j].axis());
    }
    __device__ __forceinline__ void fetch(unsigned tok) {
        if (tpw > 1 || tok >= total) return;
#pragma unroll
        for (int k = 0; k < kMost; ++k)
            if (first + k * gap < r.pairs) pos[k] = position(tok, first + k * gap);
    }
    // of tokens tok .. tok + tpw - 1, those that there are
    __device__ __forceinline__ void make(unsigned tok) const {
        meet();  // the tokens before have been read
        if (tpw == 1) {
            if (tok < total) {
#pragma unroll
                for (int k = 0; k < kMost; ++k)
                    if (first + k * gap < r.pairs) cs[first + k * gap] = pair_angle(r, freqs[first + k * gap], pos[k]);
            }
        } else {
            int sub = 0, j = first;
            for (int e = first; e < tpw * r.pairs; e += gap, j += gap) {
                while (j >= r.pairs) j -= r.pairs, ++sub;
                if (tok + sub < total) cs[e] = pair_angle(r, freqs[j], position(tok + sub, j));
            }
        }
        meet();
    }
};

// The heads that a warp works through, of N tensors of one shape (the input, and the
// incoming gradient): those of its share of a token, `step` apart, token after token.
// fetch() brings the next ones, kStages of them ahead of take(), which gives them in
// order.  Lanes whose group has no head at a step, and steps past the last, copy
// nothing.
template <class Head, class T, int N, int kStages>
struct HeadStream {
    static constexpr uint32_t kRound = kStages * N * Head::kSlotBytes;
    const Head& head;
    const QkPlace& place;
    const FastDiv& by_tokens;
    const void* base[N];
    int64_t sb[N], st[N], sh[N];
    const T* at[N];
    int64_t ahead[N];     // elements from a step's head to the next one's
    uint32_t ring;        // this lane's places in the warp's slots
    uint32_t fill, drain;  // the slots in turn, in bytes
    unsigned tok, tokens, total;
    int i, steps, mine;  // step of the token, steps of a token, steps with a head of this lane
    __device__ __forceinline__ HeadStream(const Head& hd, const QkPlace& pl, uint32_t ring_, const RopeParams& r, int heads,
                                          const FastDiv& d)
        : head(hd), place(pl), by_tokens(d), ring(ring_), fill(0), drain(0), tok(pl.tok), tokens((unsigned)r.tokens),
          total((unsigned)(r.batch * r.tokens)), i(0) {
        auto in_steps = [&](int from) { return heads > from ? (heads - from + pl.step - 1) / pl.step : 0; };
        steps = in_steps(pl.h_first);
        mine = pl.part ? in_steps(pl.h0) : 0;
        if (steps == 0) tok = total;  // nothing to fetch
    }
    __device__ __forceinline__ void tensor(int k, const void* p, int64_t b, int64_t t, int64_t h) {
        base[k] = p;
        sb[k] = b, st[k] = t, sh[k] = h;
        ahead[k] = place.step * h;
    }
    __device__ __forceinline__ void aim() {
        if (tok >= total) return;
        const unsigned b = batch_of(tok, by_tokens);
#pragma unroll
        for (int k = 0; k < N; ++k) at[k] = static_cast<const T*>(base[k]) + b * sb[k] + (tok - b * tokens) * st[k] + place.h0 * sh[k];
    }
    __device__ __forceinline__ void next() {
#pragma unroll
        for (int k = 0; k < N; ++k) at[k] += ahead[k];
        if (++i == steps) {
            i = 0;
            tok += place.stride;
            aim();
        }
    }
    __device__ __forceinline__ void fetch() {
        if constexpr (Head::kRing) {
            if (tok < total) {
                if (i < mine) {
#pragma unroll
                    for (int k = 0; k < N; ++k) head.copy(ring + fill + k * Head::kSlotBytes, at[k]);
                }
                next();
            }
            copies_commit();
            fill = fill + N * Head::kSlotBytes == kRound ? 0 : fill + N * Head::kSlotBytes;
        }
    }
    __device__ __forceinline__ void start() {
        aim();
        if constexpr (Head::kRing) {
#pragma unroll 1
            for (int k = 0; k < kStages; ++k) fetch();
        }
    }
    // The values of the next step; call fetch() once they have been used.
    __device__ __forceinline__ void take(typename Head::Raw (&r)[N]) {
        if constexpr (Head::kRing) {
            copies_wait<kStages - 1>();
#pragma unroll
            for (int k = 0; k < N; ++k) head.read(r[k], ring + drain + k * Head::kSlotBytes);
            drain = drain + N * Head::kSlotBytes == kRound ? 0 : drain + N * Head::kSlotBytes;
        } else {
            if (tok < total) {
                if (i < mine) {
#pragma unroll
                    for (int k = 0; k < N; ++k) head.load(r[k], at[k]);
                }
                next();
            }
        }
    }
};

// How a head lies in the lanes: accesses of `w` elements, as wide as divides the head
// and, where pairs lie in halves, the number of pairs; `u` units a lane, kElems
// elements at most, or 12 for units of 4; groups of `g` lanes, a power of two, or as
// many as there are units where more groups fit in a warp so.  The form that leaves the
// fewest of the lanes' places empty, of equal ones the one with the most elements, an
// access of 8 bytes only where it fills an eighth more of them (heads of 96,
// gradients: two groups of 16 lanes with 12 in use 111 us, four of 8 with all).
struct HeadShape {
    int w, u, g;
    bool vec;
};
template <int kElems, int kWidest>  // of a bfloat16 head; a float32 one has accesses of 4
inline HeadShape head_shape(int hd, int n, bool f32, bool interleaved, int align) {
    const int esize = f32 ? 4 : 2;
    HeadShape best = {};
    double most = 0.0;
    for (int w = f32 ? 4 : kWidest; w; w /= 2) {
        if (hd % w || (!interleaved && n % w)) continue;
        if (best.w && w * esize < 8) break;
        const bool one = interleaved && w > 1;  // one access a unit
        const int units = one ? hd / w : n / w + ((hd - 2 * n) / w + 1) / 2, e = one ? w : 2 * w;
        for (int u = 1; u <= 4; ++u) {
            const bool wide = units > 32 * (u == 4 ? 2 : u == 3 ? 2 : u / 2);  // no smaller u takes the head
            if (u == 3 ? kElems != 8 || e != 4 : u > 1 && u * e > kElems && !wide) continue;
            const int lanes = (units + u - 1) / u;
            if (lanes > 32) continue;
            HeadShape s{w, u, 1, align >= w * esize};
            while (s.g < lanes) s.g *= 2;
            if (32 / lanes > 32 / s.g) s.g = lanes;
            const double used = (double)hd * (32 / s.g) / (32 * e * u) * (best.w && w != best.w ? 1.0 / 1.125 : 1.0);
            if (used >= most * (best.w == w ? 1.0 : 1.0001)) {
                most = used;
                best = s;
            }
        }
    }
    return best;
}

// Calls f with a head's shape as types: the element, and Int or Bool of INTERLEAVED, W,
// U, VEC and the group (0: as given).
template <int kElems, int kWidest, bool INTERLEAVED, class F>
cudaError_t for_head_shape(const HeadShape& s, bool f32, F&& f) {
    auto with_g = [&](auto t, auto inter, auto w, auto u, auto v) {
        if constexpr (decltype(v)::value && decltype(w)::value >= 4) {
            if (s.g == 4) return f(t, inter, w, u, v, Int<4>());
            if (s.g == 5) return f(t, inter, w, u, v, Int<5>());
            if (s.g == 6) return f(t, inter, w, u, v, Int<6>());
            if (s.g == 8) return f(t, inter, w, u, v, Int<8>());
            if (s.g == 9) return f(t, inter, w, u, v, Int<9>());
            if (s.g == 10) return f(t, inter, w, u, v, Int<10>());
            if (s.g == 16) return f(t, inter, w, u, v, Int<16>());
            if (s.g == 32) return f(t, inter, w, u, v, Int<32>());
        }
        return f(t, inter, w, u, v, Int<0>());
    };
    auto with_u = [&](auto t, auto inter, auto w, auto v) {
        constexpr int kW = decltype(w)::value, kOne = decltype(inter)::value && kW > 1, kUnit = kOne ? kW : 2 * kW;
        constexpr int kUnits = 256 / kUnit;  // of the largest head
        if (s.u == 1) return with_g(t, inter, w, Int<1>(), v);
        if constexpr (2 * kUnit <= kElems || kUnits > 32)
            if (s.u == 2) return with_g(t, inter, w, Int<2>(), v);
        if constexpr (kElems == 8 && kUnit == 4)
            if (s.u == 3) return with_g(t, inter, w, Int<3>(), v);
        if constexpr (4 * kUnit <= kElems || kUnits > 64)
            if (s.u == 4) return with_g(t, inter, w, Int<4>(), v);
        return cudaErrorInvalidConfiguration;  // not reached
    };
    auto with_v = [&](auto t, auto inter, auto w) {
        return s.vec ? with_u(t, inter, w, Bool<true>()) : with_u(t, inter, w, Bool<false>());
    };
    auto with_w = [&](auto t, auto inter) {
        if constexpr (sizeof(t) == 2 && kWidest == 8)
            if (s.w == 8) return with_v(t, inter, Int<8>());
        if (s.w == 4) return with_v(t, inter, Int<4>());
        if (s.w == 2) return with_v(t, inter, Int<2>());
        return with_u(t, inter, Int<1>(), Bool<true>());
    };
    return f32 ? with_w(0.0f, Bool<INTERLEAVED>()) : with_w((uint16_t)0, Bool<INTERLEAVED>());
}

// Lets a kernel have `bytes` of shared memory.
inline cudaError_t allow_smem(SmemOptIn& opt, const void* kernel, size_t bytes) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    RingShape ring = {};
    ring.stages = 1;
    ring.smem = (int)bytes;
    return opt.allow(kernel, ring);
}

}  // namespace mbx
