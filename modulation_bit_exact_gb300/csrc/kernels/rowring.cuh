// rowring.cuh -- rows streamed through shared memory for the LayerNorm kernels.
//
// A row group of `tpr` threads (8, 16 or 32 lanes of a warp, or whole warps)
// works on R rows at a time; thread t owns E = NCH*CE columns of every row.
// Rows arrive by cp.async in a ring of stages, and later rows are in flight
// while a row is reduced.
//
// kVec: chunk j of thread t is columns (j*tpr + t)*CE ..., moved in 16-byte
// pieces.  Each thread copies exactly the pieces that it reads, so its own
// cp.async.wait_group is the only synchronisation.
//
// kScalar (a width that is no multiple of CE, or a row that starts at no 16-byte
// boundary): element e is column e*tpr + t.  The row is copied by its aligned
// 16-byte pieces, and by 4 bytes at its ends, to the same place modulo 16 bytes,
// whatever thread owns the columns; so the group meets at a barrier before it
// reads a stage, and again before the stage is filled anew.  Copied element by
// element instead, [57394, 561] bfloat16 gradients took 335 us, now TIME us.
// kQuad is kScalar with four consecutive columns of a thread at a time, which
// share one call of the dropout generator.
#pragma once

#include "rowgroup.cuh"

namespace mbx {

__device__ __forceinline__ void ring_cp16(void* dst, const void* src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void ring_cp4(void* dst, const void* src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}
// The first 2 of 4 bytes; the others are zeroed in shared memory and not read.
__device__ __forceinline__ void ring_cp2(void* dst, const void* src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, 2;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest stages-1 groups have landed (stages <= 4): the oldest
// stage is ready.  Its rows go to registers at once and the stage is filled
// again, so that every stage but that one is always on its way.
__device__ __forceinline__ void ring_wait(int stages) {
    if (stages == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// This thread's place in its row group and the columns that it owns.
struct Lane {
    int t, tpr, D;
    int nv;  // kVec: chunks that exist; else elements that exist
};
template <int E, int CE, Access A>
__device__ __forceinline__ Lane make_lane(int t, int tpr, int D) {
    int nv = 0;
    if constexpr (A == kQuad) {
#pragma unroll
        for (int q = 0; q < E / 4; ++q) nv += min(max(D - (q * tpr + t) * 4, 0), 4);
    } else {
        const int units = A == kVec ? D / CE : D;
        nv = units > t ? (units - t + tpr - 1) / tpr : 0;
    }
    return Lane{t, tpr, D, nv};
}
// This thread's first column, and how far element e lies beyond it.
template <int CE, Access A>
__device__ __forceinline__ int first_col(const Lane& L) {
    return A == kVec ? L.t * CE : A == kQuad ? L.t * 4 : L.t;
}
template <Access A>
__device__ __forceinline__ int elem_off(int e, const Lane& L) {
    return A == kQuad ? e / 4 * L.tpr * 4 + e % 4 : e * L.tpr;
}

// While the previous kernel of the stream drains: bring a row that the ring will
// be filled with first into L2 (L2 is the point of coherence, so a row that the
// previous kernel still writes is the written one there).
template <class Q, Access A>
__device__ __forceinline__ void prefetch_row(const Q* row, int D, int t) {
    if constexpr (A == kVec)
        if (t == 0) prefetch_l2_bulk(row, (uint32_t)(D * (int)sizeof(Q)));
}

// A staged row that is not kVec begins with this, 16 bytes; its element c lies
// `shift` + c * size bytes behind.
struct StagedHead {
    int shift;       // the row's address modulo 16
    const void* row;  // the row in memory
};
static_assert(sizeof(StagedHead) == 16, "");

// Start the copy of this thread's part of a row to its place in a stage; `row`
// points at its first column.
template <class Q, int NCH, int CE, Access A>
__device__ __forceinline__ void ring_fill(char* dst, const Q* row, const Lane& L) {
    if constexpr (A == kVec) {
        constexpr int P = CE * (int)sizeof(Q) / 16;  // 16-byte pieces of a chunk
#pragma unroll
        for (int j = 0; j < NCH; ++j)
            if (j < L.nv) {
#pragma unroll
                for (int h = 0; h < P; ++h)
                    ring_cp16(dst + ((j * P + h) * L.tpr + L.t) * 16, row + j * L.tpr * CE + h * (16 / (int)sizeof(Q)));
            }
    } else {
        const Q* start = row - first_col<CE, A>(L);
        const int shift = (int)(reinterpret_cast<uintptr_t>(start) & 15);
        if (L.t == 0) *reinterpret_cast<StagedHead*>(dst) = StagedHead{shift, start};
        const char* src = reinterpret_cast<const char*>(start) - shift;
        const int end = shift + L.D * (int)sizeof(Q);
        dst += sizeof(StagedHead);
        for (int i = L.t * 16; i < end; i += L.tpr * 16) {
            if (i >= shift && i + 16 <= end) {
                ring_cp16(dst + i, src + i);
                continue;
            }
#pragma unroll
            for (int w = i; w < i + 16; w += 4) {  // an end of the row: nothing outside it is read
                if (w >= shift && w + 4 <= end) ring_cp4(dst + w, src + w);
                else if (sizeof(Q) == 2 && w >= shift && w + 2 <= end) ring_cp2(dst + w, src + w);
            }
        }
    }
}

// Whether a thread reads what others copied (and the group must meet first).
template <Access A>
constexpr bool kShared = A != kVec;

// Chunk j of a staged row as CE/2 pairs (0 where no column exists; kVec: see
// ring_clear).
template <class Q, int CE, Access A>
__device__ __forceinline__ void ring_read(u64 (&p)[CE / 2], const char* src, int j, const Lane& L) {
    if constexpr (A == kVec) {
        if constexpr (sizeof(Q) == 2) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + (j * L.tpr + L.t) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = widen2(w_of(v, i));
        } else {
#pragma unroll
            for (int h = 0; h < CE / 4; ++h) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(src + ((j * (CE / 4) + h) * L.tpr + L.t) * 16);
                p[2 * h] = v.x;
                p[2 * h + 1] = v.y;
            }
        }
    } else {
        const StagedHead& head = *reinterpret_cast<const StagedHead*>(src);
        const Q* row = reinterpret_cast<const Q*>(src + sizeof(StagedHead) + head.shift) + first_col<CE, A>(L);
#pragma unroll
        for (int i = 0; i < CE; i += 2) {
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int e = j * CE + i + h;
                v[h] = 0.0f;
                if (e < L.nv) {
                    if constexpr (sizeof(Q) == 4) v[h] = row[elem_off<A>(e, L)];
                    else v[h] = __uint_as_float((uint32_t)row[elem_off<A>(e, L)] << 16);
                }
                // a bfloat16 row that starts in the upper half of a word: cp.async
                // cannot move its first element alone
                if (sizeof(Q) == 2 && e == 0 && L.t == 0 && (head.shift & 2))
                    v[h] = load_elem(static_cast<const Q*>(head.row));
            }
            p[i / 2] = f2(v[0], v[1]);
        }
    }
}

// Before the first fill.  kVec: zero this thread's places that hold no column and
// that no copy ever writes, so that reading needs no mask.  Else: a head that
// points nowhere, for a group that has no row in a round and reads the stage all
// the same.
template <class Q, int NCH, int CE, Access A>
__device__ __forceinline__ void ring_clear(char* dst, const Lane& L) {
    if constexpr (A == kVec) {
        constexpr int P = CE * (int)sizeof(Q) / 16;
        for (int j = L.nv; j < NCH; ++j)
            for (int h = 0; h < P; ++h)
                *reinterpret_cast<uint4*>(dst + ((j * P + h) * L.tpr + L.t) * 16) = make_uint4(0, 0, 0, 0);
    } else if (L.t == 0) {
        *reinterpret_cast<StagedHead*>(dst) = StagedHead{0, nullptr};
    }
}

// A staged row as pairs.
template <class Q, int NCH, int CE, Access A>
__device__ __forceinline__ void read_row(u64 (&v)[NCH * CE / 2], const char* src, const Lane& L) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        u64 c[CE / 2];
        ring_read<Q, CE, A>(c, src, j, L);
#pragma unroll
        for (int i = 0; i < CE / 2; ++i) v[j * (CE / 2) + i] = c[i];
    }
}

// v for the columns of pair i of chunk j, 0 for the rest: subtracted from a
// row's 0 there, the mean must leave 0.
template <int CE, Access A>
__device__ __forceinline__ u64 where_column(float v, int j, int i, const Lane& L) {
    if constexpr (A == kVec) {
        const float w = j < L.nv ? v : 0.0f;
        return f2(w, w);
    }
    const int e = j * CE + 2 * i;
    return f2(e < L.nv ? v : 0.0f, e + 1 < L.nv ? v : 0.0f);
}

// Whether chunk j is stored (kScalar masks its elements instead).
template <Access A>
__device__ __forceinline__ bool has_chunk(int j, const Lane& L) {
    return A == kVec ? j < L.nv : true;
}

// A staged row as it came, widened where it is used: 16-byte pieces of T, or
// (kScalar) single elements packed the same way.
template <class T, int NCH, Access A>
__device__ __forceinline__ void read_pieces(uint4 (&v)[NCH], const char* src, const Lane& L) {
    constexpr int CE = ChunkOf<T>::CE;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        if constexpr (A == kVec) {
            v[j] = *reinterpret_cast<const uint4*>(src + (j * L.tpr + L.t) * 16);
        } else {
            u64 c[CE / 2];
            ring_read<T, CE, A>(c, src, j, L);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) w_set(v[j], i, pack2_rn(c[i]));
                else w_set(v[j], i, (uint32_t)(c[i / 2] >> (i % 2 * 32)));
            }
        }
    }
}
template <class T, int NCH>
__device__ __forceinline__ u64 piece_pair(const uint4 (&v)[NCH], int e) {
    if constexpr (sizeof(T) == 2) return widen2(w_of(v[e / 4], e % 4));
    else return f2(__uint_as_float(w_of(v[e / 2], e % 2 * 2)), __uint_as_float(w_of(v[e / 2], e % 2 * 2 + 1)));
}

// Chunk j to a row in memory, each element rounded once to Q; `row` points at
// the thread's first column.
template <class Q, int CE, Access A>
__device__ __forceinline__ void put_chunk(Q* row, const u64 (&p)[CE / 2], int j, const Lane& L) {
    if constexpr (A == kVec) {
        Q* d = row + j * L.tpr * CE;
        if constexpr (sizeof(Q) == 2) {
            st_v4(d, make_uint4(pack2_rn(p[0]), pack2_rn(p[1]), pack2_rn(p[2]), pack2_rn(p[3])));
        } else {
#pragma unroll
            for (int h = 0; h < CE / 4; ++h)
                st_v4(d + 4 * h, make_uint4((uint32_t)p[2 * h], (uint32_t)(p[2 * h] >> 32), (uint32_t)p[2 * h + 1],
                                            (uint32_t)(p[2 * h + 1] >> 32)));
        }
    } else {
#pragma unroll
        for (int i = 0; i < CE; ++i) {
            const int e = j * CE + i;
            if (e < L.nv) store_elem(row + elem_off<A>(e, L), i % 2 ? f2hi(p[i / 2]) : f2lo(p[i / 2]));
        }
    }
}
// The same for a parameter's row, bfloat16 or binary32 whatever the rows are.
template <class T, int CE, Access A>
__device__ __forceinline__ void put_param_chunk(void* p, int64_t off, bool p_f32, const u64 (&v)[CE / 2], int j,
                                                const Lane& L) {
    if constexpr (sizeof(T) == 4) put_chunk<float, CE, A>(static_cast<float*>(p) + off, v, j, L);
    else if (p_f32) put_chunk<float, CE, A>(static_cast<float*>(p) + off, v, j, L);
    else put_chunk<uint16_t, CE, A>(static_cast<uint16_t*>(p) + off, v, j, L);
}

// Chunk j of a row in memory, 0 where no column exists.  For
// parameters, which no output overlaps.
template <class Q, int CE, Access A>
__device__ __forceinline__ void get_chunk(u64 (&p)[CE / 2], const Q* row, int j, const Lane& L) {
    if constexpr (A == kVec) {
#pragma unroll
        for (int i = 0; i < CE / 2; ++i) p[i] = 0;
        if (j < L.nv) {
            const Q* s = row + j * L.tpr * CE;
            if constexpr (sizeof(Q) == 2) {
                const uint4 v = ld_shared_row(s);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = widen2(w_of(v, i));
            } else {
#pragma unroll
                for (int h = 0; h < CE / 4; ++h) {
                    const uint4 v = ld_shared_row(s + 4 * h);
                    p[2 * h] = f2(__uint_as_float(v.x), __uint_as_float(v.y));
                    p[2 * h + 1] = f2(__uint_as_float(v.z), __uint_as_float(v.w));
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < CE; i += 2) {
            const int e = j * CE + i;
            p[i / 2] = f2(e < L.nv ? load_elem(row + elem_off<A>(e, L)) : 0.0f,
                          e + 1 < L.nv ? load_elem(row + elem_off<A>(e + 1, L)) : 0.0f);
        }
    }
}
template <class T, int CE, Access A>
__device__ __forceinline__ void get_param_chunk(u64 (&v)[CE / 2], const void* p, int64_t off, bool p_f32, int j,
                                                const Lane& L) {
    if constexpr (sizeof(T) == 4) get_chunk<float, CE, A>(v, static_cast<const float*>(p) + off, j, L);
    else if (p_f32) get_chunk<float, CE, A>(v, static_cast<const float*>(p) + off, j, L);
    else get_chunk<uint16_t, CE, A>(v, static_cast<const uint16_t*>(p) + off, j, L);
}

// The threads of a row group meet: a named barrier of its warps, or its lanes of
// one warp.
__device__ __forceinline__ void group_sync(int tpr, int bar_id) {
    if (tpr > 32) named_bar(bar_id, tpr);
    else if (tpr == 32) __syncwarp();
    else __syncwarp(((1u << tpr) - 1u) << (threadIdx.x % 32 / tpr * tpr));
}

// Sums of V values (a power of two, at most 4) over a row group, in every
// thread.  Inside a warp the first log2(V) shuffle steps halve the number of
// values that a lane carries, so that V sums take about V + log2(lanes)
// shuffles instead of V*log2(lanes); then the warps' sums meet in shared
// memory, one barrier, and every thread adds them in warp order (reading them
// all costs less time than five more dependent shuffles).  The published sums
// alternate between two buffers: a buffer is written again two calls later,
// after the barrier of the call in between, which every reader has passed.
struct GroupSums {
    float* buf;  // [2][kMaxWarpsPerRow][4] of this group, zeroed
    int t, tpr, bar_id, par;
    template <int V>
    __device__ __forceinline__ void operator()(float (&v)[V]) {
        if (tpr >= 32) run<V, 32>(v);
        else if (tpr == 16) run<V, 16>(v);
        else run<V, 8>(v);
    }

    // The sums of W published warps (those that are not there hold 0).
    template <int V, int W>
    __device__ __forceinline__ void add_warps(float (&v)[V], const float* slot) {
        float r[W * V];
#pragma unroll
        for (int i = 0; i < W * V; i += 4) {
            const float4 q = *reinterpret_cast<const float4*>(slot + i);
            r[i] = q.x;
            r[i + 1] = q.y;
            r[i + 2] = q.z;
            r[i + 3] = q.w;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = r[k];
#pragma unroll
        for (int i = V; i < W * V; ++i) v[i % V] += r[i];
    }

    template <int V, int LANES>
    __device__ __forceinline__ void run(float (&v)[V]) {
        const int lane = t % LANES;
        float c[V];
#pragma unroll
        for (int k = 0; k < V; ++k) c[k] = v[k];
        constexpr int kPer = LANES / V;  // lanes that end up with the same value
#pragma unroll
        for (int n = V / 2, s = LANES / 2; n >= 1; n /= 2, s /= 2) {
            const bool hi = lane & s;
#pragma unroll
            for (int k = 0; k < n; ++k) {
                const float give = hi ? c[k] : c[k + n], keep = hi ? c[k + n] : c[k];
                c[k] = keep + __shfl_xor_sync(0xffffffffu, give, s);
            }
        }
        float a = c[0];  // of value lane / kPer, over the lanes that differ in the bits above
#pragma unroll
        for (int s = kPer / 2; s >= 1; s /= 2) a += __shfl_xor_sync(0xffffffffu, a, s);
        if constexpr (LANES == 32) {
            if (tpr > 32) {
                float* slot = buf + par * 4 * kMaxWarpsPerRow;
                par ^= 1;
                if (lane % kPer == 0) slot[t / 32 * V + lane / kPer] = a;
                named_bar(bar_id, tpr);
                if (tpr <= 128) add_warps<V, 4>(v, slot);
                else if (tpr <= 256) add_warps<V, 8>(v, slot);
                else add_warps<V, 16>(v, slot);
                return;
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = __shfl_sync(0xffffffffu, a, k * kPer, LANES);
    }
};
constexpr int kSumFloats = 2 * 4 * kMaxWarpsPerRow;  // of one group

}  // namespace mbx
