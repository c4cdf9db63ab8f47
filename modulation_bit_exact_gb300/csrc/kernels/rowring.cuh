// rowring.cuh -- rows streamed through shared memory for the LayerNorm and
// dropout kernels.
//
// A row group of `tpr` threads (8, 16 or 32 lanes of a warp, or whole warps)
// works on one row at a time (R rows in the LayerNorm forward pass); thread t
// owns the NCH chunks j*tpr + t of it, CE elements each (8 bfloat16 or 4
// binary32: 16 bytes).  Rows arrive by cp.async in a ring of stages, and later
// rows are in flight while a row is reduced.
//
// kVec: rows are 16-byte aligned and their width is a multiple of CE.  Each
// thread copies exactly the chunks that it reads, so its own
// cp.async.wait_group is the only synchronisation.
//
// kShift: any other row.  It is copied by its aligned 16-byte pieces (by 4 bytes
// at its ends, so that nothing outside the row is read) to the same place modulo
// 16 bytes, whatever thread owns the columns; the group meets at a barrier
// before it reads the stage, and a thread takes its chunk out of two neighbouring
// pieces, shifted.  An output row goes the same way back: into the stage that was
// read, a barrier, and out by aligned pieces.  Against single-element loads and
// stores (the columns dealt out one by one) AdaLN's gradients with a modulation row
// each of [32000, 561] bfloat16 rows went from 140 to 107 us and of [57394, 561] from
// 335 to 188 (560 columns, kVec: 44 and 74; into one row 85 and 145, 39 and 61).
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
// again (kVec), so that every stage but that one is always on its way.
__device__ __forceinline__ void ring_wait(int stages) {
    if (stages == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// This thread's place in its row group and the chunks that it owns.
struct Lane {
    int t, tpr, D, bar_id;
    int nv;  // chunks of this thread that hold a column
};
template <int CE>
__device__ __forceinline__ Lane make_lane(int t, int tpr, int D, int bar_id) {
    const int chunks = (D + CE - 1) / CE;
    return Lane{t, tpr, D, bar_id, chunks > t ? (chunks - t + tpr - 1) / tpr : 0};
}
// Columns of chunk j: CE, but for the row's last chunk and beyond it.
template <int CE, Access A>
__device__ __forceinline__ int columns(int j, const Lane& L) {
    return A == kVec ? CE : min(max(L.D - (j * L.tpr + L.t) * CE, 0), CE);
}

// The threads of a row group meet: a named barrier of its warps, or its lanes of
// one warp.
__device__ __forceinline__ void group_sync(const Lane& L) {
    if (L.tpr > 32) named_bar(L.bar_id, L.tpr);
    else if (L.tpr == 32) __syncwarp();
    else __syncwarp(((1u << L.tpr) - 1u) << (threadIdx.x % 32 / L.tpr * L.tpr));
}

// While the previous kernel of the stream drains: bring a row that the ring will
// be filled with first into L2 (L2 is the point of coherence, so a row that the
// previous kernel still writes is the written one there).
template <class Q, Access A>
__device__ __forceinline__ void prefetch_row(const Q* row, int D, int t) {
    if constexpr (A == kVec)
        if (t == 0) prefetch_l2_bulk(row, (uint32_t)(D * (int)sizeof(Q)));
}

// A staged kShift row begins with this, 16 bytes; its element c lies
// `shift` + c * size bytes behind.
struct StagedHead {
    int shift;        // the row's address modulo 16
    const void* row;  // the row in memory
};
static_assert(sizeof(StagedHead) == 16, "");

// Start the copy of this thread's part of a row to its place in a stage; `row`
// points at the row's first element.
template <class Q, int NCH, int CE, Access A>
__device__ __forceinline__ void ring_fill(char* dst, const Q* row, const Lane& L) {
    if constexpr (A == kVec) {
        constexpr int P = CE * (int)sizeof(Q) / 16;  // 16-byte pieces of a chunk
        row += L.t * CE;
#pragma unroll
        for (int j = 0; j < NCH; ++j)
            if (j < L.nv) {
#pragma unroll
                for (int h = 0; h < P; ++h)
                    ring_cp16(dst + ((j * P + h) * L.tpr + L.t) * 16, row + j * L.tpr * CE + h * (16 / (int)sizeof(Q)));
            }
    } else {
        const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 15);
        if (L.t == 0) *reinterpret_cast<StagedHead*>(dst) = StagedHead{shift, row};
        const char* src = reinterpret_cast<const char*>(row) - shift;
        const int end = shift + L.D * (int)sizeof(Q), first = shift ? 16 : 0, last = max(end & ~15, first);
        dst += sizeof(StagedHead);
#pragma unroll
        for (int j = 0; j < NCH * CE * (int)sizeof(Q) / 16; ++j) {
            const int i = first + (j * L.tpr + L.t) * 16;
            if (i < last) ring_cp16(dst + i, src + i);
        }
        // the row's ends by 4 bytes, nothing outside it: four threads each
        const int w = L.t < 4 ? L.t * 4 : last + L.t * 4 - 16;
        if (L.t < 8 && w >= shift && (L.t >= 4 || w < first)) {
            if (w + 4 <= end) ring_cp4(dst + w, src + w);
            else if (sizeof(Q) == 2 && w + 2 <= end) ring_cp2(dst + w, src + w);
        }
    }
}

// Before the first fill.  kVec: zero this thread's places that hold no column and
// that no copy ever writes, so that reading needs no mask.  kShift: a head that
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

// 16 bytes out of the 32 of a and b, from byte r (a multiple of SIZE, below 16).
template <int SIZE>
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int r) {
    const uint32_t in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t u[6], v[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) u[i] = (r & 8) ? in[i + 2] : in[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = (r & 4) ? u[i + 1] : u[i];
    if constexpr (SIZE == 4) return make_uint4(v[0], v[1], v[2], v[3]);
    const uint32_t bits = (r & 2) * 8;
    return make_uint4(__funnelshift_r(v[0], v[1], bits), __funnelshift_r(v[1], v[2], bits),
                      __funnelshift_r(v[2], v[3], bits), __funnelshift_r(v[3], v[4], bits));
}

// Words of a 16-byte piece with its elements from the n-th on zeroed.
template <int SIZE>
__device__ __forceinline__ uint4 first_elements(uint4 v, int n) {
    constexpr int PER = 4 / SIZE;  // elements of a word
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i * PER >= n) w_set(v, i, 0);
        else if (PER == 2 && i * PER + 1 >= n) w_set(v, i, w_of(v, i) & 0xffffu);
    }
    return v;
}

// Piece h (of 16 bytes) of chunk j of a staged row; 0 where no column exists.
template <class Q, int CE, Access A>
__device__ __forceinline__ uint4 ring_piece(const char* src, int j, int h, const Lane& L) {
    constexpr int P = CE * (int)sizeof(Q) / 16, PER = 16 / (int)sizeof(Q);
    if constexpr (A == kVec) {
        return *reinterpret_cast<const uint4*>(src + ((j * P + h) * L.tpr + L.t) * 16);
    } else {
        const StagedHead& head = *reinterpret_cast<const StagedHead*>(src);
        const int i = (j * L.tpr + L.t) * P + h;
        const uint4* q = reinterpret_cast<const uint4*>(src + sizeof(StagedHead)) + i;
        uint4 v = shifted<(int)sizeof(Q)>(q[0], q[1], head.shift);
        // a bfloat16 row that starts in the upper half of a word: cp.async cannot
        // move its first element alone
        if (sizeof(Q) == 2 && i == 0 && (head.shift & 2))
            v.x = (v.x & 0xffff0000u) | ld_u16_rw(head.row);
        const int n = columns<CE, A>(j, L) - h * PER;
        if (n < PER) v = first_elements<(int)sizeof(Q)>(v, n);
        return v;
    }
}

// A 16-byte store that marks its line as streamed.
__device__ __forceinline__ void st_stream(void* p, uint4 v) {
    asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ u64 word_pair(uint32_t a, uint32_t b) { return f2(__uint_as_float(a), __uint_as_float(b)); }

// A staged row as pairs.
template <class Q, int NCH, int CE, Access A>
__device__ __forceinline__ void read_row(u64 (&v)[NCH * CE / 2], const char* src, const Lane& L) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        u64* p = v + j * (CE / 2);
        if constexpr (sizeof(Q) == 2) {
            const uint4 w = ring_piece<Q, CE, A>(src, j, 0, L);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = widen2(w_of(w, i));
        } else {
#pragma unroll
            for (int h = 0; h < CE / 4; ++h) {
                const uint4 w = ring_piece<Q, CE, A>(src, j, h, L);
                p[2 * h] = word_pair(w.x, w.y);
                p[2 * h + 1] = word_pair(w.z, w.w);
            }
        }
    }
}

// A staged row as it came, one 16-byte piece a chunk, widened where it is used.
template <class T, int NCH, Access A>
__device__ __forceinline__ void read_pieces(uint4 (&v)[NCH], const char* src, const Lane& L) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) v[j] = ring_piece<T, ChunkOf<T>::CE, A>(src, j, 0, L);
}
template <class T, int NCH>
__device__ __forceinline__ u64 piece_pair(const uint4 (&v)[NCH], int e) {
    if constexpr (sizeof(T) == 2) return widen2(w_of(v[e / 4], e % 4));
    else return word_pair(w_of(v[e / 2], e % 2 * 2), w_of(v[e / 2], e % 2 * 2 + 1));
}

// v for the columns of pair i of chunk j, 0 for the rest: subtracted from a
// row's 0 there, the mean must leave 0.
template <int CE, Access A>
__device__ __forceinline__ u64 where_column(float v, int j, int i, const Lane& L) {
    if constexpr (A == kVec) {
        const float w = j < L.nv ? v : 0.0f;
        return f2(w, w);
    }
    const int n = columns<CE, A>(j, L);
    return f2(2 * i < n ? v : 0.0f, 2 * i + 1 < n ? v : 0.0f);
}

// Pairs as the 16-byte piece h of a chunk, each element rounded once to Q.
template <class Q, int CE>
__device__ __forceinline__ uint4 narrow(const u64 (&p)[CE / 2], int h) {
    if constexpr (sizeof(Q) == 2) return make_uint4(pack2_rn(p[0]), pack2_rn(p[1]), pack2_rn(p[2]), pack2_rn(p[3]));
    else
        return make_uint4((uint32_t)p[2 * h], (uint32_t)(p[2 * h] >> 32), (uint32_t)p[2 * h + 1],
                          (uint32_t)(p[2 * h + 1] >> 32));
}

// Chunk j of an output row.  kVec: to the row itself (`row` points at its first
// element).  kShift: to `stage`, from where flush_row() moves the row when every
// thread of the group has put its chunks.
template <class Q, int CE, Access A, bool STREAM = false>
__device__ __forceinline__ void put_row_chunk(Q* row, char* stage, const u64 (&p)[CE / 2], int j, const Lane& L) {
    if (j >= L.nv) return;
    constexpr int P = CE * (int)sizeof(Q) / 16;
    const int i = j * L.tpr + L.t;
#pragma unroll
    for (int h = 0; h < P; ++h) {
        if constexpr (A == kVec && STREAM) st_stream(row + i * CE + h * (16 / (int)sizeof(Q)), narrow<Q, CE>(p, h));
        else if constexpr (A == kVec) st_v4(row + i * CE + h * (16 / (int)sizeof(Q)), narrow<Q, CE>(p, h));
        else reinterpret_cast<uint4*>(stage)[i * P + h] = narrow<Q, CE>(p, h);
    }
}
// The same for an output in a parameter's type, bfloat16 or binary32.
template <class T, int CE, Access A, bool STREAM = false>
__device__ __forceinline__ void put_param_row_chunk(void* p, int64_t off, bool p_f32, char* stage,
                                                    const u64 (&v)[CE / 2], int j, const Lane& L) {
    if (sizeof(T) == 4 || p_f32) put_row_chunk<float, CE, A, STREAM>(static_cast<float*>(p) + off, stage, v, j, L);
    else if constexpr (sizeof(T) == 2) put_row_chunk<uint16_t, CE, A, STREAM>(static_cast<uint16_t*>(p) + off, stage, v, j, L);
}

__device__ __forceinline__ void st_bits(uint16_t* p, uint16_t v) { st_u16(p, v); }
__device__ __forceinline__ void st_bits(float* p, float v) { store_elem(p, v); }

// kShift: the row that the group has put into `stage`, out by aligned 16-byte
// pieces and by elements at its ends.  Begins and ends with a barrier: the stage
// is complete, and free again.
template <class Q>
__device__ __forceinline__ void flush_row(Q* row, const char* stage, const Lane& L) {
    group_sync(L);
    constexpr int SIZE = (int)sizeof(Q);
    const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 15);
    const int first = shift ? 16 - shift : 0, last = ((shift + L.D * SIZE) & ~15) - shift;  // of the aligned pieces
#pragma unroll
    for (int j = 0; j < SIZE; ++j) {  // 16 elements a thread
        const int o = first + (j * L.tpr + L.t) * 16;
        if (o < last) {
            const uint4* q = reinterpret_cast<const uint4*>(stage + (o & ~15));
            st_v4(reinterpret_cast<char*>(row) + o, shift ? shifted<SIZE>(q[0], q[1], 16 - shift) : q[0]);
        }
    }
    if (L.t < 8) {  // the ends by elements
        const int head = L.t, tail = max(last, first) / SIZE + L.t;
        const Q* s = reinterpret_cast<const Q*>(stage);
        if (head < first / SIZE && head < L.D) st_bits(row + head, s[head]);
        if (tail < L.D) st_bits(row + tail, s[tail]);
    }
    group_sync(L);
}
template <class T>
__device__ __forceinline__ void flush_param_row(void* p, int64_t off, bool p_f32, const char* stage, const Lane& L) {
    if (sizeof(T) == 4 || p_f32) flush_row(static_cast<float*>(p) + off, stage, L);
    else flush_row(static_cast<uint16_t*>(p) + off, stage, L);
}

// Chunk j of a row that is written once a block (sums of columns); `row` points
// at its first element.
template <class Q, int CE, Access A>
__device__ __forceinline__ void put_chunk(Q* row, const u64 (&p)[CE / 2], int j, const Lane& L) {
    if constexpr (A == kVec) {
        put_row_chunk<Q, CE, A>(row, nullptr, p, j, L);
    } else {
        const int n = columns<CE, A>(j, L);
        row += (j * L.tpr + L.t) * CE;
#pragma unroll
        for (int i = 0; i < CE; ++i)
            if (i < n) store_elem(row + i, i % 2 ? f2hi(p[i / 2]) : f2lo(p[i / 2]));
    }
}
template <class T, int CE, Access A>
__device__ __forceinline__ void put_param_chunk(void* p, int64_t off, bool p_f32, const u64 (&v)[CE / 2], int j,
                                                const Lane& L) {
    if (sizeof(T) == 4 || p_f32) put_chunk<float, CE, A>(static_cast<float*>(p) + off, v, j, L);
    else if constexpr (sizeof(T) == 2) put_chunk<uint16_t, CE, A>(static_cast<uint16_t*>(p) + off, v, j, L);
}

// Chunk j of a parameter's row in memory (no output overlaps it), 0 where no
// column exists; `row` points at its first element.
template <class Q, int CE, Access A>
__device__ __forceinline__ void get_chunk(u64 (&p)[CE / 2], const Q* row, int j, const Lane& L) {
    row += (j * L.tpr + L.t) * CE;
#pragma unroll
    for (int i = 0; i < CE / 2; ++i) p[i] = 0;
    if constexpr (A == kVec) {
        if (j >= L.nv) return;
        if constexpr (sizeof(Q) == 2) {
            const uint4 v = ld_shared_row(row);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = widen2(w_of(v, i));
        } else {
#pragma unroll
            for (int h = 0; h < CE / 4; ++h) {
                const uint4 v = ld_shared_row(row + 4 * h);
                p[2 * h] = word_pair(v.x, v.y);
                p[2 * h + 1] = word_pair(v.z, v.w);
            }
        }
    } else {
        const int n = columns<CE, A>(j, L);
#pragma unroll
        for (int i = 0; i < CE / 2; ++i)
            p[i] = f2(2 * i < n ? load_elem(row + 2 * i) : 0.0f, 2 * i + 1 < n ? load_elem(row + 2 * i + 1) : 0.0f);
    }
}
template <class T, int CE, Access A>
__device__ __forceinline__ void get_param_chunk(u64 (&v)[CE / 2], const void* p, int64_t off, bool p_f32, int j,
                                                const Lane& L) {
    if (sizeof(T) == 4 || p_f32) get_chunk<float, CE, A>(v, static_cast<const float*>(p) + off, j, L);
    else if constexpr (sizeof(T) == 2) get_chunk<uint16_t, CE, A>(v, static_cast<const uint16_t*>(p) + off, j, L);
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
        if constexpr (V == 4) {  // five warps at a time: all 64 values at once spill registers
            const float4* s = reinterpret_cast<const float4*>(slot);
            float4 a = s[0];
#pragma unroll 5
            for (int i = 1; i < W; ++i) {
                const float4 q = s[i];
                a = make_float4(a.x + q.x, a.y + q.y, a.z + q.z, a.w + q.w);
            }
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            return;
        }
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
