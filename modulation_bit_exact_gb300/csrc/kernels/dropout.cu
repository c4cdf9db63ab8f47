// dropout.cu -- dropout whose mask is a function of a counter, alone or in the
// gated residual, and the gradients of the latter.
//
// keep(r, c): word c mod 4 of Philox4x32-10 (Salmon, Moraes, Dror & Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011) with the key rng[0]
// and the counter (c / 4, r, rng[1] + offset) is at least floor(p * 2^32).  It
// depends on the row and column alone, not on strides, threads or launches, so
// the backward pass forms the same mask again and nothing is stored.
//
//   dropout:       out = keep ? x / (1-p) : 0
//   gated add:     out = keep ? x + gate * y / (1-p) : x
//   its gradients: dy = keep ? dout * gate / (1-p) : 0
//                  dgate = sum over the gate's rows of keep ? dout * y / (1-p) : 0
//
// A dropped element contributes nothing: it is selected away, so an infinity
// or a NaN in its y or gate does not reach an output.  binary32 throughout,
// one rounding at each output.
#include "rowring.cuh"

namespace mbx {

// Philox4x32-10 for the quads (four columns) that a thread keeps for many rows.
// A round maps (w0, w1, w2, w3) to (hi(b)^w1^k0, lo(b), hi(a)^w3^k1, lo(a)) with
// a = M0*w0, b = M1*w2.  The counter's words are (quad, row, c2, c3), so after
// the first round w0 depends on the row alone and w2, w3 on the quad alone;
// followed through, what depends on one of them alone can be formed once for
// it, and a call is left with 15 of the 20 products, which bound this kernel.
constexpr uint32_t kM0 = 0xD2511F53u, kM1 = 0xCD9E8D57u, kW0 = 0x9E3779B9u, kW1 = 0xBB67AE85u;

__device__ __forceinline__ uint32_t hi32(uint64_t v) { return (uint32_t)(v >> 32); }

template <int NQ>
struct Philox {
    uint32_t k0[7], k1[7];               // keys of rounds 3 to 9 (counted from 0)
    uint32_t base;                       // round 0: w0 = base ^ row
    uint32_t c[NQ], d[NQ], e[NQ], f[NQ];  // of each quad
    uint64_t a;                          // M0 * (base ^ row)

    __device__ __forceinline__ Philox(const DropParams& p, const uint32_t (&quad)[NQ]) {
        const uint64_t seed = (uint64_t)p.rng[0], ctr = (uint64_t)p.rng[1] + (uint64_t)p.offset;
        const uint32_t s0 = (uint32_t)seed, s1 = hi32(seed), c2 = (uint32_t)ctr, c3 = hi32(ctr);
#pragma unroll
        for (int r = 0; r < 7; ++r) {
            k0[r] = s0 + (r + 3) * kW0;
            k1[r] = s1 + (r + 3) * kW1;
            // kept in registers: formed again at every use they would be a
            // third of the generator's instructions
            asm volatile("" : "+r"(k0[r]), "+r"(k1[r]));
        }
        const uint64_t b0 = (uint64_t)kM1 * c2;
        base = hi32(b0) ^ s0;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const uint64_t a0 = (uint64_t)kM0 * quad[q], b1 = (uint64_t)kM1 * (hi32(a0) ^ c3 ^ s1);
            const uint64_t a2 = (uint64_t)kM0 * (hi32(b1) ^ (uint32_t)b0 ^ (s0 + kW0));
            c[q] = (uint32_t)a0 ^ (s1 + kW1);
            d[q] = hi32(a2) ^ (s1 + 2 * kW1);
            e[q] = (uint32_t)a2;
            f[q] = (uint32_t)b1 ^ (s0 + 2 * kW0);
            asm volatile("" : "+r"(c[q]), "+r"(d[q]), "+r"(e[q]), "+r"(f[q]));
        }
    }
    __device__ __forceinline__ void row(uint32_t r) { a = (uint64_t)kM0 * (base ^ r); }
    // The four words of quad q of the row.
    __device__ __forceinline__ uint4 operator()(int q) const {
        const uint64_t b2 = (uint64_t)kM1 * (hi32(a) ^ c[q]);  // rounds 1 and 2
        uint32_t w0 = hi32(b2) ^ f[q], w1 = (uint32_t)b2, w2 = d[q] ^ (uint32_t)a, w3 = e[q];
#pragma unroll
        for (int r = 0; r < 7; ++r) {
            const uint64_t x = (uint64_t)kM0 * w0, y = (uint64_t)kM1 * w2;
            w0 = hi32(y) ^ w1 ^ k0[r];
            w1 = (uint32_t)y;
            w2 = hi32(x) ^ w3 ^ k1[r];
            w3 = (uint32_t)x;
        }
        return make_uint4(w0, w1, w2, w3);
    }
};

// A thread's quads: column / 4 of its elements 4i .. 4i+3.
template <int NQ, int CE, Access A>
__device__ __forceinline__ Philox<NQ> make_philox(const DropParams& p, const Lane& L) {
    static_assert(A != kScalar, "four columns of a thread are consecutive");
    uint32_t quad[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i)
        quad[i] = A == kVec && CE == 8 ? (uint32_t)(i / 2 * L.tpr + L.t) * 2 + i % 2 : (uint32_t)(i * L.tpr + L.t);
    return Philox<NQ>(p, quad);
}

// v where the element is kept, else 0.
__device__ __forceinline__ u64 keep_pair(u64 v, uint32_t a, uint32_t b, uint32_t threshold) {
    return f2(a >= threshold ? f2lo(v) : 0.0f, b >= threshold ? f2hi(v) : 0.0f);
}
// acc + v * w where the element is kept, else acc.
__device__ __forceinline__ u64 keep_fma(u64 v, u64 w, u64 acc, uint32_t a, uint32_t b, uint32_t threshold) {
    float lo = f2lo(acc), hi = f2hi(acc);
    if (a >= threshold) lo = fmaf(f2lo(v), f2lo(w), lo);
    if (b >= threshold) hi = fmaf(f2hi(v), f2hi(w), hi);
    return f2(lo, hi);
}

// GATED: out = x + gate * drop(y); otherwise out = drop(x).  Rows stream
// through a ring (rowring.cuh).
template <class T, int NCH, Access A, bool GATED>
__global__ void __launch_bounds__(kRingThreads) dropout_kernel(DropParams p, RingShape sh) {
    constexpr int CE = ChunkOf<T>::CE, H = CE / 2, P = NCH * H;
    extern __shared__ __align__(16) char smem[];
    const int tpr = sh.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const Lane L = make_lane<16, CE, A>(t, tpr, p.D);
    char* ring = smem + g * sh.group_bytes;
    const int64_t step = (int64_t)gridDim.x * sh.groups;
    int64_t row = (int64_t)blockIdx.x * sh.groups + g, fill_row = row;
    if (row < p.rows) {
        prefetch_row<T, A>(static_cast<const T*>(p.x) + row * p.x_stride, p.D, t);
        if constexpr (GATED) prefetch_row<T, A>(static_cast<const T*>(p.y) + row * p.y_stride, p.D, t);
    }
    grid_dep_wait();  // launched programmatically: the previous kernel has finished
    grid_dep_launch();
    Philox<P / 2> philox = make_philox<P / 2, CE, A>(p, L);
    const int row_bytes = sh.row_bytes, stage_bytes = (GATED ? 2 : 1) * row_bytes, c0 = first_col<CE, A>(L);
    auto fill = [&](int st) {
        char* dst = ring + st * stage_bytes;
        if (fill_row < p.rows) {
            ring_fill<T, NCH, CE, A>(dst, static_cast<const T*>(p.x) + fill_row * p.x_stride + c0, L);
            if constexpr (GATED)
                ring_fill<T, NCH, CE, A>(dst + row_bytes, static_cast<const T*>(p.y) + fill_row * p.y_stride + c0, L);
        }
        fill_row += step;
        ring_commit();
    };
    for (int i = 0; i < sh.stages; ++i) fill(i);
    u64 gate[GATED ? P : 1];  // gate / (1-p)
    int64_t seg_end = 0;  // the rows below it share the gate that is loaded
    int stage = 0;
    const u64 inv = f2(p.inv_keep, p.inv_keep);
    for (; row < p.rows; row += step) {
        if constexpr (GATED) {
            if (row >= seg_end) {
                const int64_t m = p.mod_rows == p.rows ? row : row / p.seq;
                seg_end = (m + 1) * p.seq;
#pragma unroll
                for (int j = 0; j < NCH; ++j) {
                    u64 c[H];
                    get_param_chunk<T, CE, A>(c, p.gate, m * p.gate_stride + c0, p.p_f32, j, L);
#pragma unroll
                    for (int i = 0; i < H; ++i) gate[j * H + i] = mul2(c[i], inv);
                }
            }
        }
        ring_wait(sh.stages);
        if constexpr (kShared<A>) group_sync(tpr, g + 1);
        uint4 xr[NCH], yr[GATED ? NCH : 1];
        read_pieces<T, NCH, A>(xr, ring + stage * stage_bytes, L);
        if constexpr (GATED) read_pieces<T, NCH, A>(yr, ring + stage * stage_bytes + row_bytes, L);
        if constexpr (kShared<A>) group_sync(tpr, g + 1);  // every thread has read the stage
        fill(stage);
        if (++stage == sh.stages) stage = 0;
        philox.row((uint32_t)row);
        T* dst = static_cast<T*>(p.out) + row * p.out_stride + c0;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            u64 o[H];
#pragma unroll
            for (int i = 0; i < H; i += 2) {
                const int e = j * H + i;
                const uint4 w = philox(e / 2);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w0 = h ? w.z : w.x, w1 = h ? w.w : w.y;
                    const u64 x = piece_pair<T>(xr, e + h);
                    if constexpr (GATED)
                        o[i + h] = keep_fma(piece_pair<T>(yr, e + h), gate[e + h], x, w0, w1, p.threshold);
                    else o[i + h] = keep_pair(mul2(x, inv), w0, w1, p.threshold);
                }
            }
            if (has_chunk<A>(j, L)) put_chunk<T, CE, A>(dst, o, j, L);
        }
    }
}

// The gradients.  TOKEN: one gate row for every row, and dgate is a row too.
// Otherwise the parts of a segment as in the gradients of LayerNorm's
// parameters (layernorm_bwd.cu): every thread sums its own columns.
template <class T, int NCH, Access A, bool TOKEN>
__global__ void __launch_bounds__(kGradThreads) dropout_backward_kernel(DropParams p, RingShape sh) {
    constexpr int CE = ChunkOf<T>::CE, H = CE / 2, P = NCH * H;
    extern __shared__ __align__(16) char smem[];
    const int tpr = sh.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr, groups = sh.groups;
    const Lane L = make_lane<16, CE, A>(t, tpr, p.D);
    char* ring = smem + g * sh.group_bytes;
    {
        int64_t r = (int64_t)blockIdx.x * groups + g;
        if constexpr (!TOKEN) {
            const int64_t seg = blockIdx.x / p.plan.parts;
            r = seg * p.seq + (blockIdx.x - seg * p.plan.parts) * p.plan.rows_per_part + g;
        }
        if (r < p.rows) {
            prefetch_row<T, A>(static_cast<const T*>(p.x) + r * p.x_stride, p.D, t);
            prefetch_row<T, A>(static_cast<const T*>(p.y) + r * p.y_stride, p.D, t);
        }
    }
    grid_dep_wait();
    grid_dep_launch();
    Philox<P / 2> philox = make_philox<P / 2, CE, A>(p, L);
    const int row_bytes = sh.row_bytes, stage_bytes = 2 * row_bytes, c0 = first_col<CE, A>(L);
    const u64 inv = f2(p.inv_keep, p.inv_keep);
    const int64_t units = TOKEN ? 1 : p.mod_rows * p.plan.parts;
    for (int64_t unit = TOKEN ? 0 : blockIdx.x; unit < units; unit += gridDim.x) {
        int64_t seg = 0, row, end, step;
        if constexpr (TOKEN) {
            row = (int64_t)blockIdx.x * groups + g;
            end = p.rows;
            step = (int64_t)gridDim.x * groups;
        } else {
            seg = unit / p.plan.parts;
            const int64_t r0 = seg * p.seq + (unit - seg * p.plan.parts) * p.plan.rows_per_part;
            end = min(r0 + p.plan.rows_per_part, (seg + 1) * p.seq);
            row = r0 + g;
            step = groups;
        }
        int64_t fill_row = row;
        auto fill = [&](int st) {
            char* dst = ring + st * stage_bytes;
            if (fill_row < end) {
                ring_fill<T, NCH, CE, A>(dst, static_cast<const T*>(p.x) + fill_row * p.x_stride + c0, L);
                ring_fill<T, NCH, CE, A>(dst + row_bytes, static_cast<const T*>(p.y) + fill_row * p.y_stride + c0, L);
            }
            fill_row += step;
            ring_commit();
        };
        for (int i = 0; i < sh.stages; ++i) fill(i);
        u64 gate[P], acc[P];
        auto load_gate = [&](int64_t m) {
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                u64 c[H];
                get_param_chunk<T, CE, A>(c, p.gate, m * p.gate_stride + c0, p.p_f32, j, L);
#pragma unroll
                for (int i = 0; i < H; ++i) gate[j * H + i] = mul2(c[i], inv);
            }
        };
        if constexpr (!TOKEN) {
            load_gate(seg);
#pragma unroll
            for (int e = 0; e < P; ++e) acc[e] = 0;
        }
        int stage = 0;
        for (; row < end; row += step) {
            if constexpr (TOKEN) load_gate(row);
            ring_wait(sh.stages);
            if constexpr (kShared<A>) group_sync(tpr, g + 1);
            uint4 dr[NCH], yr[NCH];
            read_pieces<T, NCH, A>(dr, ring + stage * stage_bytes, L);
            read_pieces<T, NCH, A>(yr, ring + stage * stage_bytes + row_bytes, L);
            if constexpr (kShared<A>) group_sync(tpr, g + 1);  // every thread has read the stage
            fill(stage);
            if (++stage == sh.stages) stage = 0;
            philox.row((uint32_t)row);
            T* dst = static_cast<T*>(p.out) + row * p.out_stride + c0;
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                u64 o[H], og[H];
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const int e = j * H + i;
                    const uint4 w = philox(e / 2);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w0 = h ? w.z : w.x, w1 = h ? w.w : w.y;
                        const u64 d = piece_pair<T>(dr, e + h);
                        const u64 y = piece_pair<T>(yr, e + h);
                        o[i + h] = keep_pair(mul2(d, gate[e + h]), w0, w1, p.threshold);
                        if constexpr (TOKEN) og[i + h] = keep_pair(mul2(mul2(d, inv), y), w0, w1, p.threshold);
                        else acc[e + h] = keep_fma(d, y, acc[e + h], w0, w1, p.threshold);
                    }
                }
                if (!has_chunk<A>(j, L)) continue;
                put_chunk<T, CE, A>(dst, o, j, L);
                if constexpr (TOKEN)
                    if (p.dgate) put_param_chunk<T, CE, A>(p.dgate, row * p.dgate_stride + c0, p.p_f32, og, j, L);
            }
        }
        if constexpr (!TOKEN) {
            if (p.dgate == nullptr) continue;
            if (groups > 1) {
                u64* sums = reinterpret_cast<u64*>(smem);  // [P][block], in the place of the drained ring
                const int n = groups * tpr;
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                __syncthreads();
#pragma unroll
                for (int e = 0; e < P; ++e) sums[e * n + threadIdx.x] = acc[e];
                __syncthreads();
                if (g == 0) {
#pragma unroll
                    for (int e = 0; e < P; ++e)
                        for (int k = 1; k < groups; ++k) acc[e] = add2(acc[e], sums[e * n + k * tpr + t]);
                }
                __syncthreads();
            }
            if (g == 0) {
#pragma unroll
                for (int j = 0; j < NCH; ++j) {
                    if (!has_chunk<A>(j, L)) continue;
                    u64 c[H];
#pragma unroll
                    for (int i = 0; i < H; ++i) c[i] = mul2(acc[j * H + i], inv);
                    if (p.plan.parts == 1)
                        put_param_chunk<T, CE, A>(p.dgate, seg * p.dgate_stride + c0, p.p_f32, c, j, L);
                    else put_chunk<float, CE, A>(p.ws + unit * p.D + c0, c, j, L);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- launch

template <class T, int NCH, Access A, bool GATED>
static cudaError_t drop_fwd(const DropParams& p, cudaStream_t s) {
    auto k = dropout_kernel<T, NCH, A, GATED>;
    const int tpr = row_threads(p.D);
    RingShape sh = ring_shape(tpr, staged_row_bytes(tpr, (int)sizeof(T), A == kVec), GATED ? 2 : 1, 0, 0, kRingThreads, 2);
    sh.smem -= sh.sums_bytes;  // no row sums
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.allow(reinterpret_cast<const void*>(k), sh)) return e;
    const int64_t need = (p.rows + sh.groups - 1) / sh.groups, most = (int64_t)sm_count() * sh.ctas_per_sm;
    return launch_pdl(k, (unsigned)(need < most ? need : most), sh.groups * tpr, sh.smem, s, p, sh);
}

template <class T, int NCH>
static cudaError_t drop_fwd_any(const DropParams& p, bool vec, cudaStream_t s) {
    if (vec) return p.gate ? drop_fwd<T, NCH, kVec, true>(p, s) : drop_fwd<T, NCH, kVec, false>(p, s);
    return p.gate ? drop_fwd<T, NCH, kQuad, true>(p, s) : drop_fwd<T, NCH, kQuad, false>(p, s);
}

cudaError_t launch_dropout(const DropParams& p, bool f32, bool vec, cudaStream_t s) {
    return f32 ? drop_fwd_any<float, 4>(p, vec, s) : drop_fwd_any<uint16_t, 2>(p, vec, s);
}

template <class T, int NCH, Access A, bool TOKEN>
static cudaError_t drop_bwd(const DropParams& p0, cudaStream_t s) {
    DropParams p = p0;
    auto k = dropout_backward_kernel<T, NCH, A, TOKEN>;
    const int tpr = row_threads(p.D);
    RingShape sh = ring_shape(tpr, staged_row_bytes(tpr, (int)sizeof(T), A == kVec), 2, 0, 0, kGradThreads, TOKEN ? 2 : 1);
    sh.smem -= sh.sums_bytes;
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.allow(reinterpret_cast<const void*>(k), sh)) return e;
    if constexpr (TOKEN) {
        const int64_t need = (p.rows + sh.groups - 1) / sh.groups, most = (int64_t)sm_count() * sh.ctas_per_sm;
        return launch_pdl(k, (unsigned)(need < most ? need : most), sh.groups * tpr, sh.smem, s, p, sh);
    } else {
        p.plan = grad_plan(p.rows, p.mod_rows, p.D, (int)sizeof(T));
        const int64_t units = p.mod_rows * p.plan.parts, most = 1 << 30;
        const cudaError_t e = launch_pdl(k, (unsigned)(units < most ? units : most), sh.groups * tpr, sh.smem, s, p, sh);
        if (e != cudaSuccess || p.plan.parts == 1 || !p.dgate) return e;
        ColSumParams c{p.ws, p.plan.parts, p.mod_rows, p.D, 1, {p.dgate, nullptr}, {p.dgate_stride, 0}, p.p_f32};
        return launch_column_sums(c, s);
    }
}

template <class T, int NCH>
static cudaError_t drop_bwd_any(const DropParams& p, bool vec, cudaStream_t s) {
    if (p.seq == 1) return vec ? drop_bwd<T, NCH, kVec, true>(p, s) : drop_bwd<T, NCH, kQuad, true>(p, s);
    return vec ? drop_bwd<T, NCH, kVec, false>(p, s) : drop_bwd<T, NCH, kQuad, false>(p, s);
}

cudaError_t launch_dropout_backward(const DropParams& p, bool f32, bool vec, cudaStream_t s) {
    return launch_all_or_none([&] {
        return f32 ? drop_bwd_any<float, 4>(p, vec, s) : drop_bwd_any<uint16_t, 2>(p, vec, s);
    });
}

}  // namespace mbx
