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
//
// A row of 5120 bfloat16 takes 19,200 of the generator's 32-bit products to 30 KB
// of memory: the forward pass comes near memory ([32760, 5120]: 152 us, 6.6 TB/s
// of 6.77 that a copy reaches).  The gradients, which also sum, have registers for
// 16 warps an SM; these issue in 59% of the cycles and wait for the integer
// multiplier, each quad's products being a chain ([8704, 4096] into two rows: 44.5
// us, 4.8 TB/s).
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
template <int NQ, int CE>
__device__ __forceinline__ Philox<NQ> make_philox(const DropParams& p, const Lane& L) {
    uint32_t quad[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i)
        quad[i] = CE == 8 ? (uint32_t)(i / 2 * L.tpr + L.t) * 2 + i % 2 : (uint32_t)(i * L.tpr + L.t);
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
template <class T, int NCH, bool GATED>
__global__ void __launch_bounds__(kRingThreads) dropout_kernel(DropParams p, RingShape sh) {
    constexpr Access A = kVec;
    constexpr int CE = ChunkOf<T>::CE, H = CE / 2, P = NCH * H;
    extern __shared__ __align__(16) char smem[];
    const int tpr = sh.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const Lane L = make_lane<CE>(t, tpr, p.D, g + 1);
    char* ring = smem + g * sh.group_bytes;
    const int64_t step = (int64_t)gridDim.x * sh.groups;
    int64_t row = (int64_t)blockIdx.x * sh.groups + g, fill_row = row;
    if (row < p.rows) {
        prefetch_row<T, A>(static_cast<const T*>(p.x) + row * p.x_stride, p.D, t);
        if constexpr (GATED) prefetch_row<T, A>(static_cast<const T*>(p.y) + row * p.y_stride, p.D, t);
    }
    grid_dep_wait();  // launched programmatically: the previous kernel has finished
    grid_dep_launch();
    Philox<P / 2> philox = make_philox<P / 2, CE>(p, L);
    const int row_bytes = sh.row_bytes, stage_bytes = (GATED ? 2 : 1) * row_bytes;
    auto fill = [&](int st) {
        char* dst = ring + st * stage_bytes;
        if (fill_row < p.rows) {
            ring_fill<T, NCH, CE, A>(dst, static_cast<const T*>(p.x) + fill_row * p.x_stride, L);
            if constexpr (GATED)
                ring_fill<T, NCH, CE, A>(dst + row_bytes, static_cast<const T*>(p.y) + fill_row * p.y_stride, L);
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
                    get_param_chunk<T, CE, A>(c, p.gate, m * p.gate_stride, p.p_f32, j, L);
#pragma unroll
                    for (int i = 0; i < H; ++i) gate[j * H + i] = mul2(c[i], inv);
                }
            }
        }
        ring_wait(sh.stages);
        uint4 xr[NCH], yr[GATED ? NCH : 1];
        read_pieces<T, NCH, A>(xr, ring + stage * stage_bytes, L);
        if constexpr (GATED) read_pieces<T, NCH, A>(yr, ring + stage * stage_bytes + row_bytes, L);
        fill(stage);
        if (++stage == sh.stages) stage = 0;
        philox.row((uint32_t)row);
        T* dst = static_cast<T*>(p.out) + row * p.out_stride;
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
            put_row_chunk<T, CE, A>(dst, nullptr, o, j, L);
        }
    }
}

// The same for rows that are not 16-byte aligned or whose width is no multiple of
// a chunk.  A thread takes an aligned 16-byte piece of the output row, so both
// accesses are whole pieces where x and y lie the same way to 16 bytes as out
// does (elements at the row's ends, and where they do not); there is no stage and
// no barrier.  A piece starts anywhere within a quad, so its last columns belong
// to the first quad of the next lane, which passes their bits down: a warp's last
// lane only computes them, and a warp takes 31 pieces at a time.
// [4096, 2731] binary32: 22.3 us by single elements, 27.7 through kShift stages,
// 26.8 when a thread computes both quads, 19.5 here (2728 columns: 18.6).
template <class T, bool GATED>
__global__ void __launch_bounds__(256) dropout_shift_kernel(DropParams p, int tpr) {
    constexpr int CE = ChunkOf<T>::CE, NQ = CE / 4;
    const int g = threadIdx.x / tpr, groups = blockDim.x / tpr, lane = threadIdx.x % 32;
    const int warp = threadIdx.x % tpr / 32, warps = tpr / 32;
    grid_dep_wait();
    grid_dep_launch();
    const uint64_t seed = (uint64_t)p.rng[0], ctr = (uint64_t)p.rng[1] + (uint64_t)p.offset;
    uint32_t k0[10], k1[10];
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        k0[r] = (uint32_t)seed + r * kW0;
        k1[r] = hi32(seed) + r * kW1;
        asm volatile("" : "+r"(k0[r]), "+r"(k1[r]));
    }
    const int64_t step = (int64_t)gridDim.x * groups;
    for (int64_t row = (int64_t)blockIdx.x * groups + g; row < p.rows; row += step) {
        const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
        const T* y = GATED ? static_cast<const T*>(p.y) + row * p.y_stride : x;
        T* out = static_cast<T*>(p.out) + row * p.out_stride;
        const uintptr_t at = reinterpret_cast<uintptr_t>(out);
        const bool alike = ((reinterpret_cast<uintptr_t>(x) ^ at) & 15) == 0 && ((reinterpret_cast<uintptr_t>(y) ^ at) & 15) == 0;
        const int shift = (int)(at & 15) / (int)sizeof(T);
        const int64_t gate = GATED ? (p.mod_rows == p.rows ? row : p.mod_rows == 1 ? 0 : row / p.seq) * p.gate_stride : 0;
        for (int c = warp * 31 * CE - shift; c < p.D; c += warps * 31 * CE) {  // the same for a warp
            const int c0 = c + lane * CE;
            const bool mine = lane < 31 && c0 < p.D, whole = mine && c0 >= 0 && c0 + CE <= p.D;
            float v[CE], w[CE];
            if (whole && alike) {
                const uint4 rx = ld_stream_rw(x + c0);
                if constexpr (GATED) widen_chunk(ld_stream_rw(y + c0), w);
                widen_chunk(rx, v);
            } else {
#pragma unroll
                for (int i = 0; i < CE; ++i) {
                    const bool in = mine && c0 + i >= 0 && c0 + i < p.D;
                    v[i] = in ? load_elem(x + c0 + i) : 0.0f;
                    if constexpr (GATED) w[i] = in ? load_elem(y + c0 + i) : 0.0f;
                }
            }
            const int quad = c0 >> 2, rem = c0 & 3;  // c0 = 4*quad + rem
            uint32_t keep = 0;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                uint32_t u0 = (uint32_t)(quad + q), u1 = (uint32_t)row, u2 = (uint32_t)ctr, u3 = hi32(ctr);
#pragma unroll
                for (int r = 0; r < 10; ++r) {
                    const uint64_t a = (uint64_t)kM0 * u0, b = (uint64_t)kM1 * u2;
                    u0 = hi32(b) ^ u1 ^ k0[r];
                    u1 = (uint32_t)b;
                    u2 = hi32(a) ^ u3 ^ k1[r];
                    u3 = (uint32_t)a;
                }
                const uint32_t thr = p.threshold;
                keep |= ((u0 >= thr ? 1u : 0u) | (u1 >= thr ? 2u : 0u) | (u2 >= thr ? 4u : 0u) | (u3 >= thr ? 8u : 0u)) << (4 * q);
            }
            keep |= (__shfl_down_sync(0xffffffffu, keep, 1) & 15u) << (4 * NQ);
            keep >>= rem;  // bit i: element i of the piece
            if (!mine) continue;
#pragma unroll
            for (int i = 0; i < CE; ++i) {
                if constexpr (GATED) {
                    if (c0 + i >= 0 && c0 + i < p.D && (keep >> i & 1)) {
                        const float f = p.p_f32 ? load_elem(static_cast<const float*>(p.gate) + gate + c0 + i)
                                                : load_elem(static_cast<const uint16_t*>(p.gate) + gate + c0 + i);
                        v[i] = fmaf(w[i], f * p.inv_keep, v[i]);
                    }
                } else {
                    v[i] = (keep >> i & 1) ? v[i] * p.inv_keep : 0.0f;
                }
            }
            if (whole) {
                st_v4(out + c0, narrow_chunk(v));
            } else {
#pragma unroll
                for (int i = 0; i < CE; ++i)
                    if (c0 + i >= 0 && c0 + i < p.D) store_elem(out + c0 + i, v[i]);
            }
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
    const Lane L = make_lane<CE>(t, tpr, p.D, g + 1);
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
    Philox<P / 2> philox = make_philox<P / 2, CE>(p, L);
    const int row_bytes = sh.row_bytes, stage_bytes = 2 * row_bytes;
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
                ring_fill<T, NCH, CE, A>(dst, static_cast<const T*>(p.x) + fill_row * p.x_stride, L);
                ring_fill<T, NCH, CE, A>(dst + row_bytes, static_cast<const T*>(p.y) + fill_row * p.y_stride, L);
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
                get_param_chunk<T, CE, A>(c, p.gate, m * p.gate_stride, p.p_f32, j, L);
#pragma unroll
                for (int i = 0; i < H; ++i) gate[j * H + i] = c[i];
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
            if constexpr (A == kShift) group_sync(L);
            uint4 dr[NCH], yr[NCH];
            read_pieces<T, NCH, A>(dr, ring + stage * stage_bytes, L);
            read_pieces<T, NCH, A>(yr, ring + stage * stage_bytes + row_bytes, L);
            if constexpr (A == kVec) fill(stage);
            else group_sync(L);  // every thread has read the stage
            philox.row((uint32_t)row);
            T* dst = static_cast<T*>(p.out) + row * p.out_stride;
            char* out = ring + stage * stage_bytes;
            u64 dgate[TOKEN ? NCH : 1][H];
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
                        const u64 d = piece_pair<T>(dr, e + h);
                        const u64 y = piece_pair<T>(yr, e + h);
                        // in the formula's order: the product of two bfloat16 is exact, so
                        // dy is rounded once in binary32.  gate / (1-p), rounded, in its
                        // place turned 0.2% of the outputs at p = 0.1, where 10/9 of a
                        // product often lies just between two bfloat16
                        o[i + h] = keep_pair(mul2(mul2(d, gate[e + h]), inv), w0, w1, p.threshold);
                        if constexpr (TOKEN) dgate[j][i + h] = keep_pair(mul2(d, mul2(y, inv)), w0, w1, p.threshold);
                        else acc[e + h] = keep_fma(d, y, acc[e + h], w0, w1, p.threshold);
                    }
                }
                put_row_chunk<T, CE, A>(dst, out, o, j, L);
            }
            if constexpr (A == kShift) flush_row(dst, out, L);
            if constexpr (TOKEN) {
                if (p.dgate) {
                    const int64_t off = row * p.dgate_stride;
#pragma unroll
                    for (int j = 0; j < NCH; ++j)
                        put_param_row_chunk<T, CE, A>(p.dgate, off, p.p_f32, out, dgate[j], j, L);
                    if constexpr (A == kShift) flush_param_row<T>(p.dgate, off, p.p_f32, out, L);
                }
            }
            if constexpr (A == kShift) fill(stage);
            if (++stage == sh.stages) stage = 0;
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
                    if (j >= L.nv) continue;
                    u64 c[H];
#pragma unroll
                    for (int i = 0; i < H; ++i) c[i] = mul2(acc[j * H + i], inv);
                    if (p.plan.parts == 1)
                        put_param_chunk<T, CE, A>(p.dgate, seg * p.dgate_stride, p.p_f32, c, j, L);
                    else put_chunk<float, CE, A>(p.ws + unit * p.D, c, j, L);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- launch

template <class T, int NCH, bool GATED>
static cudaError_t drop_fwd(const DropParams& p, cudaStream_t s) {
    auto k = dropout_kernel<T, NCH, GATED>;
    const int tpr = row_threads(p.D);
    RingShape sh = ring_shape(tpr, staged_row_bytes(tpr, (int)sizeof(T), true), GATED ? 2 : 1, 0, 0, kRingThreads, 2);
    sh.smem -= sh.sums_bytes;  // no row sums
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.allow(reinterpret_cast<const void*>(k), sh)) return e;
    const int64_t need = (p.rows + sh.groups - 1) / sh.groups, most = (int64_t)sm_count() * sh.ctas_per_sm;
    return launch_pdl(k, (unsigned)(need < most ? need : most), sh.groups * tpr, sh.smem, s, p, sh);
}

template <class T, bool GATED>
static cudaError_t drop_fwd_shift(const DropParams& p, cudaStream_t s) {
    auto k = dropout_shift_kernel<T, GATED>;
    const int warps = (p.D / ChunkOf<T>::CE + 2 + 30) / 31;  // 31 pieces of a row each
    const int tpr = warps >= 8 ? 256 : warps * 32, groups = 256 / tpr;
    const int grid = grid_for_rows(reinterpret_cast<const void*>(k), p.rows, groups, groups * tpr);
    if (grid < 0) return cudaErrorUnknown;
    return launch_pdl(k, grid, groups * tpr, 0, s, p, tpr);
}

template <class T, int NCH>
static cudaError_t drop_fwd_any(const DropParams& p, bool vec, cudaStream_t s) {
    if (vec) return p.gate ? drop_fwd<T, NCH, true>(p, s) : drop_fwd<T, NCH, false>(p, s);
    return p.gate ? drop_fwd_shift<T, true>(p, s) : drop_fwd_shift<T, false>(p, s);
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
    if (p.seq == 1) return vec ? drop_bwd<T, NCH, kVec, true>(p, s) : drop_bwd<T, NCH, kShift, true>(p, s);
    return vec ? drop_bwd<T, NCH, kVec, false>(p, s) : drop_bwd<T, NCH, kShift, false>(p, s);
}

cudaError_t launch_dropout_backward(const DropParams& p, bool f32, bool vec, cudaStream_t s) {
    return launch_all_or_none([&] {
        return f32 ? drop_bwd_any<float, 4>(p, vec, s) : drop_bwd_any<uint16_t, 2>(p, vec, s);
    });
}

}  // namespace mbx
