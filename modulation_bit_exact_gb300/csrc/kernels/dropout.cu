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
#include "rowgroup.cuh"

namespace mbx {

struct PhiloxKey {
    uint32_t k0, k1, c2, c3;
};

__device__ __forceinline__ PhiloxKey philox_key(const DropParams& p) {
    const uint64_t seed = (uint64_t)p.rng[0], ctr = (uint64_t)p.rng[1] + (uint64_t)p.offset;
    return PhiloxKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)ctr, (uint32_t)(ctr >> 32)};
}

__device__ __forceinline__ uint4 philox(uint32_t quad, uint32_t row, const PhiloxKey& key) {
    uint32_t c0 = quad, c1 = row, c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Bit e of the result: whether this thread's element e of the row is kept.
// Elements come in fours that share a counter.
template <class T, int NCH, Access A>
__device__ __forceinline__ uint32_t keep_bits(const PhiloxKey& key, uint32_t row, uint32_t threshold, int t, int tpr) {
    constexpr int E = NCH * ChunkOf<T>::CE;
    static_assert(A != kScalar, "four columns of a thread are consecutive");
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < E; e += 4) {
        const uint4 w = philox((uint32_t)col_of<T, A>(e, t, tpr) / 4u, row, key);
#pragma unroll
        for (int i = 0; i < 4; ++i) bits |= (w_of(w, i) >= threshold ? 1u : 0u) << (e + i);
    }
    return bits;
}

// GATED: out = x + gate * drop(y); otherwise out = drop(x).
template <class T, int NCH, Access A, bool GATED>
__global__ void __launch_bounds__(512) dropout_kernel(DropParams p) {
    constexpr int E = NCH * ChunkOf<T>::CE;
    const int tpr = p.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr, groups = blockDim.x / tpr;
    grid_dep_wait();  // launched programmatically: the previous kernel has finished
    grid_dep_launch();
    const PhiloxKey key = philox_key(p);
    const int64_t step = (int64_t)gridDim.x * groups;
    float gate[E];
    int64_t seg = -1;
    for (int64_t row = (int64_t)blockIdx.x * groups + g; row < p.rows; row += step) {
        RawRow<T, NCH, A> rx, ry;
        rx.load(static_cast<const T*>(p.x) + row * p.x_stride, p.D, t, tpr);
        if constexpr (GATED) {
            ry.load(static_cast<const T*>(p.y) + row * p.y_stride, p.D, t, tpr);
            const int64_t m = p.seq == 1 ? row : row / p.seq;
            if (m != seg) load_params<T, NCH, A>(gate, p.gate, m * p.gate_stride, p.p_f32, p.D, t, tpr, 0.0f);
            seg = m;
        }
        const uint32_t keep = keep_bits<T, NCH, A>(key, (uint32_t)row, p.threshold, t, tpr);
        float v[E];
        rx.widen(v);
        if constexpr (GATED) {
            float y[E];
            ry.widen(y);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (keep >> e & 1) v[e] = fmaf(gate[e], y[e] * p.inv_keep, v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = (keep >> e & 1) ? v[e] * p.inv_keep : 0.0f;
        }
        store_row<T, NCH, A>(static_cast<T*>(p.out) + row * p.out_stride, v, p.D, t, tpr);
    }
}

// One gate row for every row: dgate is a row too.
template <class T, int NCH, Access A>
__global__ void __launch_bounds__(512) dropout_backward_token_kernel(DropParams p) {
    constexpr int E = NCH * ChunkOf<T>::CE;
    const int tpr = p.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr, groups = blockDim.x / tpr;
    grid_dep_wait();
    grid_dep_launch();
    const PhiloxKey key = philox_key(p);
    const int64_t step = (int64_t)gridDim.x * groups;
    for (int64_t row = (int64_t)blockIdx.x * groups + g; row < p.rows; row += step) {
        RawRow<T, NCH, A> rd, ry;
        rd.load(static_cast<const T*>(p.x) + row * p.x_stride, p.D, t, tpr);
        ry.load(static_cast<const T*>(p.y) + row * p.y_stride, p.D, t, tpr);
        float gate[E], d[E], y[E];
        load_params<T, NCH, A>(gate, p.gate, row * p.gate_stride, p.p_f32, p.D, t, tpr, 0.0f);
        const uint32_t keep = keep_bits<T, NCH, A>(key, (uint32_t)row, p.threshold, t, tpr);
        rd.widen(d);
        ry.widen(y);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float k = d[e] * p.inv_keep;
            d[e] = (keep >> e & 1) ? k * gate[e] : 0.0f;
            y[e] = (keep >> e & 1) ? k * y[e] : 0.0f;
        }
        store_row<T, NCH, A>(static_cast<T*>(p.out) + row * p.out_stride, d, p.D, t, tpr);
        if (p.dgate) store_params<T, NCH, A>(p.dgate, row * p.dgate_stride, p.p_f32, y, p.D, t, tpr);
    }
}

// Gate rows shared by seq rows: the parts of a segment as in the gradients of
// LayerNorm's parameters (layernorm.cu).
template <class T, int NCH, Access A>
__global__ void __launch_bounds__(512) dropout_backward_kernel(DropParams p) {
    constexpr int E = NCH * ChunkOf<T>::CE;
    extern __shared__ float acc_smem[];  // [E][block]
    const int tpr = p.tpr, g = threadIdx.x / tpr, t = threadIdx.x % tpr, groups = blockDim.x / tpr;
    grid_dep_wait();
    grid_dep_launch();
    const PhiloxKey key = philox_key(p);
    const int64_t units = p.mod_rows * p.plan.parts;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t seg = unit / p.plan.parts, part = unit - seg * p.plan.parts;
        const int64_t r0 = seg * p.seq + part * p.plan.rows_per_part;
        int64_t r1 = r0 + p.plan.rows_per_part;
        if (r1 > (seg + 1) * p.seq) r1 = (seg + 1) * p.seq;
        float gate[E], acc[E];
        load_params<T, NCH, A>(gate, p.gate, seg * p.gate_stride, p.p_f32, p.D, t, tpr, 0.0f);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        for (int64_t row = r0 + g; row < r1; row += groups) {
            RawRow<T, NCH, A> rd, ry;
            rd.load(static_cast<const T*>(p.x) + row * p.x_stride, p.D, t, tpr);
            ry.load(static_cast<const T*>(p.y) + row * p.y_stride, p.D, t, tpr);
            const uint32_t keep = keep_bits<T, NCH, A>(key, (uint32_t)row, p.threshold, t, tpr);
            float d[E], y[E];
            rd.widen(d);
            ry.widen(y);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float k = d[e] * p.inv_keep;
                d[e] = (keep >> e & 1) ? k * gate[e] : 0.0f;
                if (keep >> e & 1) acc[e] = fmaf(k, y[e], acc[e]);
            }
            store_row<T, NCH, A>(static_cast<T*>(p.out) + row * p.out_stride, d, p.D, t, tpr);
        }
        if (p.dgate == nullptr) continue;
        if (groups > 1) {
            const int n = blockDim.x;
#pragma unroll
            for (int e = 0; e < E; ++e) acc_smem[e * n + threadIdx.x] = acc[e];
            __syncthreads();
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    for (int k = 1; k < groups; ++k) acc[e] += acc_smem[e * n + k * tpr + t];
            }
            __syncthreads();
        }
        if (g == 0) {
            if (p.plan.parts == 1)
                store_params<T, NCH, A>(p.dgate, seg * p.dgate_stride, p.p_f32, acc, p.D, t, tpr);
            else store_params<T, NCH, A>(p.ws, unit * p.D, true, acc, p.D, t, tpr);
        }
    }
}

// ---------------------------------------------------------------- launch

template <class T, int NCH>
static cudaError_t drop_fwd(const DropParams& p0, bool vec, cudaStream_t s) {
    DropParams p = p0;
    p.tpr = row_threads(p.D);
    if (p.tpr < 32) p.tpr = 32;
    p.groups = p.tpr >= 256 ? 1 : 256 / p.tpr;
    const int block = p.tpr * p.groups;
    auto k = p.gate ? (vec ? dropout_kernel<T, NCH, kVec, true> : dropout_kernel<T, NCH, kQuad, true>)
                    : (vec ? dropout_kernel<T, NCH, kVec, false> : dropout_kernel<T, NCH, kQuad, false>);
    const int grid = grid_for_rows(reinterpret_cast<const void*>(k), p.rows, p.groups, block);
    if (grid < 0) return cudaErrorUnknown;
    return launch_pdl(k, grid, block, 0, s, p);
}

cudaError_t launch_dropout(const DropParams& p, bool f32, bool vec, cudaStream_t s) {
    return f32 ? drop_fwd<float, 4>(p, vec, s) : drop_fwd<uint16_t, 2>(p, vec, s);
}

template <class T, int NCH>
static cudaError_t drop_bwd(const DropParams& p0, bool vec, cudaStream_t s) {
    DropParams p = p0;
    p.tpr = row_threads(p.D);
    if (p.tpr < 32) p.tpr = 32;
    p.groups = p.tpr >= 256 ? 1 : 256 / p.tpr;
    const int block = p.tpr * p.groups;
    if (p.seq == 1) {
        auto k = vec ? dropout_backward_token_kernel<T, NCH, kVec> : dropout_backward_token_kernel<T, NCH, kQuad>;
        const int grid = grid_for_rows(reinterpret_cast<const void*>(k), p.rows, p.groups, block);
        if (grid < 0) return cudaErrorUnknown;
        return launch_pdl(k, grid, block, 0, s, p);
    }
    p.plan = grad_plan(p.rows, p.mod_rows, p.D, (int)sizeof(T));
    const size_t smem = p.groups > 1 ? (size_t)block * 16 * sizeof(float) : 0;
    const int64_t units = p.mod_rows * p.plan.parts;
    auto k = vec ? dropout_backward_kernel<T, NCH, kVec> : dropout_backward_kernel<T, NCH, kQuad>;
    cudaError_t e = launch_pdl(k, (unsigned)(units < (1 << 30) ? units : (1 << 30)), block, smem, s, p);
    if (e != cudaSuccess || p.plan.parts == 1 || !p.dgate) return e;
    ColSumParams c{p.ws, p.plan.parts, p.mod_rows, p.D, 1, {p.dgate, nullptr}, {p.dgate_stride, 0}, p.p_f32};
    return launch_column_sums(c, s);
}

cudaError_t launch_dropout_backward(const DropParams& p, bool f32, bool vec, cudaStream_t s) {
    return launch_all_or_none([&] {
        return f32 ? drop_bwd<float, 4>(p, vec, s) : drop_bwd<uint16_t, 2>(p, vec, s);
    });
}

}  // namespace mbx
