// qknorm_bwd.cu -- gradients of qknorm.cu.  With g = dout turned back, xh = x * rstd
// and gy = g * w:
//   dx = rstd * (gy - xh * mean(gy * xh)),   dw = sum over batch, tokens and heads of g * xh
// Statistics are taken from x again.  mean(gy * xh) = rstd * mean(gy * x), so
// both row sums are formed in one exchange.
//
// The walk is that of qknorm.cu, with the incoming gradient beside the input.  A warp
// keeps its lanes' part of dw in registers; a block adds its warps' parts in shared
// memory, and column_sums (colsum.cu) the blocks' parts, in a fixed order.
//
// Floor: two arrays read, one written.  32760 tokens of 40 + 40 heads of 128, bfloat16:
// 324 us, 6.2 TB/s of 6.7 that a copy reaches; 8704 of 24 + 24: 62 us, 5.2 TB/s, of which 4
// join the parts (issue 61%: 44 M warp instructions, 211 for two heads of 128).
#include "qknorm.cuh"

namespace mbx {

// Heads on their way to a lane: as many as make 64 bytes of each tensor.
constexpr int grad_stages(int bytes) { return 64 / bytes < 2 ? 2 : 64 / bytes; }

template <class T, bool INTERLEAVED, int W, int U, bool VEC, int GT>
__global__ void __launch_bounds__(32 * kQkWarps, kQkBlocks)
    qk_norm_rope_bwd_kernel(QkNormParams p, int g, QkShare sh) {
    using Head = HeadUnits<T, INTERLEAVED, W, U, VEC>;
    constexpr int E = Head::E, NP = Head::NP, kStages = grad_stages(U * E * (int)sizeof(T));
    extern __shared__ uint4 smem[];  // [warps][stages][2] slots, the pairs' frequencies, [tokens of the block][pairs]
    const RopeParams& r = p.rope;
    const int G = GT ? GT : g, groups = 32 / G, hd = r.hd, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const QkPlace at(sh, r.q.heads, r.k.heads, G, groups, Bool<false>());
    const RopeTensor& t = at.k ? r.k : r.q;
    const GradIn& d = p.dout[at.k];
    const unsigned tokens = (unsigned)r.tokens, total = (unsigned)r.batch * tokens;
    const Head head(lane % G, G, hd, r.pairs);
    PairFreq* freqs = reinterpret_cast<PairFreq*>(reinterpret_cast<char*>(smem) + kQkWarps * kStages * 2 * Head::kSlotBytes);
    float2* cs = reinterpret_cast<float2*>(freqs + r.pairs) + at.slot * at.tpw * r.pairs;
    HeadStream<Head, T, 2, kStages> in(
        head, at, (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * 2 * Head::kSlotBytes + lane * Head::kAccessBytes, r,
        t.heads, sh.by_tokens);
    in.tensor(0, t.in, t.ib, t.it, t.ih);
    in.tensor(1, d.in, d.ib, d.it, d.ih);
    typename Head::Raw raw[2];
    raw[0].clear();
    raw[1].clear();
    grid_dep_wait();
    grid_dep_launch();
    in.start();
    for (int j = threadIdx.x; j < r.pairs; j += blockDim.x) freqs[j] = pair_freq(r, j);
    __syncthreads();
    TokenAngles angle(r, freqs, cs, at.share, sh.wpt, at.tpw, total, sh.by_tokens);
    angle.fetch(at.tok - at.sub);
    const typename Head::Values w = head.weight(p.w[at.k], p.w_f32);
    typename Head::Values acc;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < NP; ++j) acc.first[u][j] = acc.second[u][j] = 0;

    // the same number of rounds for all warps of the block, which may meet in them
    const unsigned first = at.block * (kQkWarps / sh.wpt) * at.tpw;
#pragma unroll 1
    for (unsigned round = first, tok = at.tok; round < total; round += at.stride, tok += at.stride) {
        angle.make(tok - at.sub);
        angle.fetch(tok - at.sub + at.stride);
        if (tok - at.sub >= total) continue;
        const bool has = tok < total;
        const unsigned b = has ? batch_of(tok, sh.by_tokens) : 0, s = has ? tok - b * tokens : 0;
        const typename Head::Rotation turn = head.rotation(cs + at.sub * r.pairs);
        T* out = static_cast<T*>(t.out) + b * t.ob + s * t.ot + at.h0 * t.oh;
#pragma unroll 1
        for (int i = 0; i < in.steps; ++i, out += at.step * t.oh) {
            in.take(raw);
            const bool real = has && i < in.mine;
            typename Head::Values x = Head::values(raw[0]), gr = Head::values(raw[1]), gy;
            head.turn(gr, turn);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    gy.first[u][j] = mul2(gr.first[u][j], w.first[u][j]);
                    gy.second[u][j] = mul2(gr.second[u][j], w.second[u][j]);
                }
            float ss = dot(x.first, x.second, x), gx = dot(gy.first, gy.second, x);
            group_sums<GT>(ss, gx, G);
            in.fetch();
            const float rstd = rsqrtf(__fmaf_rn(ss, p.inv_hd, p.eps));
            const float c2 = -(gx * p.inv_hd * rstd);
            const u64 r2 = f2(rstd, rstd), m2 = f2(c2, c2);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const u64 x0 = mul2(x.first[u][j], r2), x1 = mul2(x.second[u][j], r2);
                    if (real) {
                        acc.first[u][j] = fma2(gr.first[u][j], x0, acc.first[u][j]);
                        acc.second[u][j] = fma2(gr.second[u][j], x1, acc.second[u][j]);
                    }
                    x.first[u][j] = mul2(fma2(x0, m2, gy.first[u][j]), r2);
                    x.second[u][j] = mul2(fma2(x1, m2, gy.second[u][j]), r2);
                }
            if (real) head.store(out, x);
        }
    }
    if (!p.ws) return;
    float* sums = reinterpret_cast<float*>(smem);  // [warps][hd], in the slots' place
    __syncthreads();
    // the warp's groups side by side, then the block's warps in order
    float a[U][E];
    Head::unpack(a, acc);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float v = a[u][e];
            for (int k = 1; k < groups; ++k) v += __shfl_sync(0xffffffffu, a[u][e], lane % G + k * G);
            a[u][e] = v;
        }
        if (lane < G) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if (head.off0[u] >= 0) sums[warp * hd + head.off0[u] + i] = a[u][i];
                if constexpr (Head::kTwo)
                    if (head.off1[u] >= 0) sums[warp * hd + head.off1[u] + i] = a[u][W + i];
            }
        }
    }
    __syncthreads();
    const bool alone = at.block >= (at.k ? sh.q.blocks : sh.k.blocks);  // the other tensor has no such block
    for (int e = threadIdx.x; e < hd; e += blockDim.x) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kQkWarps; ++i) v += sums[i * hd + e];
        float* part = p.ws + (int64_t)at.block * 2 * hd + e;
        part[at.k * hd] = v;
        if (alone) part[!at.k * hd] = 0.0f;
    }
}

// A call has at most as many parts as there are blocks for Q or for K.
int64_t qk_norm_grad_parts(int64_t batch, int64_t tokens) {
    const int64_t most = (int64_t)kQkBlocks * sm_count(), total = batch * tokens;
    return total < most ? total : most;
}

// 8 elements a lane: two tensors, the sums and the weights fill the registers of two
// blocks an SM.
template <bool INTERLEAVED>
static cudaError_t backward(const QkNormParams& p, bool f32, int align, ColSumParams& sums, cudaStream_t s) {
    constexpr int kWidest = INTERLEAVED ? 8 : 4;
    const RopeParams& r = p.rope;
    const HeadShape shape = head_shape<8, kWidest>(r.hd, r.pairs, f32, INTERLEAVED, align);
    return for_head_shape<8, kWidest, INTERLEAVED>(shape, f32, [&](auto t, auto inter, auto w, auto u, auto vec, auto gt) {
        using Head = HeadUnits<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value, decltype(vec)::value>;
        constexpr int kStages = grad_stages(Head::E * decltype(u)::value * (int)sizeof(t));
        const QkShare sh = qk_share(r, kQkBlocks * (int64_t)sm_count(), 32 / shape.g, false);
        sums.parts = sh.q.blocks > sh.k.blocks ? sh.q.blocks : sh.k.blocks;
        auto* k = qk_norm_rope_bwd_kernel<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value,
                                          decltype(vec)::value, decltype(gt)::value>;
        const int most = sh.q.tpw > sh.k.tpw ? sh.q.tpw : sh.k.tpw;
        size_t smem = kQkWarps * kStages * 2 * Head::kSlotBytes + r.pairs * sizeof(PairFreq) +
                      kQkWarps / sh.wpt * most * r.pairs * sizeof(float2);
        if (smem < kQkWarps * r.hd * sizeof(float)) smem = kQkWarps * r.hd * sizeof(float);  // the sums
        static SmemOptIn opt;
        if (cudaError_t e = allow_smem(opt, reinterpret_cast<const void*>(k), smem)) return e;
        return launch_pdl(k, (unsigned)(sh.q.blocks + sh.k.blocks), 32 * kQkWarps, smem, s, p, shape.g, sh);
    });
}

cudaError_t launch_qk_norm_rope_backward(const QkNormParams& p, bool f32, bool interleaved, int align, ColSumParams sums,
                                         cudaStream_t s) {
    const cudaError_t e = interleaved ? backward<true>(p, f32, align, sums, s) : backward<false>(p, f32, align, sums, s);
    if (e != cudaSuccess || !p.ws) return e;
    return launch_column_sums(sums, s);
}

}  // namespace mbx
