// qknorm.cu -- RMSNorm of every head of Q and K and the rotation by positions on
// several axes, in one pass:
//   n = x * rstd * w,  rstd = 1 / sqrt(mean(x^2) + eps) over the head,
//   out = the pairs of n turned as in rope.cu; elements past the pairs pass.
// binary32, one rounding at the output.
//
// A warp walks tokens, of Q or of K, or a share of their heads where that divides
// the tokens better: with the other warps of a token it computes the sines and cosines,
// keeps its own in registers and takes the heads, 32 / G of them side by side, out of a
// ring in shared memory that it fills ahead (qknorm.cuh).
#include "qknorm.cuh"

namespace mbx {

QkShare qk_share(int64_t total, int64_t most, int q_heads, int k_heads) {
    QkShare best = {1, 1, k_heads ? 1 : 0};
    double cost = 1e30;
    for (int wpt = 1; wpt <= kQkWarps; wpt *= 2) {
        const int64_t per_block = kQkWarps / wpt, need = (total + per_block - 1) / per_block;
        int64_t q = k_heads ? most * q_heads / (q_heads + k_heads) : most;
        q = q < 1 ? 1 : k_heads && q >= most ? most - 1 : q;
        int64_t k = k_heads ? most - q : 0;
        if (q > need) q = need;
        if (k > need) k = need;
        double c = (double)((need + q - 1) / q) * (1.0 / wpt + 0.1) * q_heads;
        if (k) {
            const double ck = (double)((need + k - 1) / k) * (1.0 / wpt + 0.1) * k_heads;
            if (ck > c) c = ck;
        }
        if (c < cost) {
            cost = c;
            best = QkShare{wpt, (int)q, (int)k};
        }
    }
    return best;
}

// Blocks of an SM, by the elements of a head that a lane holds: what the registers allow.
// Heads on their way to a lane: as many as make 96 bytes.
constexpr int forward_blocks(int elems) { return elems <= 8 ? 3 : 2; }
constexpr int forward_stages(int bytes) { return 96 / bytes < 2 ? 2 : 96 / bytes; }

template <class T, bool INTERLEAVED, int W, int U, bool VEC, int GT>
__global__ void __launch_bounds__(32 * kQkWarps, forward_blocks(HeadUnits<T, INTERLEAVED, W, U, VEC>::E * U))
    qk_norm_rope_kernel(QkNormParams p, int g, QkShare sh) {
    using Head = HeadUnits<T, INTERLEAVED, W, U, VEC>;
    constexpr int kStages = forward_stages(U * Head::E * (int)sizeof(T));
    extern __shared__ uint4 smem[];  // [warps][stages] slots, the pairs' frequencies, [tokens of the block][pairs]
    const RopeParams& r = p.rope;
    const int G = GT ? GT : g, groups = 32 / G, wpt = sh.wpt, per_block = kQkWarps / wpt;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, slot = warp / wpt, share = warp % wpt;
    const bool which = (int)blockIdx.x >= sh.q_blocks;
    const int block = which ? blockIdx.x - sh.q_blocks : blockIdx.x, blocks = which ? sh.k_blocks : sh.q_blocks;
    const RopeTensor& t = which ? r.k : r.q;
    const unsigned tokens = (unsigned)r.tokens, total = (unsigned)r.batch * tokens;
    const Head head(lane % G, G, r.hd, r.pairs);
    PairFreq* freqs = reinterpret_cast<PairFreq*>(reinterpret_cast<char*>(smem) + kQkWarps * kStages * Head::kSlotBytes);
    float2* cs = reinterpret_cast<float2*>(freqs + r.pairs) + slot * r.pairs;
    const int h0 = share * groups + lane / G, step = wpt * groups;
    HeadStream<Head, T, 1, kStages> in(
        head, (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * Head::kSlotBytes + lane * Head::kAccessBytes,
        block * per_block + slot, blocks * per_block, tokens, total, h0, lane / G, step, t.heads, lane / G < groups);
    in.tensor(0, t.in, t.ib, t.it, t.ih);
    typename Head::Raw raw[1];
    raw[0].clear();
    grid_dep_wait();
    grid_dep_launch();
    in.start();
    for (int j = threadIdx.x; j < r.pairs; j += blockDim.x) freqs[j] = pair_freq(r, j);
    __syncthreads();
    TokenAngles angle(r, freqs, cs, share, wpt);
    angle.fetch(block * per_block + slot, tokens, total);
    const typename Head::Values w = head.weight(p.w[which], p.w_f32);

    // the same number of rounds for all warps of the block, which may meet in them
#pragma unroll 1
    for (unsigned tok0 = block * per_block; tok0 < total; tok0 += blocks * per_block) {
        const unsigned tok = tok0 + slot, b = tok / tokens, s = tok - b * tokens;
        const bool has = tok < total;
        angle.make(has);
        angle.fetch(tok + blocks * per_block, tokens, total);
        if (!has) continue;
        const typename Head::Angles angles = head.angles(cs);
        T* out = static_cast<T*>(t.out) + b * t.ob + s * t.ot + h0 * t.oh;
#pragma unroll 1
        for (int i = 0; i < in.steps; ++i, out += step * t.oh) {
            in.take(raw);
            typename Head::Values x = Head::values(raw[0]);
            const float ss = group_sum<GT>(dot(x.first, x.second, x), G);
            in.fetch();
            const float rstd = rsqrtf(__fmaf_rn(ss, p.inv_hd, p.eps));
            const u64 r2 = f2(rstd, rstd);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < Head::NP; ++j) {
                    x.first[u][j] = mul2(mul2(x.first[u][j], r2), w.first[u][j]);
                    x.second[u][j] = mul2(mul2(x.second[u][j], r2), w.second[u][j]);
                }
            head.turn(x, angles);
            if (i < in.mine) head.store(out, x);
        }
    }
}

// 16 elements a lane: fewer exchanges for an element than with 8.
template <bool INTERLEAVED>
static cudaError_t forward(const QkNormParams& p, bool f32, int align, cudaStream_t s) {
    const RopeParams& r = p.rope;
    const HeadShape shape = head_shape<16, 8>(r.hd, r.pairs, f32, INTERLEAVED, align);
    return for_head_shape<16, 8, INTERLEAVED>(shape, f32, [&](auto t, auto inter, auto w, auto u, auto vec, auto gt) {
        using Head = HeadUnits<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value, decltype(vec)::value>;
        constexpr int kElems = Head::E * decltype(u)::value, kStages = forward_stages(kElems * (int)sizeof(t));
        const QkShare sh = qk_share(r.batch * r.tokens, forward_blocks(kElems) * (int64_t)sm_count(), r.q.heads, r.k.heads);
        auto* k = qk_norm_rope_kernel<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value,
                                      decltype(vec)::value, decltype(gt)::value>;
        const size_t smem = kQkWarps * kStages * Head::kSlotBytes + r.pairs * sizeof(PairFreq) +
                            kQkWarps / sh.wpt * r.pairs * sizeof(float2);
        static SmemOptIn opt;
        if (cudaError_t e = allow_smem(opt, reinterpret_cast<const void*>(k), smem)) return e;
        return launch_pdl(k, (unsigned)(sh.q_blocks + sh.k_blocks), 32 * kQkWarps, smem, s, p, shape.g, sh);
    });
}

cudaError_t launch_qk_norm_rope(const QkNormParams& p, bool f32, bool interleaved, int align, cudaStream_t s) {
    return interleaved ? forward<true>(p, f32, align, s) : forward<false>(p, f32, align, s);
}

}  // namespace mbx
