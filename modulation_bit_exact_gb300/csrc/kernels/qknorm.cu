// qknorm.cu -- RMSNorm of every head of Q and K and the rotation by positions on
// several axes, in one pass:
//   n = x * rstd * w,  rstd = 1 / sqrt(mean(x^2) + eps) over the head,
//   out = the pairs of n turned as in rope.cu; elements past the pairs pass.
// binary32, one rounding at the output: w goes into a token's cosines and sines, once,
// and rstd follows the turn.
//
// A warp walks tokens, of Q or of K, or a share of their heads where that divides
// the tokens better: with the other warps of a token it computes the sines and cosines,
// keeps its own in registers and takes the heads, 32 / G of them side by side, out of a
// ring in shared memory that it fills ahead (qknorm.cuh).
//
// Floor: every element read and written once.  32760 tokens of 40 + 40 heads of 128,
// bfloat16: 210 us, 6.4 TB/s of 6.7 that a copy reaches; 8704 of 24 + 24: 40 us, 5.4 TB/s,
// where issue shows (57% of the slots: 24 M warp instructions, 230 for four heads of 128)
// and the start of the blocks, 3 us, is not hidden; 24 single tokens: 3.2 us in a graph.
#include "qknorm.cuh"

namespace mbx {

// The cheapest division by a model in steps of a warp (a head of each of its groups):
// a round of tokens costs its steps and 2.5 more, for the angles and the chain of
// one token's work, and a quarter for each further token of a warp.
QkShare qk_share(const RopeParams& r, int64_t most, int groups, bool may_be_together) {
    const int64_t total = r.batch * r.tokens;
    QkShare best = {};
    double cost = 1e30;
    for (int wpt = 1; wpt <= kQkWarps; wpt *= 2) {
        auto of = [&](int heads, QkDeal* d) {  // the cost of a token
            d->tpw = wpt == 1 && heads * 2 <= groups ? groups / heads : 1;
            const int steps = (heads + groups * wpt - 1) / (groups * wpt);
            return (steps + 2.5 + 0.25 * (d->tpw - 1)) * wpt / d->tpw;
        };
        auto rounds = [&](const QkDeal& d) {
            const int64_t per = (int64_t)d.blocks * (kQkWarps / wpt) * d.tpw;
            return (double)((total + per - 1) / per);
        };
        auto blocks = [&](QkDeal& d, int64_t share) {
            const int64_t per = kQkWarps / wpt * d.tpw, need = (total + per - 1) / per;
            d.blocks = (int)(share < 1 ? 1 : share < need ? share : need);
        };
        QkDeal q = {}, k = {};
        const double cq = of(r.q.heads, &q), ck = r.k.heads ? of(r.k.heads, &k) : 0.0;
        blocks(q, r.k.heads ? (int64_t)(most * cq / (cq + ck)) : most);
        double c = rounds(q) * cq * q.tpw / wpt;
        if (r.k.heads) {
            blocks(k, most - q.blocks);
            const double o = rounds(k) * ck * k.tpw / wpt;
            c = o > c ? o : c;
        }
        if (c < cost) {
            cost = c;
            best.q = q;
            best.k = k;
            best.wpt = wpt;
        }
    }
    if (may_be_together && r.k.heads && r.q.heads + r.k.heads <= groups) {
        QkDeal d = {};
        d.tpw = groups / (r.q.heads + r.k.heads);
        const int64_t per = kQkWarps * d.tpw, need = (total + per - 1) / per;
        d.blocks = (int)(need < most ? need : most);
        const double c = (double)((need + d.blocks - 1) / d.blocks) * (3.5 + 0.25 * (d.tpw - 1));
        if (c <= cost) {
            best.q = d;
            best.k = QkDeal{0, d.tpw};
            best.wpt = 1;
            best.together = true;
        }
    }
    best.by_tokens = make_fastdiv((unsigned)r.tokens);
    return best;
}

// Heads on their way to a lane: as many as make 96 bytes.
constexpr int forward_stages(int bytes) { return 96 / bytes < 2 ? 2 : 96 / bytes; }

template <class T, bool INTERLEAVED, int W, int U, bool VEC, int GT>
__global__ void __launch_bounds__(32 * kQkWarps, kQkBlocks)
    qk_norm_rope_kernel(QkNormParams p, int g, QkShare sh) {
    using Head = HeadUnits<T, INTERLEAVED, W, U, VEC>;
    constexpr int kStages = forward_stages(U * Head::E * (int)sizeof(T));
    extern __shared__ uint4 smem[];  // [warps][stages] slots, the pairs' frequencies, [tokens of the block][pairs]
    const RopeParams& r = p.rope;
    const int G = GT ? GT : g, groups = 32 / G, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const QkPlace at(sh, r.q.heads, r.k.heads, G, groups, Bool<true>());
    const RopeTensor& t = at.k ? r.k : r.q;
    const unsigned tokens = (unsigned)r.tokens, total = (unsigned)r.batch * tokens;
    const Head head(lane % G, G, r.hd, r.pairs);
    PairFreq* freqs = reinterpret_cast<PairFreq*>(reinterpret_cast<char*>(smem) + kQkWarps * kStages * Head::kSlotBytes);
    float2* cs = reinterpret_cast<float2*>(freqs + r.pairs) + at.slot * at.tpw * r.pairs;
    HeadStream<Head, T, 1, kStages> in(
        head, at, (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * Head::kSlotBytes + lane * Head::kAccessBytes, r,
        t.heads, sh.by_tokens);
    in.tensor(0, t.in, t.ib, t.it, t.ih);
    typename Head::Raw raw[1];
    raw[0].clear();
    grid_dep_wait();
    grid_dep_launch();
    in.start();
    for (int j = threadIdx.x; j < r.pairs; j += blockDim.x) freqs[j] = pair_freq(r, j);
    __syncthreads();
    TokenAngles angle(r, freqs, cs, at.share, sh.wpt, at.tpw, total, sh.by_tokens);
    angle.fetch(at.tok - at.sub);
    const typename Head::Values w = head.weight(p.w[at.k], p.w_f32);

    // the same number of rounds for all warps of the block, which may meet in them
    const unsigned first = at.block * (kQkWarps / sh.wpt) * at.tpw;
#pragma unroll 1
    for (unsigned round = first, tok = at.tok; round < total; round += at.stride, tok += at.stride) {
        angle.make(tok - at.sub);
        angle.fetch(tok - at.sub + at.stride);
        if (tok - at.sub >= total) continue;
        const bool has = tok < total;
        const unsigned b = has ? batch_of(tok, sh.by_tokens) : 0, s = has ? tok - b * tokens : 0;
        const typename Head::Turn turn = head.turn_of(cs + at.sub * r.pairs, w);
        T* out = static_cast<T*>(t.out) + b * t.ob + s * t.ot + at.h0 * t.oh;
#pragma unroll 1
        for (int i = 0; i < in.steps; ++i, out += at.step * t.oh) {
            in.take(raw);
            typename Head::Values x = Head::values(raw[0]);
            const float ss = group_sum<GT>(dot(x.first, x.second, x), G);
            in.fetch();
            const float rstd = rsqrtf(__fmaf_rn(ss, p.inv_hd, p.eps));
            const u64 r2 = f2(rstd, rstd);
            head.turn(x, turn);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < Head::NP; ++j) {
                    x.first[u][j] = mul2(x.first[u][j], r2);
                    x.second[u][j] = mul2(x.second[u][j], r2);
                }
            if (has && i < in.mine) head.store(out, x);
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
        constexpr int kStages = forward_stages(Head::E * decltype(u)::value * (int)sizeof(t));
        const QkShare sh = qk_share(r, kQkBlocks * (int64_t)sm_count(), 32 / shape.g, true);
        auto* k = qk_norm_rope_kernel<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value,
                                      decltype(vec)::value, decltype(gt)::value>;
        const int most = sh.q.tpw > sh.k.tpw ? sh.q.tpw : sh.k.tpw;
        const size_t smem = kQkWarps * kStages * Head::kSlotBytes + r.pairs * sizeof(PairFreq) +
                            kQkWarps / sh.wpt * most * r.pairs * sizeof(float2);
        static SmemOptIn opt;
        if (cudaError_t e = allow_smem(opt, reinterpret_cast<const void*>(k), smem)) return e;
        return launch_pdl(k, (unsigned)(sh.q.blocks + sh.k.blocks), 32 * kQkWarps, smem, s, p, shape.g, sh);
    });
}

cudaError_t launch_qk_norm_rope(const QkNormParams& p, bool f32, bool interleaved, int align, cudaStream_t s) {
    return interleaved ? forward<true>(p, f32, align, s) : forward<false>(p, f32, align, s);
}

}  // namespace mbx
