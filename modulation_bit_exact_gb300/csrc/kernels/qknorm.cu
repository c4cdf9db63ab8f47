// qknorm.cu -- RMSNorm of every head of Q and K and the rotation by positions on
// several axes, in one pass:
//   n = x * rstd * w,  rstd = 1 / sqrt(mean(x^2) + eps) over the head,
//   out = the pairs of n turned as in rope.cu; elements past the pairs pass.
// binary32, one rounding at the output.
//
// A warp takes one token, or a share of its heads where tokens are few: with the
// other warps of the token it computes the sines and cosines once, keeps its own in
// registers and walks the heads, 32 / G of them side by side (qknorm.cuh).
#include "qknorm.cuh"

namespace mbx {

template <class T, bool INTERLEAVED, int W, int U, bool VEC, int GT>
__global__ void __launch_bounds__(32 * kQkWarps) qk_norm_rope_kernel(QkNormParams p, int g, int wpt) {
    using Head = HeadUnits<T, INTERLEAVED, W, U, VEC>;
    constexpr int kAtOnce = U * Head::E <= 8 ? 4 : U * Head::E <= 16 ? 2 : 1;  // heads of a group in flight
    extern __shared__ float2 cs_smem[];                                        // [tokens of the block][pairs]
    const RopeParams& r = p.rope;
    const int G = GT ? GT : g, groups = 32 / G;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, slot = warp / wpt, share = warp % wpt;
    const unsigned tokens = (unsigned)r.tokens, total = (unsigned)r.batch * tokens;
    const unsigned tok = blockIdx.x * (unsigned)(kQkWarps / wpt) + slot;
    const Head head(lane % G, G, r.hd, r.pairs);
    grid_dep_wait();
    grid_dep_launch();
    const bool has = tok < total;
    const unsigned b = has ? tok / tokens : 0, s = has ? tok - b * tokens : 0;
    const int h0 = share * groups + lane / G, step = wpt * groups;

    typename Head::Raw raw[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) raw[i].clear();
    const T* in = static_cast<const T*>(r.q.in) + b * r.q.ib + s * r.q.it;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
        if (has && h0 + i * step < r.q.heads) head.load(raw[i], in + (h0 + i * step) * r.q.ih);
    float2* cs = cs_smem + slot * r.pairs;
    token_angles(cs, r, tok, s, has, share, wpt);
    if (!has) return;
    const typename Head::Angles angles = head.angles(cs);

#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const RopeTensor& t = which ? r.k : r.q;
        if (t.heads == 0) break;
        const typename Head::Values w = head.weight(p.w[which], p.w_f32);
        in = static_cast<const T*>(t.in) + b * t.ib + s * t.it;
        T* out = static_cast<T*>(t.out) + b * t.ob + s * t.ot;
        // every lane of the warp takes part in the sums, also one past the last head
#pragma unroll 1
        for (int h = h0; h - lane / G < t.heads; h += kAtOnce * step) {
            if (which || h != h0) {
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (h + i * step < t.heads) head.load(raw[i], in + (h + i * step) * t.ih);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                typename Head::Values x = Head::values(raw[i]);
                const float ss = group_sum<GT>(dot(x.first, x.second, x), G);
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
                if (h + i * step < t.heads) head.store(out + (h + i * step) * t.oh, x);
            }
        }
    }
}

cudaError_t launch_qk_norm_rope(const QkNormParams& p, bool f32, bool interleaved, int align, cudaStream_t s) {
    const RopeParams& r = p.rope;
    return for_head_shape(r.hd, r.pairs, f32, interleaved, align,
                          [&](auto t, auto inter, auto w, auto u, auto vec, auto gt, int G) {
        const int64_t total = r.batch * r.tokens;
        const int most = r.q.heads > r.k.heads ? r.q.heads : r.k.heads;
        int wpt = 1;
        while (wpt < kQkWarps && wpt * (32 / G) < most && total * wpt < 8 * sm_count()) wpt *= 2;
        const int64_t per_block = kQkWarps / wpt, grid = (total + per_block - 1) / per_block;
        auto* k = qk_norm_rope_kernel<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value,
                                      decltype(vec)::value, decltype(gt)::value>;
        return launch_pdl(k, (unsigned)grid, 32 * kQkWarps, per_block * r.pairs * sizeof(float2), s, p, G, wpt);
    });
}

}  // namespace mbx
