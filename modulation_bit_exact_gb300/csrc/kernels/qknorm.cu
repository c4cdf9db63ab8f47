// qknorm.cu -- RMSNorm of every head of Q and K and the rotation by positions on
// several axes, in one pass:
//   n = x * rstd * w,  rstd = 1 / sqrt(mean(x^2) + eps) over the head,
//   out = the pairs of n turned as in rope.cu; elements past the pairs pass.
// binary32, one rounding at the output.
//
// A warp takes one token, or a share of its heads where tokens are few: it
// computes the token's sines and cosines once, keeps its own in registers and
// walks the heads, 32 / G of them side by side (qknorm.cuh).  Memory bound.
#include <type_traits>

#include "qknorm.cuh"

namespace mbx {

constexpr int kQkWarps = 8;

template <class T, bool INTERLEAVED, int W, int U, bool VEC>
__global__ void __launch_bounds__(32 * kQkWarps) qk_norm_rope_kernel(QkNormParams p, int G, int splits) {
    using Head = HeadUnits<T, INTERLEAVED, W, U, VEC>;
    constexpr int E = Head::E, P = Head::P;
    constexpr int kAtOnce = U * E <= 8 ? 4 : U * E <= 16 ? 2 : 1;  // heads of a group in flight
    extern __shared__ float2 cs_smem[];                              // [warps][pairs]
    const RopeParams& r = p.rope;
    const int n = r.pairs, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const unsigned tokens = (unsigned)r.tokens, total = (unsigned)r.batch * tokens;
    const int64_t unit = (int64_t)blockIdx.x * kQkWarps + warp;
    const unsigned tok = (unsigned)(unit / splits);
    const int split = (int)(unit - (int64_t)tok * splits);
    const int in_head = lane % G, groups = 32 / G;
    const Head head(in_head, G, r.hd, n);
    grid_dep_wait();
    grid_dep_launch();
    if (unit >= (int64_t)total * splits) return;
    const unsigned b = tok / tokens, s = tok - b * tokens;
    const int h0 = split * groups + lane / G, step = splits * groups;

    typename Head::Raw raw[kAtOnce];
    const T* in = static_cast<const T*>(r.q.in) + b * r.q.ib + s * r.q.it;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
        if (h0 + i * step < r.q.heads) head.load(raw[i], in + (h0 + i * step) * r.q.ih);
    float2* cs = cs_smem + warp * n;
    for (int j = lane; j < n; j += 32) cs[j] = token_cos_sin(r, tok, s, j);
    __syncwarp();
    float c[U][P], sn[U][P];
    head.angles(c, sn, cs);

#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const RopeTensor& t = which ? r.k : r.q;
        if (t.heads == 0) break;
        float w[U][E];
        head.weight(w, p.w[which], p.w_f32);
        in = static_cast<const T*>(t.in) + b * t.ib + s * t.it;
        T* out = static_cast<T*>(t.out) + b * t.ob + s * t.ot;
        // every lane of the warp takes part in the sums: a group past the last head adds zeros
#pragma unroll 1
        for (int h = h0; h - lane / G < t.heads; h += kAtOnce * step) {
            if (which || h != h0) {
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (h + i * step < t.heads) head.load(raw[i], in + (h + i * step) * t.ih);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                float x[U][E];
                head.values(x, raw[i]);
                float ss = 0.0f;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < E; ++e) ss = __fmaf_rn(x[u][e], x[u][e], ss);
                const float rstd = 1.0f / sqrtf(group_sum(ss, G) * p.inv_hd + p.eps);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < E; ++e) x[u][e] = x[u][e] * rstd * w[u][e];
                head.turn(x, c, sn);
                if (h + i * step < t.heads) head.store(out + (h + i * step) * t.oh, x);
            }
        }
    }
}

cudaError_t launch_qk_norm_rope(const QkNormParams& p, bool f32, bool interleaved, int align, cudaStream_t s) {
    const RopeParams& r = p.rope;
    return for_head_shape(r.hd, r.pairs, f32, interleaved, align,
                          [&](auto t, auto inter, auto w, auto u, auto vec, int G) {
        const int64_t total = r.batch * r.tokens;
        const int most = r.q.heads > r.k.heads ? r.q.heads : r.k.heads, groups = 32 / G;
        int splits = 1;
        while (splits * groups < most && total * splits < 8 * sm_count()) splits *= 2;
        const int64_t grid = (total * splits + kQkWarps - 1) / kQkWarps;
        auto* k = qk_norm_rope_kernel<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value,
                                      decltype(vec)::value>;
        return launch_pdl(k, (unsigned)grid, 32 * kQkWarps, kQkWarps * r.pairs * sizeof(float2), s, p, G, splits);
    });
}

}  // namespace mbx
