// qknorm_bwd.cu -- gradients of qknorm.cu.  With g = dout turned back, xh = x * rstd
// and gy = g * w:
//   dx = rstd * (gy - xh * mean(gy * xh)),   dw = sum over batch, tokens and heads of g * xh
// Statistics are taken from x again.  mean(gy * xh) = rstd * mean(gy * x), so
// both row sums are formed in one exchange.
//
// A warp walks tokens (a share of the heads each where they are few), first
// those of Q and then those of K, and keeps its lanes' part of dw in registers;
// a block adds its warps' parts in shared memory, and column_sums (colsum.cu)
// the blocks' parts, in a fixed order.
#include <type_traits>

#include "qknorm.cuh"

namespace mbx {

constexpr int kQkGradWarps = 8;

template <class T, bool INTERLEAVED, int W, int U, bool VEC>
__global__ void __launch_bounds__(32 * kQkGradWarps) qk_norm_rope_bwd_kernel(QkNormParams p, int G, int splits) {
    using Head = HeadUnits<T, INTERLEAVED, W, U, VEC>;
    constexpr int E = Head::E, P = Head::P;
    constexpr int kAtOnce = U * E <= 8 ? 2 : 1;  // heads of a group in flight
    extern __shared__ float2 cs_smem[];          // [warps][pairs], then the block's [warps][hd] sums
    const RopeParams& r = p.rope;
    const int n = r.pairs, hd = r.hd, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const unsigned tokens = (unsigned)r.tokens, total = (unsigned)r.batch * tokens;
    const int in_head = lane % G, groups = 32 / G;
    const Head head(in_head, G, hd, n);
    const int64_t units = (int64_t)total * splits, stride = (int64_t)gridDim.x * kQkGradWarps;
    float2* cs = cs_smem + warp * n;
    float* sums = reinterpret_cast<float*>(cs_smem + kQkGradWarps * n);
    grid_dep_wait();
    grid_dep_launch();

#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const RopeTensor& t = which ? r.k : r.q;
        if (t.heads == 0) break;
        const GradIn& d = p.dout[which];
        float w[U][E], acc[U][E];
        head.weight(w, p.w[which], p.w_f32);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[u][e] = 0.0f;
#pragma unroll 1
        for (int64_t unit = (int64_t)blockIdx.x * kQkGradWarps + warp; unit < units; unit += stride) {
            const unsigned tok = (unsigned)(unit / splits), b = tok / tokens, s = tok - b * tokens;
            const int h0 = (int)(unit - (int64_t)tok * splits) * groups + lane / G, step = splits * groups;
            const T* x_in = static_cast<const T*>(t.in) + b * t.ib + s * t.it;
            const T* g_in = static_cast<const T*>(d.in) + b * d.ib + s * d.it;
            T* out = static_cast<T*>(t.out) + b * t.ob + s * t.ot;
            typename Head::Raw rx[kAtOnce], rg[kAtOnce];
            auto fetch = [&](int h) {
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (h + i * step < t.heads) {
                        head.load(rx[i], x_in + (h + i * step) * t.ih);
                        head.load(rg[i], g_in + (h + i * step) * d.ih);
                    }
            };
            fetch(h0);
            __syncwarp();
            for (int j = lane; j < n; j += 32) cs[j] = token_cos_sin(r, tok, s, j);
            __syncwarp();
            float c[U][P], sn[U][P];
            head.angles(c, sn, cs);
#pragma unroll 1
            for (int h = h0; h - lane / G < t.heads; h += kAtOnce * step) {
                if (h != h0) fetch(h);
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const bool has = h + i * step < t.heads;
                    float x[U][E], g[U][E];
                    head.values(x, rx[i]);
                    head.values(g, rg[i]);
                    head.turn(g, c, sn);
                    float ss = 0.0f, gx = 0.0f;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            ss = __fmaf_rn(x[u][e], x[u][e], ss);
                            gx = __fmaf_rn(g[u][e] * w[u][e], x[u][e], gx);
                        }
                    const float rstd = 1.0f / sqrtf(group_sum(ss, G) * p.inv_hd + p.eps);
                    const float c2 = group_sum(gx, G) * p.inv_hd * rstd;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const float xh = x[u][e] * rstd, gy = g[u][e] * w[u][e];
                            if (has) acc[u][e] = __fmaf_rn(g[u][e], xh, acc[u][e]);
                            x[u][e] = rstd * __fmaf_rn(-xh, c2, gy);
                        }
                    if (has) head.store(out + (h + i * step) * t.oh, x);
                }
            }
        }
        if (!p.ws) continue;
        // the warp's groups side by side, then the block's warps in order
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                for (int m = G; m < 32; m <<= 1) acc[u][e] += __shfl_xor_sync(0xffffffffu, acc[u][e], m);
            }
            if (lane < G) {
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if (head.off0[u] >= 0) sums[warp * hd + head.off0[u] + i] = acc[u][i];
                    if constexpr (Head::kTwo)
                        if (head.off1[u] >= 0) sums[warp * hd + head.off1[u] + i] = acc[u][W + i];
                }
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < hd; e += blockDim.x) {
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < kQkGradWarps; ++i) a += sums[i * hd + e];
            p.ws[((int64_t)blockIdx.x * 2 + which) * hd + e] = a;
        }
        __syncthreads();
    }
}

int64_t qk_norm_grad_parts(int64_t batch, int64_t tokens) {
    const int64_t blocks = (batch * tokens + kQkGradWarps - 1) / kQkGradWarps, most = 3 * (int64_t)sm_count();
    return blocks < most ? blocks : most;
}

cudaError_t launch_qk_norm_rope_backward(const QkNormParams& p, bool f32, bool interleaved, int align, const ColSumParams& sums,
                                         cudaStream_t s) {
    const RopeParams& r = p.rope;
    const int64_t parts = qk_norm_grad_parts(r.batch, r.tokens);
    const cudaError_t e = for_head_shape(r.hd, r.pairs, f32, interleaved, align,
                                         [&](auto t, auto inter, auto w, auto u, auto vec, int G) {
        auto* k = qk_norm_rope_bwd_kernel<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value,
                                          decltype(vec)::value>;
        const size_t smem = kQkGradWarps * (r.pairs * sizeof(float2) + r.hd * sizeof(float));
        return launch_pdl(k, (unsigned)parts, 32 * kQkGradWarps, smem, s, p, G, 1);
    });
    if (e != cudaSuccess || !p.ws) return e;
    return launch_column_sums(sums, s);
}

}  // namespace mbx
