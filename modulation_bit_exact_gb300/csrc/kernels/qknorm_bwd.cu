// qknorm_bwd.cu -- gradients of qknorm.cu.  With g = dout turned back, xh = x * rstd
// and gy = g * w:
//   dx = rstd * (gy - xh * mean(gy * xh)),   dw = sum over batch, tokens and heads of g * xh
// Statistics are taken from x again.  mean(gy * xh) = rstd * mean(gy * x), so
// both row sums are formed in one exchange.
//
// A warp walks tokens (a share of the heads each, where that divides the tokens
// better among the warps), first those of Q and then those of K, and keeps its
// lanes' part of dw in registers; a block adds its warps' parts in shared memory,
// and column_sums (colsum.cu) the blocks' parts, in a fixed order.
#include "qknorm.cuh"

namespace mbx {

// Blocks of an SM, by the elements of a head that a lane holds: what the registers allow.
constexpr int kQkGradBlocks = 3;
constexpr int grad_blocks(int elems) { return elems <= 8 ? kQkGradBlocks : elems <= 16 ? 2 : 1; }

template <class T, bool INTERLEAVED, int W, int U, bool VEC, int GT>
__global__ void __launch_bounds__(32 * kQkWarps, grad_blocks(HeadUnits<T, INTERLEAVED, W, U, VEC>::E * U))
    qk_norm_rope_bwd_kernel(QkNormParams p, int g, int wpt) {
    using Head = HeadUnits<T, INTERLEAVED, W, U, VEC>;
    constexpr int E = Head::E, NP = Head::NP;
    constexpr int kAtOnce = U * E <= 8 ? 2 : 1;  // heads of a group in flight
    extern __shared__ float2 cs_smem[];          // [tokens of the block][pairs], then [warps][hd] sums
    const RopeParams& r = p.rope;
    const int G = GT ? GT : g, groups = 32 / G, hd = r.hd;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, slot = warp / wpt, share = warp % wpt;
    const unsigned tokens = (unsigned)r.tokens, total = (unsigned)r.batch * tokens;
    const unsigned per_block = kQkWarps / wpt, stride = gridDim.x * per_block;
    const Head head(lane % G, G, hd, r.pairs);
    float2* cs = cs_smem + slot * r.pairs;
    float* sums = reinterpret_cast<float*>(cs_smem + per_block * r.pairs);
    typename Head::Raw rx[kAtOnce], rg[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
        rx[i].clear();
        rg[i].clear();
    }
    const int h0 = share * groups + lane / G, step = wpt * groups;
    grid_dep_wait();
    grid_dep_launch();

#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const RopeTensor& t = which ? r.k : r.q;
        if (t.heads == 0) break;
        const GradIn& d = p.dout[which];
        const typename Head::Values w = head.weight(p.w[which], p.w_f32);
        typename Head::Values acc;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NP; ++j) acc.first[u][j] = acc.second[u][j] = 0;
        // the same number of rounds for all warps of the block, which may meet in them
#pragma unroll 1
        for (unsigned tok0 = blockIdx.x * per_block; tok0 < total; tok0 += stride) {
            const unsigned tok = tok0 + slot;
            const bool has = tok < total;
            const unsigned b = has ? tok / tokens : 0, s = has ? tok - b * tokens : 0;
            const int heads = has ? t.heads : 0;
            const T* x_in = static_cast<const T*>(t.in) + b * t.ib + s * t.it;
            const T* g_in = static_cast<const T*>(d.in) + b * d.ib + s * d.it;
            T* out = static_cast<T*>(t.out) + b * t.ob + s * t.ot;
            auto fetch = [&](int h) {
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (h + i * step < heads) {
                        head.load(rx[i], x_in + (h + i * step) * t.ih);
                        head.load(rg[i], g_in + (h + i * step) * d.ih);
                    }
            };
            fetch(h0);
            token_angles(cs, r, tok, s, has, share, wpt);
            const typename Head::Angles angles = head.angles(cs);
#pragma unroll 1
            for (int h = h0; h - lane / G < heads; h += kAtOnce * step) {
                if (h != h0) fetch(h);
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const bool real = h + i * step < heads;
                    typename Head::Values x = Head::values(rx[i]), gr = Head::values(rg[i]), gy;
                    head.turn(gr, angles);
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int j = 0; j < NP; ++j) {
                            gy.first[u][j] = mul2(gr.first[u][j], w.first[u][j]);
                            gy.second[u][j] = mul2(gr.second[u][j], w.second[u][j]);
                        }
                    const float ss = group_sum<GT>(dot(x.first, x.second, x), G);
                    const float gx = group_sum<GT>(dot(gy.first, gy.second, x), G);
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
                    if (real) head.store(out + (h + i * step) * t.oh, x);
                }
            }
        }
        if (!p.ws) continue;
        // the warp's groups side by side, then the block's warps in order
        float a[U][E];
        Head::unpack(a, acc);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                for (int m = G; m < 32; m <<= 1) a[u][e] += __shfl_xor_sync(0xffffffffu, a[u][e], m);
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
        for (int e = threadIdx.x; e < hd; e += blockDim.x) {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < kQkWarps; ++i) v += sums[i * hd + e];
            p.ws[((int64_t)blockIdx.x * 2 + which) * hd + e] = v;
        }
        __syncthreads();
    }
}

// Warps a token and blocks: the fewest rounds of tokens, a share of a token's heads
// counting by its size and a tenth of the token for what every share pays.
struct QkGradPlan {
    int wpt;
    int64_t blocks;
};
static QkGradPlan qk_grad_plan(int64_t total, int per_sm) {
    const int64_t most = (int64_t)per_sm * sm_count();
    QkGradPlan best = {1, 1};
    double cost = 1e30;
    for (int wpt = 1; wpt <= kQkWarps; wpt *= 2) {
        const int64_t per_block = kQkWarps / wpt, need = (total + per_block - 1) / per_block;
        const int64_t blocks = need < most ? need : most;
        const double c = (double)((need + blocks - 1) / blocks) * (1.0 / wpt + 0.1);
        if (c < cost) {
            cost = c;
            best = QkGradPlan{wpt, blocks};
        }
    }
    return best;
}
int64_t qk_norm_grad_parts(int64_t batch, int64_t tokens) {
    int64_t parts = 0;  // the most that a head's shape may lead to
    for (int n = 1; n <= kQkGradBlocks; ++n) {
        const int64_t b = qk_grad_plan(batch * tokens, n).blocks;
        parts = b > parts ? b : parts;
    }
    return parts;
}

cudaError_t launch_qk_norm_rope_backward(const QkNormParams& p, bool f32, bool interleaved, int align, ColSumParams sums,
                                         cudaStream_t s) {
    const RopeParams& r = p.rope;
    const cudaError_t e = for_head_shape(r.hd, r.pairs, f32, interleaved, align,
                                         [&](auto t, auto inter, auto w, auto u, auto vec, auto gt, int G) {
        using Head = HeadUnits<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value, decltype(vec)::value>;
        const QkGradPlan plan = qk_grad_plan(r.batch * r.tokens, grad_blocks(Head::E * decltype(u)::value));
        sums.parts = plan.blocks;
        auto* k = qk_norm_rope_bwd_kernel<decltype(t), decltype(inter)::value, decltype(w)::value, decltype(u)::value,
                                          decltype(vec)::value, decltype(gt)::value>;
        const size_t smem = kQkWarps / plan.wpt * r.pairs * sizeof(float2) + kQkWarps * r.hd * sizeof(float);
        return launch_pdl(k, (unsigned)plan.blocks, 32 * kQkWarps, smem, s, p, G, plan.wpt);
    });
    if (e != cudaSuccess || !p.ws) return e;
    return launch_column_sums(sums, s);
}

}  // namespace mbx
