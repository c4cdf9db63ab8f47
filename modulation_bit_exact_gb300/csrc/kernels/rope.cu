// rope.cu -- rotary positions on several axes (time, height, width), for Q and
// K in one launch.
//
// A head's first 2n elements form n pairs, (2j, 2j+1) interleaved or (j, j+n)
// in halves; the pairs are dealt to the axes in order, and pair j of axis a
// turns by position[token][a] * freq[j]:
//   o0 = x0*cos - x1*sin,  o1 = x0*sin + x1*cos
// or by the opposite angle (inverse), which is also the gradient of the
// rotation.  Elements past 2n pass through.
//
// The angle is formed in binary64 and reduced to an eighth of a turn there, so
// a far position loses nothing; sine and cosine of the remainder and the
// rotation are binary32, rounded once at the output.
//
// A block takes a few tokens: it computes each token's n sines and cosines
// once, in shared memory, then its threads walk the heads of Q and K, one
// 16-byte chunk (two in halves) of a head at a time.  Memory bound: every
// element is read once and written once.
#include "rowgroup.cuh"

namespace mbx {

// cos and sin of 2*pi*turns.
__device__ __forceinline__ float2 cos_sin_turns(double turns) {
    const double q = turns * 4.0, r = rint(q);
    const int quadrant = (int)(long long)r & 3;
    float s, c;
    sincospif((float)(q - r) * 0.5f, &s, &c);  // |argument| <= 1/4
    const float cc = (quadrant & 1) ? -s : c, ss = (quadrant & 1) ? c : s;
    return (quadrant & 2) ? make_float2(-cc, -ss) : make_float2(cc, ss);
}

// Threads of a block: tl = t % lanes is the lane within a head, t / lanes the
// (token, head split) slot.  VEC interleaved: a lane is one 16-byte chunk; in
// halves: a lane below half is the chunk pair (c, c + n), the rest pass-through
// chunks.  Scalar: a lane is a pair, or one pass-through element.
template <class T, bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(256) rope_axes_kernel(RopeParams p, int lanes, int tok_per_block, int splits) {
    extern __shared__ float2 cs[];  // [tok_per_block][pairs]
    constexpr int CE = ChunkOf<T>::CE;
    grid_dep_wait();  // launched programmatically: the previous kernel has finished
    grid_dep_launch();
    const int64_t total = p.batch * p.tokens;
    const int64_t tok0 = (int64_t)blockIdx.x * tok_per_block;
    const int n = p.pairs;
    for (int i = threadIdx.x; i < tok_per_block * n; i += blockDim.x) {
        const int k = i / n, j = i - k * n;
        const int64_t tok = tok0 + k;
        if (tok >= total) break;
        int a = 0;
        while (a < p.axes - 1 && j >= p.axis_end[a]) ++a;
        const int64_t prow = p.pos_batched ? tok : tok % p.tokens;
        const double pos = p.pos_f32 ? (double)static_cast<const float*>(p.pos)[prow * p.pos_stride + a]
                                     : (double)static_cast<const int*>(p.pos)[prow * p.pos_stride + a];
        float2 v = cos_sin_turns(pos * (p.freqs[j] * 0.15915494309189533577));  // 1 / (2 pi)
        if (p.inverse) v.y = -v.y;
        cs[i] = v;
    }
    __syncthreads();
    const int lane = threadIdx.x % lanes, slot = threadIdx.x / lanes;
    const int k = slot / splits, split = slot - k * splits;
    const int64_t tok = tok0 + k;
    if (k >= tok_per_block || tok >= total) return;
    const int64_t b = tok / p.tokens, s = tok - b * p.tokens;
    const float2* my = cs + k * n;

    const int heads = p.q.heads + p.k.heads;
    for (int h0 = split; h0 < heads; h0 += splits) {
        const bool is_k = h0 >= p.q.heads;
        const RopeTensor& w = is_k ? p.k : p.q;
        const int h = is_k ? h0 - p.q.heads : h0;
        const T* in = static_cast<const T*>(w.in) + b * w.ib + s * w.it + h * w.ih;
        T* out = static_cast<T*>(w.out) + b * w.ob + s * w.ot + h * w.oh;
        if constexpr (VEC && INTERLEAVED) {
            const uint4 raw = ld_stream_rw(in + lane * CE);
            float v[CE];
            widen_chunk(raw, v);
#pragma unroll
            for (int i = 0; i < CE; i += 2) {
                const int j = (lane * CE + i) / 2;
                if (j < n) {
                    const float2 c = my[j];
                    const float a0 = v[i], a1 = v[i + 1];
                    v[i] = fmaf(a0, c.x, -(a1 * c.y));
                    v[i + 1] = fmaf(a0, c.y, a1 * c.x);
                }
            }
            st_v4(out + lane * CE, narrow_chunk(v));
        } else if constexpr (VEC) {
            const int half = n / CE;  // chunks of the first half of the pairs
            if (lane < half) {
                const uint4 ra = ld_stream_rw(in + lane * CE), rb = ld_stream_rw(in + n + lane * CE);
                float va[CE], vb[CE];
                widen_chunk(ra, va);
                widen_chunk(rb, vb);
#pragma unroll
                for (int i = 0; i < CE; ++i) {
                    const float2 c = my[lane * CE + i];
                    const float a0 = va[i], a1 = vb[i];
                    va[i] = fmaf(a0, c.x, -(a1 * c.y));
                    vb[i] = fmaf(a0, c.y, a1 * c.x);
                }
                st_v4(out + lane * CE, narrow_chunk(va));
                st_v4(out + n + lane * CE, narrow_chunk(vb));
            } else {
                const int c = 2 * n + (lane - half) * CE;
                st_v4(out + c, ld_stream_rw(in + c));
            }
        } else {
            if (lane < n) {
                const int e0 = INTERLEAVED ? 2 * lane : lane, e1 = INTERLEAVED ? 2 * lane + 1 : lane + n;
                const float a0 = load_elem(in + e0), a1 = load_elem(in + e1);
                const float2 c = my[lane];
                store_elem(out + e0, fmaf(a0, c.x, -(a1 * c.y)));
                store_elem(out + e1, fmaf(a0, c.y, a1 * c.x));
            } else {
                const int c = 2 * n + (lane - n);
                store_elem(out + c, load_elem(in + c));
            }
        }
    }
}

template <class T, bool INTERLEAVED, bool VEC>
static cudaError_t launch_rope(const RopeParams& p, cudaStream_t s) {
    constexpr int CE = ChunkOf<T>::CE;
    const int lanes = !VEC ? p.hd - p.pairs : INTERLEAVED ? p.hd / CE : p.pairs / CE + (p.hd - 2 * p.pairs) / CE;
    // a slot is a token's share of the heads; a block has as many as fit in 256 threads
    const int slots = lanes >= 256 ? 1 : 256 / lanes;
    const int heads = p.q.heads + p.k.heads;
    const int splits = slots < 4 ? slots : heads < 4 ? heads : 4;
    const int tok_per_block = slots / splits;
    const int64_t total = p.batch * p.tokens, grid = (total + tok_per_block - 1) / tok_per_block;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    const int block = (lanes * splits * tok_per_block + 31) / 32 * 32;
    const size_t smem = (size_t)tok_per_block * p.pairs * sizeof(float2);
    return launch_pdl(rope_axes_kernel<T, INTERLEAVED, VEC>, (unsigned)grid, block, smem, s, p, lanes, tok_per_block, splits);
}

template <class T>
static cudaError_t rope_t(const RopeParams& p, bool interleaved, bool vec, cudaStream_t s) {
    if (interleaved) return vec ? launch_rope<T, true, true>(p, s) : launch_rope<T, true, false>(p, s);
    return vec ? launch_rope<T, false, true>(p, s) : launch_rope<T, false, false>(p, s);
}

cudaError_t launch_rope_axes(const RopeParams& p, bool f32, bool interleaved, bool vec, cudaStream_t s) {
    return f32 ? rope_t<float>(p, interleaved, vec, s) : rope_t<uint16_t>(p, interleaved, vec, s);
}

}  // namespace mbx
