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
// once, in shared memory; a thread then keeps those of its part of a head in
// registers and walks the heads of Q and K.  Memory bound: every element is
// read once and written once.
#include <type_traits>

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

// One lane's part of a head, and its rotation.  Vec, interleaved: one 16-byte
// chunk.  Vec, in halves: the chunk at c and the one at c + n; past the pairs, a
// chunk that passes through.  Scalar: one pair, or one element that passes.
template <class T, bool INTERLEAVED, bool VEC>
struct HeadPart {
    static constexpr int CE = ChunkOf<T>::CE;
    static constexpr int kPairs = VEC ? (INTERLEAVED ? CE / 2 : CE) : 1;
    static constexpr int kRaw = VEC && !INTERLEAVED ? 2 : 1;
    int first, second;  // offsets within a head; second < 0: none
    int pair0, pairs;   // pairs that turn: pair0 .. pair0 + pairs - 1
    __device__ __forceinline__ HeadPart(int lane, int n) {
        if constexpr (VEC && INTERLEAVED) {
            first = lane * CE;
            second = -1;
            pair0 = first / 2;
            pairs = min(max(n - pair0, 0), kPairs);
        } else if constexpr (VEC) {
            const bool turns = lane < n / CE;
            first = turns ? lane * CE : 2 * n + (lane - n / CE) * CE;
            second = turns ? first + n : -1;
            pair0 = first;
            pairs = turns ? CE : 0;
        } else {
            const bool turns = lane < n;
            first = turns ? (INTERLEAVED ? 2 * lane : lane) : n + lane;
            second = turns ? (INTERLEAVED ? first + 1 : first + n) : -1;
            pair0 = lane;
            pairs = turns ? 1 : 0;
        }
    }
    struct Raw {
        typename std::conditional<VEC, uint4, float>::type a, b;
    };
    __device__ __forceinline__ Raw load(const T* head) const {
        Raw r;
        if constexpr (VEC) {
            r.a = ld_stream_rw(head + first);
            if constexpr (!INTERLEAVED)
                if (second >= 0) r.b = ld_stream_rw(head + second);
        } else {
            r.a = load_elem(head + first);
            r.b = second >= 0 ? load_elem(head + second) : 0.0f;
        }
        return r;
    }
    __device__ __forceinline__ void store(T* head, const Raw& r, const float2 (&cs)[kPairs]) const {
        if constexpr (VEC && INTERLEAVED) {
            float v[CE];
            widen_chunk(r.a, v);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const float a0 = v[2 * i], a1 = v[2 * i + 1];
                if (i < pairs) {
                    v[2 * i] = fmaf(a0, cs[i].x, -(a1 * cs[i].y));
                    v[2 * i + 1] = fmaf(a0, cs[i].y, a1 * cs[i].x);
                }
            }
            st_v4(head + first, narrow_chunk(v));
        } else if constexpr (VEC) {
            if (second < 0) {
                st_v4(head + first, r.a);
                return;
            }
            float va[CE], vb[CE];
            widen_chunk(r.a, va);
            widen_chunk(r.b, vb);
#pragma unroll
            for (int i = 0; i < CE; ++i) {
                const float a0 = va[i], a1 = vb[i];
                va[i] = fmaf(a0, cs[i].x, -(a1 * cs[i].y));
                vb[i] = fmaf(a0, cs[i].y, a1 * cs[i].x);
            }
            st_v4(head + first, narrow_chunk(va));
            st_v4(head + second, narrow_chunk(vb));
        } else if (second < 0) {
            store_elem(head + first, r.a);
        } else {
            store_elem(head + first, fmaf(r.a, cs[0].x, -(r.b * cs[0].y)));
            store_elem(head + second, fmaf(r.a, cs[0].y, r.b * cs[0].x));
        }
    }
};

constexpr int kHeadsAtOnce = 4;  // heads of a thread in flight

// Thread: lane within a head, then the share (1 of `splits`) of the heads, then
// the token of the block.
template <class T, bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(256) rope_axes_kernel(RopeParams p, int lanes, int tok_per_block, int splits) {
    using Part = HeadPart<T, INTERLEAVED, VEC>;
    extern __shared__ float2 cs_smem[];  // [tok_per_block][pairs]
    const int n = p.pairs;
    const unsigned tokens = (unsigned)p.tokens, total = (unsigned)p.batch * tokens;
    const unsigned tok0 = blockIdx.x * (unsigned)tok_per_block;
    const int lane = threadIdx.x % lanes, slot = threadIdx.x / lanes;
    const int k = slot / splits, split = slot - k * splits;
    const unsigned tok = tok0 + k;
    const bool active = k < tok_per_block && tok < total;
    const unsigned b = tok / tokens, s = tok - b * tokens;
    const Part part(lane, n);
    grid_dep_wait();  // launched programmatically: the previous kernel has finished
    grid_dep_launch();

    // the first heads are on their way while the sines and cosines are computed
    auto head_in = [&](const RopeTensor& w, int h) {
        return static_cast<const T*>(w.in) + b * w.ib + s * w.it + h * w.ih;
    };
    auto head_out = [&](const RopeTensor& w, int h) {
        return static_cast<T*>(w.out) + b * w.ob + s * w.ot + h * w.oh;
    };
    typename Part::Raw raw[kHeadsAtOnce];
    if (active) {
#pragma unroll
        for (int u = 0; u < kHeadsAtOnce; ++u)
            if (split + u * splits < p.q.heads) raw[u] = part.load(head_in(p.q, split + u * splits));
    }
    for (int i = threadIdx.x; i < tok_per_block * n; i += blockDim.x) {
        const int kk = i / n, j = i - kk * n;
        const unsigned tk = tok0 + kk;
        if (tk >= total) break;
        int a = 0;
        while (a < p.axes - 1 && j >= p.axis_end[a]) ++a;
        const int64_t prow = p.pos_batched ? tk : tk % tokens;
        const double pos = p.pos_f32 ? (double)static_cast<const float*>(p.pos)[prow * p.pos_stride + a]
                                     : (double)static_cast<const int*>(p.pos)[prow * p.pos_stride + a];
        float2 v = cos_sin_turns(pos * (p.freqs[j] * 0.15915494309189533577));  // 1 / (2 pi)
        if (p.inverse) v.y = -v.y;
        cs_smem[i] = v;
    }
    __syncthreads();
    if (!active) return;
    float2 cs[Part::kPairs];
#pragma unroll
    for (int i = 0; i < Part::kPairs; ++i)
        cs[i] = i < part.pairs ? cs_smem[k * n + part.pair0 + i] : make_float2(1.0f, 0.0f);

    const int batch = kHeadsAtOnce * splits;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const RopeTensor& w = which ? p.k : p.q;
#pragma unroll 1
        for (int h0 = split; h0 < w.heads; h0 += batch) {
            if (which || h0 != split) {
#pragma unroll
                for (int u = 0; u < kHeadsAtOnce; ++u)
                    if (h0 + u * splits < w.heads) raw[u] = part.load(head_in(w, h0 + u * splits));
            }
#pragma unroll
            for (int u = 0; u < kHeadsAtOnce; ++u)
                if (h0 + u * splits < w.heads) part.store(head_out(w, h0 + u * splits), raw[u], cs);
        }
    }
}

template <class T, bool INTERLEAVED, bool VEC>
static cudaError_t launch_rope(const RopeParams& p, cudaStream_t s) {
    constexpr int CE = ChunkOf<T>::CE;
    const int lanes = !VEC ? p.hd - p.pairs : INTERLEAVED ? p.hd / CE : p.pairs / CE + (p.hd - 2 * p.pairs) / CE;
    // a slot is a token's share of the heads; a block has as many as fit in 256 threads
    const int slots = lanes >= 256 ? 1 : 256 / lanes;
    const int64_t total = p.batch * p.tokens;
    const int most = p.q.heads > p.k.heads ? p.q.heads : p.k.heads;
    int splits = slots < 4 ? slots : 4;
    // few tokens: spread each over more threads while the SMs are not full
    while (splits * 2 <= slots && (total * splits + slots - 1) / slots < 2 * sm_count()) splits *= 2;
    if (splits > most) splits = most;
    const int tok_per_block = slots / splits;
    const int64_t grid = (total + tok_per_block - 1) / tok_per_block;
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
