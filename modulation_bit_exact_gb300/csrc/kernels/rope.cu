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
// read once and written once (32760 tokens of 40 heads of 128, Q and K,
// bfloat16: 200 us, 6.7 TB/s of 6.77 that a copy reaches).
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

// One lane's part of a head, and its rotation.  W elements an access (16 or 8
// bytes), interleaved: one access; in halves: the access at c and the one at
// c + n, or past the pairs one that passes through.  W = 1: one pair, or one
// element that passes.
template <class T, bool INTERLEAVED, int W>
struct HeadPart {
    static constexpr int kPairs = W == 1 ? 1 : INTERLEAVED ? W / 2 : W;
    static constexpr int NC = (kPairs + 1) / 2;                           // register pairs of cosines
    static constexpr int NW = W == 1 ? 1 : W * (int)sizeof(T) / 4;        // words of an access
    // heads of a thread in flight; halves hold two accesses of each (4000 tokens of
    // 48 heads of 128: four heads 25.4 us, two 19.0)
    static constexpr int kHeadsAtOnce = INTERLEAVED || W == 1 ? 4 : 2;
    int first, second;  // offsets within a head; second < 0: none
    int pair0, pairs;   // pairs that turn: pair0 .. pair0 + pairs - 1
    __device__ __forceinline__ HeadPart(int lane, int n) {
        if constexpr (W > 1 && INTERLEAVED) {
            first = lane * W;
            second = -1;
            pair0 = first / 2;
            pairs = min(max(n - pair0, 0), kPairs);
        } else if constexpr (W > 1) {
            const bool turns = lane < n / W;
            first = turns ? lane * W : 2 * n + (lane - n / W) * W;
            second = turns ? first + n : -1;
            pair0 = first;
            pairs = turns ? W : 0;
        } else {
            const bool turns = lane < n;
            first = turns ? (INTERLEAVED ? 2 * lane : lane) : n + lane;
            second = turns ? (INTERLEAVED ? first + 1 : first + n) : -1;
            pair0 = lane;
            pairs = turns ? 1 : 0;
        }
    }
    struct Raw {  // W = 1: binary32 bits
        uint32_t a[NW], b[NW];
    };
    static __device__ __forceinline__ void get(uint32_t (&w)[NW], const T* p) {
        if constexpr (W == 1) {
            w[0] = __float_as_uint(load_elem(p));
        } else if constexpr (NW == 4) {
            const uint4 v = ld_stream_rw(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
        }
    }
    static __device__ __forceinline__ void put(T* p, const uint32_t (&w)[NW]) {
        if constexpr (W == 1) store_elem(p, __uint_as_float(w[0]));
        else if constexpr (NW == 4) st_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
        else st_v2(p, w[0], w[1]);
    }
    __device__ __forceinline__ Raw load(const T* head) const {
        Raw r;
        get(r.a, head + first);
        if constexpr (W == 1 || !INTERLEAVED)
            if (second >= 0) get(r.b, head + second);
        return r;
    }
    // Elements 0 and 1 of pairs i and i+1 of an interleaved access, side by side.
    static __device__ __forceinline__ u64 elem(const uint32_t (&w)[NW], int i, int which) {
        const int j = i + 1 < kPairs ? i + 1 : i;
        if constexpr (sizeof(T) == 2) return which ? f2(hi_f(w[i]), hi_f(w[j])) : f2(lo_f(w[i]), lo_f(w[j]));
        else return f2(__uint_as_float(w[2 * i + which]), __uint_as_float(w[2 * j + which]));
    }
    // c, s: the cosines and sines of two neighbouring pairs each.
    __device__ __forceinline__ void store(T* head, const Raw& r, const u64 (&c)[NC], const u64 (&s)[NC]) const {
        uint32_t oa[NW], ob[NW];
        if constexpr (W > 1 && INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < kPairs; i += 2) {
                const u64 x0 = elem(r.a, i, 0), x1 = elem(r.a, i, 1);
                const u64 o0 = turn0(x0, x1, c[i / 2], s[i / 2]), o1 = turn1(x0, x1, c[i / 2], s[i / 2]);
                if constexpr (sizeof(T) == 2) {
                    oa[i] = pack_rn(f2lo(o0), f2lo(o1));
                    if (i + 1 < kPairs) oa[i + 1] = pack_rn(f2hi(o0), f2hi(o1));
                } else {
                    oa[2 * i] = __float_as_uint(f2lo(o0));
                    oa[2 * i + 1] = __float_as_uint(f2lo(o1));
                    if (i + 1 < kPairs) {
                        oa[2 * i + 2] = __float_as_uint(f2hi(o0));
                        oa[2 * i + 3] = __float_as_uint(f2hi(o1));
                    }
                }
            }
            if (pairs < kPairs) {  // the rest of the access passes through
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    if (i * kPairs / NW >= pairs) oa[i] = r.a[i];
            }
            put(head + first, oa);
        } else if (second < 0) {
            put(head + first, r.a);
        } else {
            if constexpr (W == 1) {
                const u64 x0 = f2(__uint_as_float(r.a[0]), 0.0f), x1 = f2(__uint_as_float(r.b[0]), 0.0f);
                oa[0] = (uint32_t)turn0(x0, x1, c[0], s[0]);
                ob[0] = (uint32_t)turn1(x0, x1, c[0], s[0]);
            } else if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const u64 x0 = widen2(r.a[i]), x1 = widen2(r.b[i]);
                    oa[i] = pack2_rn(turn0(x0, x1, c[i], s[i]));
                    ob[i] = pack2_rn(turn1(x0, x1, c[i], s[i]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < NW; i += 2) {
                    const u64 x0 = f2(__uint_as_float(r.a[i]), __uint_as_float(r.a[i + 1]));
                    const u64 x1 = f2(__uint_as_float(r.b[i]), __uint_as_float(r.b[i + 1]));
                    const u64 o0 = turn0(x0, x1, c[i / 2], s[i / 2]), o1 = turn1(x0, x1, c[i / 2], s[i / 2]);
                    oa[i] = (uint32_t)o0, oa[i + 1] = (uint32_t)(o0 >> 32);
                    ob[i] = (uint32_t)o1, ob[i + 1] = (uint32_t)(o1 >> 32);
                }
            }
            put(head + first, oa);
            put(head + second, ob);
        }
    }
    // x0*cos - x1*sin and x0*sin + x1*cos, each one product and one fused
    // multiply-add, written so that no access width lets ptxas fuse another pair
    static __device__ __forceinline__ u64 turn0(u64 x0, u64 x1, u64 c, u64 s) {
        return fma2(x1 ^ 0x8000000080000000ull, s, mul2(x0, c));
    }
    static __device__ __forceinline__ u64 turn1(u64 x0, u64 x1, u64 c, u64 s) {
        return fma2(x0, s, mul2(x1, c));
    }
};

// Thread: lane within a head, then the share (1 of `splits`) of the heads, then
// the token of the block.
template <class T, bool INTERLEAVED, int W>
__global__ void __launch_bounds__(256, 4) rope_axes_kernel(RopeParams p, int lanes, int tok_per_block, int splits) {
    using Part = HeadPart<T, INTERLEAVED, W>;
    constexpr int kHeadsAtOnce = Part::kHeadsAtOnce;
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
    const T* in = static_cast<const T*>(p.q.in) + b * p.q.ib + s * p.q.it + split * p.q.ih;
    int64_t in_step = splits * p.q.ih;
    typename Part::Raw raw[kHeadsAtOnce];
    if (active) {
#pragma unroll
        for (int u = 0; u < kHeadsAtOnce; ++u)
            if (split + u * splits < p.q.heads) raw[u] = part.load(in + u * in_step);
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
    u64 c[Part::NC], sn[Part::NC];
#pragma unroll
    for (int i = 0; i < Part::kPairs; i += 2) {
        const float2* q = cs_smem + k * n + part.pair0 + i;
        const float2 a = i < part.pairs ? q[0] : make_float2(1.0f, 0.0f);
        const float2 d = i + 1 < part.pairs ? q[1] : make_float2(1.0f, 0.0f);
        c[i / 2] = f2(a.x, d.x);
        sn[i / 2] = f2(a.y, d.y);
    }

#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const RopeTensor& w = which ? p.k : p.q;
        T* out = static_cast<T*>(w.out) + b * w.ob + s * w.ot + split * w.oh;
        const int64_t out_step = splits * w.oh;
        if (which) {
            in = static_cast<const T*>(w.in) + b * w.ib + s * w.it + split * w.ih;
            in_step = splits * w.ih;
        }
#pragma unroll 1
        for (int h0 = split; h0 < w.heads; h0 += kHeadsAtOnce * splits) {
            if (which || h0 != split) {
#pragma unroll
                for (int u = 0; u < kHeadsAtOnce; ++u)
                    if (h0 + u * splits < w.heads) raw[u] = part.load(in + u * in_step);
            }
#pragma unroll
            for (int u = 0; u < kHeadsAtOnce; ++u)
                if (h0 + u * splits < w.heads) part.store(out + u * out_step, raw[u], c, sn);
            in += kHeadsAtOnce * in_step;
            out += kHeadsAtOnce * out_step;
        }
    }
}

template <class T, bool INTERLEAVED, int W>
static cudaError_t launch_rope(const RopeParams& p, cudaStream_t s) {
    const int lanes = W == 1 ? p.hd - p.pairs : INTERLEAVED ? p.hd / W : (p.hd - p.pairs) / W;
    // a slot is a token's share of the heads; a block has as many as fit in 256 threads
    const int slots = lanes >= 256 ? 1 : 256 / lanes;
    const int64_t total = p.batch * p.tokens;
    const int most = p.q.heads > p.k.heads ? p.q.heads : p.k.heads;
    int splits = slots < 4 ? slots : 4;
    // few tokens: spread each over more threads until every SM has two blocks
    // (1000 tokens of 48 heads of 128: 5.8 us; until it has eight: 7.6)
    while (splits * 2 <= slots && (total * splits + slots - 1) / slots < 2 * sm_count()) splits *= 2;
    if (splits > most) splits = most;
    const int tok_per_block = slots / splits;
    const int64_t grid = (total + tok_per_block - 1) / tok_per_block;
    const int block = (lanes * splits * tok_per_block + 31) / 32 * 32;
    const size_t smem = (size_t)tok_per_block * p.pairs * sizeof(float2);
    return launch_pdl(rope_axes_kernel<T, INTERLEAVED, W>, (unsigned)grid, block, smem, s, p, lanes, tok_per_block, splits);
}

template <class T>
static cudaError_t rope_t(const RopeParams& p, bool interleaved, int align, cudaStream_t s) {
    // the widest access that every head's start, the width and (in halves) the
    // number of pairs are multiples of.  8 bytes against single elements: 4000
    // tokens of 48 heads of 80 of which 40 elements turn, in halves, 45 -> 21 us
    constexpr int W16 = 16 / (int)sizeof(T), W8 = 8 / (int)sizeof(T);
    auto fits = [&](int w) { return p.hd % w == 0 && (interleaved || p.pairs % w == 0); };
    if (align == 16 && fits(W16)) return interleaved ? launch_rope<T, true, W16>(p, s) : launch_rope<T, false, W16>(p, s);
    if (align >= 8 && fits(W8)) return interleaved ? launch_rope<T, true, W8>(p, s) : launch_rope<T, false, W8>(p, s);
    return interleaved ? launch_rope<T, true, 1>(p, s) : launch_rope<T, false, 1>(p, s);
}

cudaError_t launch_rope_axes(const RopeParams& p, bool f32, bool interleaved, int align, cudaStream_t s) {
    return f32 ? rope_t<float>(p, interleaved, align, s) : rope_t<uint16_t>(p, interleaved, align, s);
}

}  // namespace mbx
