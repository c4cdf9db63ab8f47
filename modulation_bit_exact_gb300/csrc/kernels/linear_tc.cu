// linear_tc.cu -- the NVFP4 product on the tensor cores, without decoding the weight.
//
// tcgen05.mma.kind::mxf4nvf4 multiplies E2M1 values with an E4M3 scale for every 16
// of them: the weight goes from memory to the tensor cores as it is stored, by TMA,
// and its scales, whose tiles of 128 x 4 are the order that the tensor memory
// wants, by tcgen05.cp.  So the few activations have to be E2M1 too.  They are cut
// into digits: a block of 16 with |x| < 2^e is x = 2^(e-22) * I with whole I,
// |I| <= 2^22, and I = sum over i < 8 of d_i * 8^i with digits d_i from -4 to 3, whose halves
// are E2M1 values.  The block's 2^e, as far as 2^-17 of the row's largest, is the
// block's E4M3 scale.  A row of x becomes eight columns of the product, one a
// digit, whose sums the epilogue adds up by their powers of 8, and one to sixteen rows
// cost the same, 8 to 128 columns.  The one rounding that binary32 products do not
// have: a value is taken to 2^-22 of the largest of its 16, or 2^-39 of its slice's.  Beside
// the product of that largest value it is as small as their roundings; an output whose
// weight there is zero has it beside its other products.  Sixteen digits would take
// 256 columns for sixteen rows, and the tensor memory holds no two such accumulators.
//
// An infinity or NaN has no digits: it counts as 0 there, and the epilogue adds its
// products, from the weight in memory, to the outputs of its row.
//
// A block of threads keeps the digits of one slice of K (up to 8 pieces of 256) and
// walks the tiles of 128 outputs of its group; the slices' sums are added in order
// by a second kernel.  One warp copies (or eight do) and one multiplies; the sixteen
// others make the digits, while the first weights are on their way, and then read the
// accumulators and write, each four of them a quarter of the rows.
//
// Floor: the weight's bytes, 9/16 of one a value.  Steady state, [1, 5120] x [245760,
// 5120]: 107 us, 6.6 TB/s, 0.985 of what a copy reaches.  [1, 5120] x [30720, 5120]:
// 17.8 us, 5.0 TB/s: 4 us until the first product, of which the copies hide most, and 2.5
// for the second kernel.  [16, 5120] x [10007, 5120]: 12.4 us; its 29 MB take 4.4, the
// digits' kernel, the product's 128 columns (0.4 us a piece of weight against 0.3 for 16)
// and the sums' way through memory the rest.  The elected lane matters: the same operations
// from `lane == 0` took 0.7 us a piece.
#include <cuda.h>

#include <atomic>
#include <mutex>

#include "linear.cuh"

namespace mbx {

constexpr int kTile = 128, kPiece = 256, kMaxPieces = 8, kPassRows = 16, kMaxStages = 15;
// Warps: the workers, the multiplying one, those that copy.  Weight rows at 16-byte
// boundaries are copied by TMA, rows at 8-byte ones (K / 2 an odd multiple of 8) by eight
// warps, 8 bytes a lane ([1, 5136] x [30720, 5136]: four warps 35.5 us, eight 30.8, the
// copies' instructions the bound; with 4 pieces under way in place of 2 31.1, for 16 rows
// 54 against 41).
constexpr int kWorkers = 512, kMmaWarp = kWorkers / 32, kCopyWarp = kMmaWarp + 1;
constexpr int copy_threads(bool tma) { return tma ? 32 : 256; }
constexpr int tc_threads(bool tma) { return kWorkers + 32 + copy_threads(tma); }
constexpr int kLag = 2;  // pieces that the copying warps leave under way before they pass one on
constexpr int kFirstStages = 3;  // copied before the block meets; a copy takes 0.1 us to issue
constexpr int kStageBytes = 16384, kStageScales = 2048;
constexpr int kMaxSmem = 227 * 1024;
// tensor memory: two accumulators, the pieces' digits' scales and then the stages' scales,
// 16 columns each
constexpr uint32_t kAccCols = 128, kDigitScaleCol = 256, kScaleCols = 16;

struct TcParams {
    LinearParams l;
    int slices, pieces_per_slice, groups, stages, tiles;
    bool x_f32, out_f32, x_vec;
    // the digits made beforehand (linear_digits_kernel), or null: images of a slice for
    // every 16 rows and slice, image_bytes apart, each followed by its SliceRows
    uint8_t* images;
    int image_bytes;
};
struct SliceRows {
    uint32_t most[kPassRows];  // bits of the largest magnitude of a row in the slice
    int odd[kPassRows];        // whether the row has an infinity or NaN there
};

// How K is cut into slices and the tiles shared out, by what a block takes, in tenths of
// a microsecond: 4 for a piece of weight, 2 for a tile's end, 2 for a piece's digits, and
// 24 for the second kernel with 1 for each slice.  The rows do not matter, so that a
// row's sums have one order.
struct TcPlan {
    int slices, pieces_per_slice, groups, tiles;
};
static TcPlan tc_plan(int64_t N, int K) {
    const int pieces = (K + kPiece - 1) / kPiece, sms = sm_count();
    const int64_t tiles = (N + kTile - 1) / kTile;
    TcPlan best = {};
    int64_t cost = INT64_MAX;
    for (int len = 1; len <= kMaxPieces && len <= pieces; ++len) {
        const int slices = (pieces + len - 1) / len;
        int64_t groups = sms / slices;
        if (groups < 1) continue;
        if (groups > tiles) groups = tiles;
        const int64_t c = (tiles + groups - 1) / groups * (4 * len + 2) + 2 * len + (slices > 1 ? 24 + slices : 0);
        if (c < cost) {
            cost = c;
            best = TcPlan{slices, len, (int)groups, (int)tiles};
        }
    }
    return best;
}

// The workspace: the slices' sums [slices][rows][N], then the digits' images.
// A block makes the digits of up to kOwnBlocks blocks of 16 itself ([1, 5120] x [30720,
// 5120]: 18.5 us, with a kernel before it 21); more are made beforehand, once for all
// that use them ([8, 1024] x [2048, 1024]: 6.3 us against 9.1).
constexpr int kQuarters = 2, kOwnBlocks = kQuarters * kWorkers / 4;
static bool digits_before(const TcPlan& p, int rows) {
    return (rows < kPassRows ? rows : kPassRows) * p.pieces_per_slice * 16 > kOwnBlocks;
}
static int64_t sums_bytes(const TcPlan& p, int rows, int64_t N) {
    return p.slices > 1 ? ((int64_t)p.slices * rows * N * 4 + 127) / 128 * 128 : 0;
}
static int image_bytes(const TcPlan& p, int rows) {
    const int cols = rows >= kPassRows ? 8 * kPassRows : (rows * 8 + 15) / 16 * 16;
    return p.pieces_per_slice * (cols * 128 + 2048) + (int)sizeof(SliceRows);
}
int64_t linear_nvfp4_workspace_bytes(int rows, int64_t N, int K) {
    const TcPlan p = tc_plan(N, K);
    const int64_t passes = (rows + kPassRows - 1) / kPassRows;
    return sums_bytes(p, rows, N) + (digits_before(p, rows) ? passes * p.slices * image_bytes(p, rows) : 0);
}

// ---------------------------------------------------------------- barriers, copies, tensor memory

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t bar, int n) { asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n)); }
__device__ __forceinline__ void bar_arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); }
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok;
}
// Waits for the phase until `ns` have passed and `rounds` of 64 tries (a block that was off
// the GPU for that time has the tries left); false when it did not come, or when *failed
// was set meanwhile.
__device__ __forceinline__ bool bar_wait_while(uint32_t bar, uint32_t parity, unsigned long long ns, int rounds, const volatile int* failed) {
    unsigned long long start = 0, now = 0;
    for (int i = 0; now - start < ns || i < rounds; ++i) {
        for (int k = 0; k < 64; ++k)
            if (bar_try(bar, parity)) return true;
        if (failed && *failed) return false;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (i == 0) start = now;
    }
    return false;
}
// A wait of the block's work, for a second and a million tries: *failed is set when it did
// not come, and ends the others.  Nothing is known to make one fail; the outputs of the
// tiles that it leaves out are NaN.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* failed) {
    if (bar_wait_while(bar, parity, 1000000000ull, 1 << 14, failed)) return true;
    *failed = 1;
    return false;
}
// A wait for what the block has under way when it ends, whatever has failed: a sixteenth of that.
__device__ __forceinline__ void bar_land(uint32_t bar, uint32_t parity) { bar_wait_while(bar, parity, 62500000ull, 1 << 10, nullptr); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// K-major operand in 128-byte rows, 128-byte swizzle: 8 rows every 1024 bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// 32 rows of 16 bytes, no swizzle: 8 rows every 128 bytes.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(128 >> 4) << 32 | 1ull << 46;
}
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// One lane of a whole warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one;
}
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, bool add) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// ---------------------------------------------------------------- activations and their digits

// Four activations, a quarter of a block of 16: x[row][k ...].
__device__ __forceinline__ void load_quarter(float (&v)[4], const TcParams& p, int row, int k) {
    const int64_t at = (int64_t)row * p.l.x_stride + k;
    if (p.x_f32) {
        const float* x = static_cast<const float*>(p.l.x) + at;
        if (p.x_vec) {
            const uint4 q = ld_stream_rw(x);
            v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = load_elem(x + i);
        }
    } else {
        const uint16_t* x = static_cast<const uint16_t*>(p.l.x) + at;
        if (p.x_vec) {
            uint32_t a, b;
            asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "l"(x));
            v[0] = lo_f(a), v[1] = hi_f(a), v[2] = lo_f(b), v[3] = hi_f(b);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = load_elem(x + i);
        }
    }
    if (p.l.silu) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = silu(v[i]);
    }
}

// The largest magnitude of the finite values, as bits; *odd set where one is not finite.
__device__ __forceinline__ uint32_t quarter_max(const float (&v)[4], int* odd) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
        if (b >= 0x7f800000u) *odd = 1;
        else m = max(m, b);
    }
    return m;
}
// Of the four lanes that have a block.
__device__ __forceinline__ uint32_t of_four(uint32_t m) {
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
// e with |v| < 2^e and, unless v is 0, |v| >= 2^(e-1); -149 of 0.
__device__ __forceinline__ int above(uint32_t bits) {
    return bits < 0x800000u ? -117 - __clz((int)bits) : (int)(bits >> 23) - 126;
}
// 2^n, n from -126 to 127
__device__ __forceinline__ float power_of_2(int n) { return __uint_as_float((uint32_t)(127 + n) << 23); }

// The digits of the whole number nearest to v, |v| <= 2^22, digit i in nibble i as an
// E2M1 code of d_i / 2.
__device__ __forceinline__ uint32_t digits(float v) {
    // digits + 4 are the octal places of I + 044444444, spread from 3 to 4 bits each
    uint32_t x = (uint32_t)(__float2int_rn(v) + 9586980);
    x = (x & 0x00000fffu) | (x & 0x00fff000u) << 4;
    x = (x & 0x003f003fu) | (x & 0x0fc00fc0u) << 2;
    x = (x & 0x07070707u) | (x & 0x38383838u) << 1;
    // 4..7: the code is the place - 4; 0..3: 8 + (4 - the place)
    const uint32_t m = (x >> 2) & 0x11111111u, up = (m << 4) - m;
    return (x & 0x33333333u & up) | ((0xccccccccu - x) & ~up);
}
// The digits of a quarter of a block whose largest magnitude has the bits `block`, of a
// row whose largest in this slice of K has the bits `most`, into the row's eight columns:
// `col` is digit 0's column in the piece (columns 128 bytes apart, 16-byte units
// swizzled), `scale` its scale (columns 16 bytes apart); b is the block's place in the
// slice, q the quarter.
__device__ __forceinline__ void put_digits(const float (&v)[4], uint32_t block, uint32_t most, int b, int q, uint8_t* col, uint8_t* scale) {
    const int top = above(most), e = max(above(block), top - 17);
    // 2^(22-e) in two exact steps: for blocks below 2^-104 it is no binary32 number
    const int up0 = min(22 - e, 126);
    const float to_int = power_of_2(up0), rest = power_of_2(22 - e - up0);
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = digits((__float_as_uint(v[i]) & 0x7f800000u) == 0x7f800000u ? 0.0f : v[i] * to_int * rest);
    // two values a byte, the first in the low half: bytes of digits 0, 2, 4, 6 and of 1, 3, 5, 7
    uint32_t even[2], odd[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        even[h] = (d[2 * h] & 0x0f0f0f0fu) | (d[2 * h + 1] & 0x0f0f0f0fu) << 4;
        odd[h] = (d[2 * h] >> 4 & 0x0f0f0f0fu) | (d[2 * h + 1] & 0xf0f0f0f0u);
    }
    const int up = 8 + e - top;  // -9 .. 8: the scale 2^up as E4M3
    const uint8_t sc = (uint8_t)(up >= -6 ? (up + 7) << 3 : 1 << (up + 9));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t two = __byte_perm(i & 1 ? odd[0] : even[0], i & 1 ? odd[1] : even[1], i / 2 | (i / 2 + 4) << 4);
        *reinterpret_cast<uint16_t*>(col + i * 128 + ((b % 16 / 2) ^ i) * 16 + b % 2 * 8 + q * 2) = (uint16_t)two;
        if (i % 4 == q) scale[i * 16] = sc;
    }
}
// Where a row's columns of a slice's digits begin, and its scales: [pieces][cols][128
// bytes], then [steps of 64][512 bytes] in the order of the weight's scale tiles.
__device__ __forceinline__ uint8_t* digit_at(uint8_t* image, int cols, int r, int b) { return image + (b / 16 * cols + r * 8) * 128; }
__device__ __forceinline__ uint8_t* digit_scale_at(uint8_t* image, int cols, int pieces, int r, int b) {
    return image + pieces * cols * 128 + b / 4 * 512 + r % 4 * 128 + r / 4 * 4 + b % 4;
}

// sum over the slice's k with a non-finite activation of a(x[row][k]) * w[n][k]
__device__ __noinline__ float odd_products(const TcParams& p, int row, int64_t n, int blk0, int blk1) {
    float sum = 0.0f;
    for (int blk = blk0; blk < blk1; ++blk) {
        float v[16];
        int odd = 0;
        for (int q = 0; q < 4; ++q) {
            load_quarter(reinterpret_cast<float(&)[4]>(v[4 * q]), p, row, 16 * blk + 4 * q);
            quarter_max(reinterpret_cast<float(&)[4]>(v[4 * q]), &odd);
        }
        if (!odd) continue;
        const uint8_t b = p.l.sf[(n / 128 * p.l.sf_col_tiles + blk / 4) * 512 + n % 32 * 16 + n % 128 / 32 * 4 + blk % 4];
        const float s = e4m3_value(b);
        for (int i = 0; i < 16; ++i) {
            if ((__float_as_uint(v[i]) & 0x7f800000u) != 0x7f800000u) continue;
            const uint32_t c = p.l.w4[n * p.l.w_stride + blk * 8 + i / 2] >> (i % 2 * 4) & 15u;
            sum += v[i] * (e2m1_value(c) * s);
        }
    }
    return sum;
}

__device__ __forceinline__ float bias_of(const TcParams& p, int64_t n) {
    return !p.l.bias || n >= p.l.N ? 0.0f
           : p.l.bias_f32 ? load_elem(static_cast<const float*>(p.l.bias) + n) : load_elem(static_cast<const uint16_t*>(p.l.bias) + n);
}
__device__ __forceinline__ void store_output(const TcParams& p, int row, int64_t n, float sum, float gs, float bias) {
    float v = sum / gs;
    if (p.l.bias) v += bias;
    const int64_t at = (int64_t)row * p.l.out_stride + n;
    if (p.out_f32) store_elem(static_cast<float*>(p.l.out) + at, v);
    else store_elem(static_cast<uint16_t*>(p.l.out) + at, v);
}

// ---------------------------------------------------------------- the product

struct TcShared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained, digits;
    uint32_t tmem;
    int failed, fetched;  // fetched: pieces whose copies were begun, when the roles meet
    SliceRows rows;
};

template <bool TMA>
__global__ void __launch_bounds__(tc_threads(TMA), 1) linear_tc_kernel(const __grid_constant__ CUtensorMap map, const TcParams p) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);
    __shared__ TcShared sh;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row0 = blockIdx.y * kPassRows, rows = min(p.l.rows - row0, kPassRows);
    const int cols = (rows * 8 + 15) / 16 * 16;  // of the product
    const int slice = blockIdx.x % p.slices, group = blockIdx.x / p.slices;
    const int blocks = p.l.K / 16, piece0 = slice * p.pieces_per_slice;
    const int piece1 = min(piece0 + p.pieces_per_slice, (p.l.K + kPiece - 1) / kPiece);
    const int blk0 = piece0 * 16, blk1 = min(piece1 * 16, blocks), steps = (blk1 - blk0 + 3) / 4;
    const int my_tiles = (p.tiles - group + p.groups - 1) / p.groups;
    uint8_t* ring = smem;
    uint8_t* dig = ring + p.stages * kStageBytes;  // the slice's digits and their scales (digit_at)
    uint8_t* dig_scales = dig + p.pieces_per_slice * cols * 128;
    uint8_t* scales = dig_scales + p.pieces_per_slice * 2048;  // the stages'

    volatile int* failed = &sh.failed;
    const int total = my_tiles * (piece1 - piece0);  // pieces of weight that this block takes
    const int copier = (int)threadIdx.x - kCopyWarp * 32;  // of the copying threads
    auto fetch = [&](int u) {                              // the u-th, into stage u % stages
        const int t = u / (piece1 - piece0), piece = piece0 + u - t * (piece1 - piece0), tile = group + t * p.groups;
        const int s = u % p.stages;
        const uint32_t bar = smem_addr(&sh.full[s]), bytes = (uint32_t)min(4, p.l.sf_col_tiles - piece * 4) * 512;
        if (copier == 0) {
            bar_expect(bar, (TMA ? kStageBytes : 0) + bytes);
            if constexpr (TMA)
                asm volatile(
                    "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                        smem_addr(ring + s * kStageBytes)),
                    "l"(&map), "r"(piece * 128), "r"(tile * kTile), "r"(bar)
                    : "memory");
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem_addr(scales + s * kStageScales)),
                         "l"(p.l.sf + ((int64_t)tile * p.l.sf_col_tiles + piece * 4) * 512), "r"(bytes), "r"(bar)
                         : "memory");
        }
        if constexpr (!TMA) {
            // sixteen lanes a row, a share of the rows a warp; in the order of the 128-byte
            // swizzle, 0 past the weight
            constexpr int kRows = kTile * 32 / copy_threads(false);  // of a warp
            const int half = copier % 32 / 16, c = copier % 16, row = copier / 32 * kRows + half;
            const int64_t n = (int64_t)tile * kTile + row;
            const uint8_t* from = p.l.w4 + n * p.l.w_stride + piece * 128 + c * 8;
            const bool in = piece * 128 + c * 8 < p.l.K / 2;
            const uint32_t to = smem_addr(ring + s * kStageBytes) + row * 128 + c % 2 * 8;
#pragma unroll
            for (int i = 0; i < kRows / 2; ++i) {
                const int size = in && n + 2 * i < p.l.N ? 8 : 0;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to + i * 256 + ((c / 2 ^ (row + 2 * i) % 8) * 16)),
                             "l"(size ? from + i * 2 * p.l.w_stride : p.l.w4), "r"(size)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    auto prefetch = [&](int u) {  // the same into L2, as a hint
        const int t = u / (piece1 - piece0), piece = piece0 + u - t * (piece1 - piece0), tile = group + t * p.groups;
        if constexpr (TMA) {
            asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(&map), "r"(piece * 128), "r"(tile * kTile)
                         : "memory");
        } else {
            const int64_t n = (int64_t)tile * kTile + copier;
            if (copier < kTile && n < p.l.N) prefetch_l2(p.l.w4 + n * p.l.w_stride + piece * 128);
        }
        if (copier == 0) prefetch_l2_bulk(p.l.sf + ((int64_t)tile * p.l.sf_col_tiles + piece * 4) * 512, (uint32_t)min(4, p.l.sf_col_tiles - piece * 4) * 512);
    };
    // the worker's quarters of blocks of activations, 0 past K: the c-th is quarter
    // id % 4 of block id / 4, id = c * kWorkers + thread
    const int per_row = steps * 4, items = rows * per_row;
    float v[kQuarters][4];
#pragma unroll
    for (int c = 0; c < kQuarters; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = 0.0f;
    const uint8_t* image = p.images ? p.images + ((int64_t)blockIdx.y * p.slices + slice) * p.image_bytes : nullptr;

    if (warp >= kCopyWarp) {
        if (copier == 0) {
            for (int i = 0; i < p.stages; ++i) {
                bar_init(smem_addr(&sh.full[i]), TMA ? 1 : 1 + copy_threads(false));
                bar_init(smem_addr(&sh.empty[i]), 1);
            }
            for (int i = 0; i < 2; ++i) {
                bar_init(smem_addr(&sh.acc_full[i]), 1);
                bar_init(smem_addr(&sh.acc_empty[i]), kWorkers / 32);
            }
            bar_init(smem_addr(&sh.drained), 1);
            bar_init(smem_addr(&sh.digits), 1);
            sh.failed = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        if (!TMA || copier == 0) {
            // Nothing is read before the wait.  Where another kernel makes the digits the first
            // weights are brought into L2 meanwhile, a hint that holds no values ([16, 5120] x
            // [10007, 5120]: 13.9 us without, 13.6 so), once for all rows.
            if (p.images && blockIdx.y == 0)
                for (int u = 0; u < kFirstStages && u < p.stages && u < total; ++u) prefetch(u);
            grid_dep_wait();
            for (int u = 0; u < kFirstStages && u < p.stages && u < total; ++u) fetch(u);
            if (p.images && copier == 0) {
                const uint32_t bytes = p.pieces_per_slice * (cols * 128 + 2048);
                bar_expect(smem_addr(&sh.digits), bytes);
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 smem_addr(dig)),
                             "l"(image), "r"(bytes), "r"(smem_addr(&sh.digits))
                             : "memory");
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        if (threadIdx.x < kPassRows && !p.images) sh.rows.most[threadIdx.x] = sh.rows.odd[threadIdx.x] = 0;
        grid_dep_wait();
        if (p.images) {
            if (threadIdx.x < sizeof(SliceRows) / 4)
                reinterpret_cast<uint32_t*>(&sh.rows)[threadIdx.x] = reinterpret_cast<const volatile uint32_t*>(image + p.image_bytes - sizeof(SliceRows))[threadIdx.x];
        } else {
#pragma unroll
            for (int c = 0; c < kQuarters; ++c) {
                const int at = (c * kWorkers + (int)threadIdx.x) / 4, r = at / per_row, blk = blk0 + at - r * per_row;
                if (at < items && blk < blk1) load_quarter(v[c], p, row0 + r, 16 * blk + threadIdx.x % 4 * 4);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    grid_dep_launch();

    if (warp >= kCopyWarp) {
        if (!TMA || copier == 0) {
            int u = min(kFirstStages, min(p.stages, total)), passed = 0;
            auto pass = [&](int until) {  // this thread's copies of the pieces before `until` have landed
                fence_async();
                for (; passed < until; ++passed) bar_arrive(smem_addr(&sh.full[passed % p.stages]));
            };
            for (; u < total; ++u) {
                if (u >= p.stages && !bar_wait(smem_addr(&sh.empty[u % p.stages]), (u / p.stages - 1) & 1, failed)) break;
                fetch(u);
                if constexpr (!TMA) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
                    pass(u + 1 - kLag);
                }
            }
            if constexpr (!TMA) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                pass(u);
            }
            if (copier == 0) sh.fetched = u;
        }
        __syncwarp();
    } else if (warp < kMmaWarp && !p.images) {
        uint32_t block[kQuarters];
#pragma unroll
        for (int c = 0; c < kQuarters; ++c) {
            if (c * kWorkers / 4 >= items) break;
            const int at = (c * kWorkers + (int)threadIdx.x) / 4, r = min(at, items - 1) / per_row;
            int odd = 0;
            block[c] = of_four(quarter_max(v[c], &odd));
            if (per_row % 8 == 0) {  // a warp's eight blocks are of one row
                const uint32_t m = __reduce_max_sync(0xffffffffu, block[c]);
                if (lane == 0) atomicMax(&sh.rows.most[r], m);
            } else if (lane % 4 == 0) {
                atomicMax(&sh.rows.most[r], block[c]);
            }
            if (odd) sh.rows.odd[r] = 1;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kWorkers) : "memory");
#pragma unroll
        for (int c = 0; c < kQuarters; ++c) {
            const int at = (c * kWorkers + (int)threadIdx.x) / 4;
            if (at >= items) break;
            const int r = at / per_row, b = at - r * per_row;
            put_digits(v[c], block[c], sh.rows.most[r], b, lane % 4, digit_at(dig, cols, r, b),
                       digit_scale_at(dig, cols, p.pieces_per_slice, r, b));
        }
        fence_async();
        asm volatile("bar.arrive 2, %0;" ::"n"(kWorkers + 32) : "memory");
    }

    if (warp == kMmaWarp) {
        bool ok = true;
        if (p.images) ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.digits), 0, failed));
        else asm volatile("bar.sync 2, %0;" ::"n"(kWorkers + 32) : "memory");
        const uint32_t idesc = 1u << 7 | 1u << 10 | (uint32_t)(cols / 8) << 17 | (uint32_t)(kTile / 16) << 24;
        const bool leader = elect_one();
        const bool ragged = blocks % 4 != 0 && blk1 == blocks;  // the last step's blocks past K: their scales are anything
        const int pieces = piece1 - piece0;
        if (leader)  // the digits' scales
            for (int k = 0; k < steps; ++k) scales_to_tmem(tmem + kDigitScaleCol + 4 * k, scale_desc(smem_addr(dig_scales)) + 32 * k);
        int stage = 0, phase = 0;
        for (int t = 0; t < my_tiles && ok; ++t) {
            const int a = t & 1;
            if (t >= 2) ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.acc_empty[a]), (t / 2 - 1) & 1, failed));
            tc_fence_after();
            for (int piece = 0; piece < pieces && ok; ++piece) {
                const int n = min(4, p.l.sf_col_tiles - (piece0 + piece) * 4);
                ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.full[stage]), phase, failed));
                if (!ok) break;
                if (ragged && piece == pieces - 1) {
                    const uint32_t keep = (1u << blocks % 4 * 8) - 1;
                    uint32_t* w = reinterpret_cast<uint32_t*>(scales + stage * kStageScales + (n - 1) * 512);
                    for (int i = lane; i < 128; i += 32) w[i] &= keep;
                    fence_async();
                    __syncwarp();
                }
                if (leader) {
                    const uint32_t sb = tmem + kDigitScaleCol + kScaleCols * piece;
                    const uint32_t sa = tmem + kDigitScaleCol + kScaleCols * (p.pieces_per_slice + stage);
                    const uint64_t wa = operand_desc(smem_addr(ring + stage * kStageBytes));
                    const uint64_t da = operand_desc(smem_addr(dig + piece * cols * 128));
                    const uint64_t sd = scale_desc(smem_addr(scales + stage * kStageScales));
                    const uint32_t acc = tmem + a * kAccCols;
                    if (n == 4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) scales_to_tmem(sa + 4 * k, sd + 32 * k);
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_fp4(acc, wa + 2 * k, da + 2 * k, idesc, sa + 4 * k, sb + 4 * k, piece > 0 || k > 0);
                    } else {
                        for (int k = 0; k < n; ++k) scales_to_tmem(sa + 4 * k, sd + 32 * k);
                        for (int k = 0; k < n; ++k) mma_fp4(acc, wa + 2 * k, da + 2 * k, idesc, sa + 4 * k, sb + 4 * k, piece > 0 || k > 0);
                    }
                    mma_commit(smem_addr(&sh.empty[stage]));
                    if (piece == pieces - 1) mma_commit(smem_addr(&sh.acc_full[a]));
                }
                __syncwarp();
                if (++stage == p.stages) stage = 0, phase ^= 1;
            }
        }
        // nothing of the block may be under way when it gives the tensor memory back
        if (leader) {
            mma_commit(smem_addr(&sh.drained));
            bar_land(smem_addr(&sh.drained), 0);
        }
        __syncwarp();
    } else if (warp < kMmaWarp) {
        const float gs = p.slices == 1 ? *p.l.gs : 1.0f;
        for (int t = 0; t < my_tiles; ++t) {
            const int a = t & 1;
            const int64_t n = (int64_t)(group + t * p.groups) * kTile + threadIdx.x % 128;
            const float bias = p.slices == 1 ? bias_of(p, n) : 0.0f;
            const bool ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.acc_full[a]), (t / 2) & 1, failed));
            tc_fence_after();
            const uint32_t acc = tmem + a * kAccCols + ((uint32_t)(warp % 4 * 32) << 16);
            for (int r = warp / 4 * 2; r < rows; r += 8) {
                uint32_t d[16];
                __syncwarp();
                asm volatile(
                    "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                    : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]), "=r"(d[7]), "=r"(d[8]),
                      "=r"(d[9]), "=r"(d[10]), "=r"(d[11]), "=r"(d[12]), "=r"(d[13]), "=r"(d[14]), "=r"(d[15])
                    : "r"(acc + r * 8));
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (r + h >= rows || n >= p.l.N) continue;
                    float s = __uint_as_float(d[8 * h + 7]);
#pragma unroll
                    for (int i = 6; i >= 0; --i) s = __fmaf_rn(s, 8.0f, __uint_as_float(d[8 * h + i]));
                    // 2^(top-29), the first step exact
                    const int top = above(sh.rows.most[r + h]), down = max(top - 29, -100);
                    s = s * power_of_2(down) * power_of_2(top - 29 - down);
                    const int row = row0 + r + h;
                    if (sh.rows.odd[r + h]) s += odd_products(p, row, n, blk0, blk1);
                    if (!ok) s = __uint_as_float(0x7fffffffu);
                    if (p.slices > 1) p.l.ws[((int64_t)slice * p.l.rows + row) * p.l.N + n] = s;
                    else store_output(p, row, n, s, gs, bias);
                }
            }
            __syncwarp();
            tc_fence_before();
            if (lane == 0) bar_arrive(smem_addr(&sh.acc_empty[a]));
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    // A block that gave up, in whichever role, ends when its bulk copies have landed in its
    // shared memory; otherwise all of them have been waited for.  The copying threads' own
    // copies were, before they met the others.
    if (*failed && copier == 0) {
        if (p.images) bar_land(smem_addr(&sh.digits), 0);
        for (int i = max(sh.fetched - p.stages, 0); i < sh.fetched; ++i) bar_land(smem_addr(&sh.full[i % p.stages]), (i / p.stages) & 1);
    }
}

// The digits of one row's part of a slice, for all blocks of the product that use it.
// Sixteen rows' digits take a block of the product 6 us, which its first copies do
// not cover; made once here they take 2.
__global__ void __launch_bounds__(64 * kMaxPieces) linear_digits_kernel(const TcParams p) {
    __shared__ uint32_t most_of[2 * kMaxPieces];
    __shared__ int odd_of[2 * kMaxPieces];
    const int slice = blockIdx.x, row = blockIdx.y, pass = row / kPassRows, r = row % kPassRows;
    const int cols = (min(p.l.rows - pass * kPassRows, kPassRows) * 8 + 15) / 16 * 16;
    const int blocks = p.l.K / 16, blk0 = slice * p.pieces_per_slice * 16, blk1 = min(blk0 + p.pieces_per_slice * 16, blocks);
    const int b = threadIdx.x / 4, q = threadIdx.x % 4, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    grid_dep_wait();
    grid_dep_launch();
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (blk0 + b < blk1) load_quarter(v, p, row, 16 * (blk0 + b) + 4 * q);
    int odd = 0;
    const uint32_t block = of_four(quarter_max(v, &odd)), m = __reduce_max_sync(0xffffffffu, block);
    odd = __any_sync(0xffffffffu, odd);
    if (lane == 0) {
        most_of[warp] = m;
        odd_of[warp] = odd;
    }
    __syncthreads();
    uint32_t most = 0;
    odd = 0;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) {
        most = max(most, most_of[i]);
        odd |= odd_of[i];
    }
    uint8_t* image = p.images + ((int64_t)pass * p.slices + slice) * p.image_bytes;
    if (b < (blk1 - blk0 + 3) / 4 * 4)
        put_digits(v, block, most, b, q, digit_at(image, cols, r, b), digit_scale_at(image, cols, p.pieces_per_slice, r, b));
    if (threadIdx.x == 0) {
        SliceRows* s = reinterpret_cast<SliceRows*>(image + p.image_bytes - sizeof(SliceRows));
        s->most[r] = most;
        s->odd[r] = odd;
    }
}

// out = the slices' sums, in order, over gs, and the bias
__global__ void __launch_bounds__(256) linear_join_kernel(const TcParams p) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    if (n >= p.l.N) return;
    const float gs = *p.l.gs, bias = bias_of(p, n);
    const int row = blockIdx.y;
    const float* w = p.l.ws + (int64_t)row * p.l.N + n;
    float s = 0.0f;
    for (int i0 = 0; i0 < p.slices; i0 += 8) {  // eight loads under way
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i0 + i < p.slices ? w[(int64_t)(i0 + i) * p.l.rows * p.l.N] : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[i];
    }
    store_output(p, row, n, s, gs, bias);
}

// ---------------------------------------------------------------- launch

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(f);
        cudaGetLastError();
    });
    return fn;
}

// The tensor map wants the weight's rows at multiples of 16 bytes, the copying warps at
// multiples of 8, the copies of scales 16.
static bool rows_at(const LinearParams& p, int bytes) {
    return reinterpret_cast<uintptr_t>(p.w4) % bytes == 0 && (p.N == 1 || p.w_stride % bytes == 0);
}
bool linear_tc_takes(const LinearParams& p) {
    return tc_plan(p.N, p.K).slices > 0 && rows_at(p, 8) && reinterpret_cast<uintptr_t>(p.sf) % 16 == 0;
}

cudaError_t launch_linear_tc(const LinearParams& l, bool x_f32, bool out_f32, cudaStream_t s) {
    static std::atomic<bool> allowed[64] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int kFixed = (int)sizeof(TcShared) + 256;  // the static part, rounded up
    constexpr int kMost = kMaxSmem - kFixed;
    if (!allowed[dev].load(std::memory_order_acquire)) {
        if (cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost)) return e;
        if (cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost)) return e;
        allowed[dev].store(true, std::memory_order_release);
    }
    const TcPlan plan = tc_plan(l.N, l.K);
    TcParams p = {};
    p.l = l;
    p.slices = plan.slices;
    p.pieces_per_slice = plan.pieces_per_slice;
    p.groups = plan.groups;
    p.tiles = plan.tiles;
    p.x_f32 = x_f32;
    p.out_f32 = out_f32;
    p.x_vec = reinterpret_cast<uintptr_t>(l.x) % 16 == 0 && (l.rows == 1 || l.x_stride * (x_f32 ? 4 : 2) % 16 == 0);
    const int rows = l.rows < kPassRows ? l.rows : kPassRows, cols = (rows * 8 + 15) / 16 * 16;
    const int dig = plan.pieces_per_slice * (cols * 128 + 4 * 512);
    p.stages = (kMost - 1024 - dig) / (kStageBytes + kStageScales);
    if (p.stages > kMaxStages + 1 - plan.pieces_per_slice) p.stages = kMaxStages + 1 - plan.pieces_per_slice;  // 512 columns
    // A ring that is filled again (one of `work` stages is not) has more stages than are copied
    // before the copying warps pass the first piece on, and than they leave under way.
    constexpr int kBySmem = (kMost - 1024 - kMaxPieces * (kPassRows * 8 * 128 + 4 * 512)) / (kStageBytes + kStageScales);
    static_assert(kBySmem > kFirstStages && kMaxStages + 1 - kMaxPieces > kFirstStages && kFirstStages >= kLag);
    const int work = (plan.tiles + plan.groups - 1) / plan.groups * plan.pieces_per_slice;
    if (p.stages > work) p.stages = work;
    const size_t smem = 1024 + dig + (size_t)p.stages * (kStageBytes + kStageScales);

    const bool tma = rows_at(l, 16);
    CUtensorMap map = {};
    if (tma) {
        EncodeTiled encode = encode_tiled();
        if (!encode) return cudaErrorNotSupported;
        const cuuint64_t dims[2] = {(cuuint64_t)l.K / 2, (cuuint64_t)l.N};
        const cuuint64_t strides[1] = {(cuuint64_t)(l.N > 1 ? l.w_stride : (l.K / 2 + 15) / 16 * 16)};
        const cuuint32_t box[2] = {128, kTile}, one[2] = {1, 1};
        if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(l.w4), dims, strides, box, one,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const unsigned passes = (unsigned)((l.rows + kPassRows - 1) / kPassRows);
    if (digits_before(plan, l.rows)) {
        p.images = reinterpret_cast<uint8_t*>(l.ws) + sums_bytes(plan, l.rows, l.N);
        p.image_bytes = image_bytes(plan, l.rows);
        const unsigned threads = (unsigned)plan.pieces_per_slice * 64;
        if (cudaError_t e = launch_pdl_2d(linear_digits_kernel, dim3((unsigned)plan.slices, (unsigned)l.rows), threads, 0, s, p)) return e;
    }
    const cudaError_t e = launch_pdl_2d(tma ? linear_tc_kernel<true> : linear_tc_kernel<false>, dim3((unsigned)(p.slices * p.groups), passes),
                                  tc_threads(tma), smem, s, map, p);
    if (e != cudaSuccess || p.slices == 1) return e;
    return launch_pdl_2d(linear_join_kernel, dim3((unsigned)((l.N + 255) / 256), (unsigned)l.rows), 256, 0, s, p);
}

}  // namespace mbx
