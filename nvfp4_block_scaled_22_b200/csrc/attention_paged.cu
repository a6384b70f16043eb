// Decode attention of a batch of sequences over a paged NVFP4 KV cache: one
// query token a sequence, grouped-query heads,
//   s_t = scale q . k_t,  o = sum_t exp(s_t) v_t / sum_t exp(s_t),
// t over the sequence's cached tokens; token t lives in pool row
// block_table[b][t / page_size] * page_size + t % page_size.
//
// Each cache byte is read once (0.5625 bytes a value) and restored in
// registers.  Bound: the read, and close behind it the instructions that
// restore and multiply -- a 16-token tile of 8 heads x 128 dims takes a warp
// about 280, two of a lane's a value -- so that the long calls end between
// the two: 64 sequences of 8192 tokens, 8 KV heads x 128, 64 query heads 120
// us (5.1 TB/s, 0.77 of a copy); one of 131072 tokens 40.6 us (3.7 TB/s; each
// further 131072 take 26 us, 5.8 TB/s, the rest is start, ending and join);
// 96 of 256 to 8192 tokens 60 us (4.2 TB/s).  One of 1000 tokens takes 9.8
// us, of one token 6: two launches and four dependent reads (length, page,
// tile, parts).
//
// Units and warps.  A unit is a KV head with up to 8 of its query heads (the 8
// columns of an MMA); larger groups are several units.  A CTA has 8 computing
// warps over neighbouring units (so that it reads whole pieces of a cache
// row), and the warps of a unit share its tokens, 16 each; every warp keeps
// its own online softmax over its tiles.  Two CTAs an SM (heads of 256 values:
// one): one CTA of 16 computing warps was 1.5 % faster on equal long
// sequences and 5 to 30 % slower elsewhere, as a sequence's ending then
// idles the SM.
//
// Copies.  Two (or four) further warps fill a ring of stages, in turn; full / empty
// mbarriers, every wait bounded.  Where 16 tokens share a page and a row's
// scales are whole 16-byte groups, a stage's parts are boxes of a 3-D tiled
// TMA load (bytes of a head x 16 rows x heads), swizzled by it; else each
// token's row is looked up and copied in 16-byte pieces by cp.async to the
// same places (64 x 8192 in pages of 20 tokens: 140 us; with addresses worked
// out piece by piece 27 % more, the copying warps' instructions being the
// bound).  Computing warps that refilled the ring themselves took 150 us where
// a producer warp took 130 (registers).
//
// Schedule.  The sequences' tiles (16 tokens times the warps of a unit; an
// empty sequence counts one), each sequence's behind some that stand for the
// cost of taking up a sequence, are one list, cut into equal ranges, one a
// CTA, on the device from seq_lens: the CTAs have equal work whatever the
// lengths, and the host needs no length.  A sequence that ends inside of its
// CTA's range is written at once; one that is cut leaves a partial (m, l, O)
// per CTA, which k_paged_combine joins in the order of the ranges: the result
// does not depend on which CTA ends first.
//
// A 16-token tile of a unit:
//   S[16 tokens x 8 heads] = K q^T, mma.sync m16n8k16, FP16 operands, FP32
//     accumulators.  e2m1 * e4m3 has at most 6 significant bits within 2^-10
//     .. 2688: exact in FP16.  The query (BF16) is scaled by a power of two
//     per head to a largest value in [2^14, 2^15) and is exact in FP16 down
//     to 2^-29 of it.
//   p = 2^(S c - m'), c = scale log2(e) / g_K and the query's power of two
//     undone.  m' is 6 below a running reference that is moved (and what was
//     summed rescaled) only when a score passes it by 8: p stays within
//     2^14, and the largest p of a head is at least 2^6 (scores past 2^23: 2^0),
//     so that rounding p to FP16 for the product with V costs 2^-11 of each
//     weight, or 2^-31 of the largest for tiny ones.  The sum l takes the
//     unrounded p in FP32.
//   O^T[dim x 8 heads] += V^T P^T, the same MMA: P goes from accumulator to
//     operand layout by movmatrix; the codes of two tokens are interleaved
//     by nibbles so that one conversion gives the two tokens of one dim.
//   The rows of an MMA are the tile's tokens in an order (token_of) in which,
//   under the copies' swizzle, neither the row-wise reads of K nor the
//   column-wise reads of V meet a shared-memory bank twice.
//   The query's fragments lie in shared memory, where the warp's O goes at
//   the end: registers (96 at two CTAs) are what limits the warps of an SM.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kLowest = -3.402823466e38f;
constexpr float kOffset = 6.0f;      // m' is this much below the reference
constexpr float kSlack = 14.0f;      // a score may pass m' by this before m' moves

constexpr int kWarps = 8;            // warps that compute
// Warps that bring the tiles in, stages in turn.  Copies by cp.async take four
// with heads of 64 values (4 x 3 .. 97886 tokens, 5 heads: 43.5 -> 39.6 us);
// with 128 the 80 registers that are left spill (64 x 8192 in pages of 20: 5 %
// slower with three), with 256 it is 3 % either way.
template <int kD, bool kTma>
struct Producers {
    static constexpr int kCount = !kTma && kD == 64 ? 4 : 2;
};
constexpr long long kDrainCycles = 2000000000ll;   // bound of the wait for copies under way (about a second)
constexpr int kTile = 16;            // tokens of a warp's tile
constexpr int kProducerBarrier = 8;  // named barrier of the producers (1 .. 4: the units')

template <int kD>
struct Shape {
    static constexpr int kCodes = kD / 2;                       // bytes of a token's codes
    static constexpr int kScales = kD / 16;
    static constexpr int kChunks = kD / 32;                     // 16-byte pieces of a token's codes
    static constexpr int kSteps = kD / 16;                      // MMA steps over the dims (and M-tiles of O^T)
    static constexpr int kCtasPerSm = kD == 256 ? 1 : 2;
};

// 16-byte piece `ch` of token t of a tile lies at this piece of the token's
// row: the swizzle of the copies (64-byte rows: by bits 1 .. 2 of t, 128-byte
// rows: by bits 0 .. 2, 32-byte rows: none).
template <int kD>
__device__ __forceinline__ int swizzled(int ch, int t) {
    if (kD == 64) return ch;
    if (kD == 128) return ch ^ ((t >> 1) & 3);
    return ch ^ (t & 7);
}

// Token of MMA row 2 c + j (rows 8 .. 15: + 8).  Under the swizzle above,
// the lanes that a shared-memory access serves at once -- two rows' K codes
// (j = 0, 1), or four tokens' V codes (c = 0 .. 3) -- meet different banks.
template <int kD>
__device__ __forceinline__ int token_of(int c, int j) {
    if (kD == 64) return 4 * j + (c ^ (3 * j));
    if (kD == 128) return ((c & 1) ^ j) + 2 * j + 4 * (c >> 1);
    return 2 * (c ^ (2 * j)) + j;
}

// 3-D tiled TMA load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *desc, uint64_t *bar, int32_t x,
                                            int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(desc)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Wait for a phase of `bar`, at most about `limit` cycles.  (A try may sleep
// for some microseconds, so that the limit is looked at before each.)
__device__ __forceinline__ bool bounded_wait(uint64_t *bar, uint32_t parity, long long limit) {
    const long long t0 = clock64();
    if (mbar_test_wait(bar, parity)) return true;
    while (clock64() - t0 <= limit)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}

// Arrives on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The four bytes of a word to f16x2 each (low nibble in the low half); the
// vector move lets the conversions take the bytes in place (twice the rate
// of shifting each byte down: 158 against 83 values a ns and SM).
__device__ __forceinline__ void f16x2_from_word(uint32_t w, uint32_t (&o)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}

__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t f16x2_from_f32(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
    return d;
}

// 1 / (l g), or 0 for no token, as a product of two factors: g is up to 2^118,
// so that neither l g nor its reciprocal need be a normal number.  `post` is a
// power of two (1 up to g = 2^60), the bits are those of one factor where it
// would do.
__device__ __forceinline__ float post_of(float g) { return g > 0x1p60f ? 0x1p-60f : 1.0f; }
__device__ __forceinline__ float share_of(float l, float g, float post) {
    return l == 0.0f ? 0.0f : __frcp_rn(__fmul_rn(l, g * post));
}

// log of a sum l of 2^(x - m), natural; lg2.approx is off by at most 2^-22
// (l is 0 or at least 1)
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -__int_as_float(0x7F800000) : (m + __log2f(l)) * kLn2;
}

// (a & m) | (b & ~m), m = 0x0F0F0F0F
__device__ __forceinline__ uint32_t nibbles(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(d) : "r"(0x0F0F0F0Fu), "r"(a), "r"(b));
    return d;
}

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(dst), "l"(src), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void prefetch_l1(const void *a) { asm volatile("prefetch.global.L1 [%0];" :: "l"(a)); }
// __syncwarp as a statement that the reads below cannot move across
__device__ __forceinline__ void warp_sync() { asm volatile("bar.warp.sync 0xFFFFFFFF;" ::: "memory"); }

__device__ __forceinline__ void unit_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint32_t lds16(const uint8_t *a) { return *reinterpret_cast<const uint16_t *>(a); }
__device__ __forceinline__ uint32_t lds8(const uint8_t *a) { return *a; }
// kWords (1, 2 or 4) words
template <int kWords>
__device__ __forceinline__ void lds_words(const uint8_t *a, uint32_t *d) {
    if (kWords == 1) {
        d[0] = *reinterpret_cast<const uint32_t *>(a);
    } else if (kWords == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(a);
        d[0] = v.x;
        d[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(a);
        d[0] = v.x;
        d[1] = v.y;
        d[2] = v.z;
        d[3] = v.w;
    }
}

// Length of sequence b (its tokens' table entries exist), and the tiles it
// counts in the schedule.
__device__ __forceinline__ int length_of(const PagedAttnParams &p, int b) {
    const int len = __ldg(p.seq_lens + b);
    return min(max(len, 0), p.capacity);
}
__device__ __forceinline__ int tiles_of(int len, int tile_shift) {
    return max(1, (int)(((uint32_t)len + (1u << tile_shift) - 1u) >> tile_shift));
}

// The list of tiles cut into ranges, the first `longer` of them one longer
// than the others (fewer tiles than CTAs: ranges of one tile).
struct Ranges {
    uint32_t length, longer, n, total;
    __device__ __forceinline__ uint32_t first(uint32_t x) const {
        return x >= n ? total : x * length + min(x, longer);
    }
    __device__ __forceinline__ uint32_t of(uint32_t tile) const {       // range of a tile
        const uint32_t split = longer * (length + 1);
        return tile < split ? tile / (length + 1) : longer + (tile - split) / length;
    }
};
__device__ __forceinline__ Ranges ranges_of(uint32_t total, uint32_t ctas) {
    Ranges r;
    r.total = total;
    r.n = min(total, ctas);
    r.length = total / r.n;
    r.longer = total - r.n * r.length;
    return r;
}

// A part of a sequence costs a CTA as much time as about three tiles (fetching
// length and query, the ending): a sequence counts so many more in the
// schedule.  None: 96 sequences of 256 to 8192 tokens 66.1 us, 32 of up to
// 3001 21.3 us; 2: 62.5 and 13.6; 3: 61.7 and 13.5; 5: 60.3 and 14.0.
constexpr uint32_t kPartTiles = 3;
constexpr int kWarpSchedule = 32;   // up to this many sequences each warp works the schedule out for itself, one a lane

// What the joining kernel has to know of a sequence that starts in this range.
__device__ __forceinline__ void write_join(const PagedAttnParams &p, const Ranges &r, int b, uint32_t at, int tiles) {
    const int x = (int)blockIdx.x, pieces = (int)r.of(at + tiles - 1) - x + 1;
    if (p.sequences <= (int)gridDim.x) p.joins[b] = make_int4(b, x, pieces, 0);
    else if (pieces > 1) p.joins[x] = make_int4(b, x, pieces, 0);
}

// A position in the list of tiles.
struct Cursor {
    int b, tile, tiles, len;
    // n tiles on, n at most to the end of the sequence
    template <int kTileShift>
    __device__ __forceinline__ void skip(const PagedAttnParams &p, int n, bool more) {
        tile += n;
        if (tile == tiles) {
            ++b;
            tile = 0;
            len = more ? length_of(p, b) : 0;
            tiles = tiles_of(len, kTileShift);
        }
    }
};

// A stage's rows by cp.async: 16-byte pieces of 2^kHeadsShift heads' codes, and
// kScales bytes of each head's scales, to where the boxes of TMA would lie.  A
// lane keeps its place in the rows; token t0 + i (t0 a lane's, i a multiple of
// the lanes' tokens) adds constants, as the swizzle is an xor of token bits.
template <int kD, int kPartsShift, int kHeadsShift>
__device__ __forceinline__ void copy_rows(const PagedAttnParams &p, const int *rows, uint32_t to, int head_first) {
    using S = Shape<kD>;
    constexpr int kHeads = 1 << kHeadsShift, kTokens = kTile << kPartsShift, kCodesTile = kTile * S::kCodes;
    constexpr uint32_t kV = kHeads * kTokens * S::kCodes;               // from K's codes to V's
    constexpr int kGroups = kHeads * S::kScales > 16 ? kHeads * S::kScales / 16 : 1;
    constexpr uint32_t kVScales = kGroups * kTokens * 16;
    const int lane = threadIdx.x & 31;
    {
        constexpr int kLanes = kHeads * S::kChunks, kStep = 32 / kLanes;    // lanes of a token, tokens of a step
        constexpr int kUnroll = kTokens / kStep < 8 ? kTokens / kStep : 8;  // 8 tokens or more: whole periods of the swizzle
        static_assert(kLanes <= 32 && kTokens % (kUnroll * kStep) == 0 && kUnroll * kStep >= 8, "whole rounds");
        const int x = lane % kLanes, t0 = lane / kLanes;
        const uint8_t *kc = p.kc + (int64_t)head_first * S::kCodes + 16 * x;
        const uint8_t *vc = p.vc + (int64_t)head_first * S::kCodes + 16 * x;
        const uint32_t dst = to + (x / S::kChunks) * kCodesTile + t0 * S::kCodes + 16 * swizzled<kD>(x % S::kChunks, t0);
#pragma unroll 1
        for (int t = 0; t < kTokens; t += kUnroll * kStep) {
            const uint32_t at = (uint32_t)(t / kTile) * (kHeads * kCodesTile) + (t % kTile) * S::kCodes;
            int r[kUnroll];
#pragma unroll
            for (int n = 0; n < kUnroll; ++n) r[n] = rows[t + t0 + n * kStep];
#pragma unroll
            for (int n = 0; n < kUnroll; ++n) {
                const int i = n * kStep;
                const uint32_t d = (dst ^ (16 * swizzled<kD>(0, i))) + at + (i / kTile) * (kHeads * kCodesTile) + (i % kTile) * S::kCodes;
                if (r[n] >= 0) {
                    copy_async<16>(d, kc + (int64_t)r[n] * p.row_codes);
                    copy_async<16>(d + kV, vc + (int64_t)r[n] * p.row_codes);
                }
            }
        }
    }
    constexpr int kStep = 32 / kHeads;
    const int h = lane % kHeads, t0 = lane / kHeads, byte = (head_first + h) * S::kScales;     // of a row's scales
    const uint32_t dst = to + 2 * kV + ((byte - ((head_first * S::kScales) & ~15)) >> 4) * (16 * kTile) + (byte & 15) +
                         (t0 / kTile) * (kGroups * 16 * kTile) + (t0 % kTile) * 16;
    const uint8_t *ks = p.ks + byte, *vs = p.vs + byte;
#pragma unroll
    for (int i = 0; i < kTokens; i += kStep) {
        const int r = rows[t0 + i];
        const uint32_t d = dst + (i / kTile) * (kGroups * 16 * kTile) + (i % kTile) * 16;
        if (r >= 0) {
            copy_async<S::kScales>(d, ks + (int64_t)r * p.row_scales);
            copy_async<S::kScales>(d + kVScales, vs + (int64_t)r * p.row_scales);
        }
    }
}

}  // namespace

template <int kD, bool kTma, int kPartsShift>
__global__ void __launch_bounds__(32 * (kWarps + Producers<kD, kTma>::kCount), Shape<kD>::kCtasPerSm)
k_paged_attention(const __grid_constant__ PagedAttnParams p, const __grid_constant__ PagedMaps maps) {
    using S = Shape<kD>;
    constexpr int kProducers = Producers<kD, kTma>::kCount, kThreads = 32 * (kWarps + kProducers);
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kPagedMaxStages], empty[kPagedMaxStages];
    __shared__ int masks[kPagedMaxStages][kWarps];
    __shared__ int armed[kPagedMaxStages];               // 1 + parity of the phase of `full` that was armed last, 0: none (TMA)
    __shared__ int rows_sh[kProducers][kWarps * kTile];  // pool rows of a stage's tokens (copies without TMA)
    __shared__ float4 ml[kWarps][4];                     // (m, l) of heads 2c and 2c + 1
    __shared__ uint32_t warp_sums[kWarps + kProducers];
    __shared__ Cursor start_sh;
    __shared__ int count_sh;
    grid_dependents_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < p.plan.stages) {
        mbar_init(&full[tid], kTma ? 1 : 33);
        mbar_init(&empty[tid], kWarps);
        armed[tid] = 0;
    }
    fence_barrier_init();
    // what is read from here on may be the result of the kernels before
    grid_dependency_wait();

    const float gk = __ldg(p.gk);        // used after the schedule, which hides the load

    // ---- schedule: this CTA's range of the tiles, and where it starts
    Cursor start;
    int count;
    if (p.sequences <= kWarpSchedule) {
        int len = 0;
        uint32_t tiles = 0;
        if (lane < p.sequences) {
            const int given = __ldg(p.seq_lens + lane);
            len = min(max(given, 0), p.capacity);
            tiles = tiles_of(len, 4 + kPartsShift);
            if (given != len && warp == 0 && blockIdx.x == 0 && blockIdx.y == 0) set_status(p.status, ST_INVALID_ARG);
        }
        const uint32_t mine = tiles > 0 ? tiles + kPartTiles : 0u;
        uint32_t upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, off);
            if (lane >= off) upto += v;
        }
        const Ranges ranges = ranges_of(__shfl_sync(0xFFFFFFFFu, upto, 31), gridDim.x);
        const uint32_t first = ranges.first(blockIdx.x), last = ranges.first(blockIdx.x + 1), at = upto - tiles;
        // tiles of this sequence in the range, and of all of them
        const uint32_t from_tile = min(tiles, first > at ? first - at : 0u), to_tile = min(tiles, last > at ? last - at : 0u);
        count = (int)__reduce_add_sync(0xFFFFFFFFu, to_tile - from_tile);
        if (warp == 0 && blockIdx.y == 0) {
            if (p.sequences > (int)gridDim.x && lane == 0) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
            __syncwarp();
            if (tiles > 0 && at >= first && at < last) write_join(p, ranges, lane, at, (int)tiles);
        }
        start = Cursor{lane, (int)from_tile, (int)tiles, len};
        const int from = __ffs(__ballot_sync(0xFFFFFFFFu, to_tile > from_tile)) - 1;
        start.b = __shfl_sync(0xFFFFFFFFu, start.b, from & 31);
        start.tile = __shfl_sync(0xFFFFFFFFu, start.tile, from & 31);
        start.tiles = __shfl_sync(0xFFFFFFFFu, start.tiles, from & 31);
        start.len = __shfl_sync(0xFFFFFFFFu, start.len, from & 31);
        __syncthreads();                                                // the barriers are set up
    } else {
        const int per = (p.sequences + kThreads - 1) / kThreads;
        const int b0 = min(p.sequences, tid * per), b1 = min(p.sequences, b0 + per);
        uint32_t mine = 0;
        bool wrong = false;
#pragma unroll 4
        for (int b = b0; b < b1; ++b) {
            const int len = __ldg(p.seq_lens + b);
            wrong |= len < 0 || len > p.capacity;
            mine += tiles_of(min(max(len, 0), p.capacity), (4 + kPartsShift)) + kPartTiles;
        }
        if (wrong && blockIdx.x == 0 && blockIdx.y == 0) set_status(p.status, ST_INVALID_ARG);
        uint32_t upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, off);
            if (lane >= off) upto += v;
        }
        if (lane == 31) warp_sums[warp] = upto;
        if (blockIdx.y == 0 && p.sequences > (int)gridDim.x && tid == 0) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
        if (tid == 0) count_sh = 0;
        __syncthreads();
        uint32_t total = 0;
#pragma unroll
        for (int w = 0; w < kWarps + kProducers; ++w) {
            if (w == warp) upto += total;
            total += warp_sums[w];
        }
        const Ranges ranges = ranges_of(total, gridDim.x);
        const uint32_t first = ranges.first(blockIdx.x), last = ranges.first(blockIdx.x + 1);
        uint32_t at = upto - mine;
        if (at < last && upto > first) {
            int tiles_here = 0;
#pragma unroll 1
            for (int b = b0; b < b1; ++b) {
                const int len = length_of(p, b);
                const uint32_t tiles = tiles_of(len, (4 + kPartsShift));
                at += kPartTiles;
                const uint32_t from_tile = min(tiles, first > at ? first - at : 0u), to_tile = min(tiles, last > at ? last - at : 0u);
                // the one sequence with the first tile at or behind the range's start
                if (to_tile > from_tile && (from_tile > 0 || at - first <= kPartTiles)) start_sh = Cursor{b, (int)from_tile, (int)tiles, len};
                tiles_here += (int)(to_tile - from_tile);
                if (blockIdx.y == 0 && at >= first && at < last) write_join(p, ranges, b, at, (int)tiles);
                at += tiles;
            }
            if (tiles_here > 0) atomicAdd(&count_sh, tiles_here);
        }
        __syncthreads();
        start = start_sh;
        count = count_sh;
    }
    if (count <= 0) return;

    const PagedPlan &plan = p.plan;
    constexpr int tw = 1 << kPartsShift;                                // warps that share a unit's tokens
    const int heads_cta = 1 << plan.heads_shift;
    const int head_block = (int)quotient(blockIdx.y, p.sub_blocks);     // CTAs over the heads, then over a head's units
    const int head_first = head_block << plan.heads_shift;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t v_codes = (uint32_t)(tw * heads_cta * kTile) * S::kCodes;   // within a stage: K codes, V codes, scales
    const uint32_t k_scales = 2 * v_codes;
    const int scale_groups = max(1, (heads_cta * S::kScales) >> 4);     // 16-byte groups of a token's scales
    const uint32_t v_scales = k_scales + tw * scale_groups * (16 * kTile);
    bool failed = false;

    if (warp >= kWarps) {
        // ================= brings the tiles in =================
        Cursor at = start;
        int left = count, stage = 0;
        uint32_t phase = 1;                                             // of `empty`: the first round passes
        auto acquire = [&]() {
            if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(&empty[stage], phase))) {
                failed = !__all_sync(0xFFFFFFFFu, bounded_wait(&empty[stage], phase, p.timeout));
                if (failed && lane == 0) set_status(p.status, ST_TIMEOUT);
            }
        };
        int turn = warp - kWarps;                                       // tiles until this warp's next one
        auto my_turn = [&]() { return turn == 0; };
        auto advance = [&]() {
            turn = turn == 0 ? kProducers - 1 : turn - 1;
            if (++stage == plan.stages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        if constexpr (kTma) {
            // Lane l looks up 16 tokens: part l % tw of tile l / tw of a batch
            // of tiles of one sequence; the next batch is looked up before
            // this one is copied.  One lane issues all copies of a stage (a
            // TMA instruction takes its operands from one thread at a time).
            const int per_batch = 32 >> kPartsShift, my_part = lane & (tw - 1);
            const int group_first = (head_first * S::kScales) >> 4;
            const uint32_t part_codes = heads_cta * kTile * S::kCodes, part_scales = scale_groups * 16 * kTile;
            struct Batch {
                int n, page, offset, tokens;
            };
            auto lookup = [&]() {
                Batch f = {0, 0, 0, 0};
                if (left > 0) {
                    f.n = min(per_batch, min(left, at.tiles - at.tile));
                    const int my_tile = lane >> kPartsShift;
                    const int t = ((at.tile + my_tile) << (4 + kPartsShift)) + kTile * my_part;
                    if (my_tile < f.n && t < at.len) {
                        const uint32_t entry = quotient((uint32_t)t, p.page_div);
                        f.offset = t - (int)(entry * p.page_div.d);
                        f.tokens = min(kTile, at.len - t);
                        f.page = __ldg(p.block_table + (int64_t)at.b * p.table_stride + entry);
                    }
                    left -= f.n;
                    at.skip<4 + kPartsShift>(p, f.n, left > 0);
                }
                return f;
            };
            const uint32_t bytes = 2u * (part_codes + part_scales);
            Batch f = lookup();
            while (f.n > 0) {
                const Batch next = lookup();
                if (f.tokens > 0 && (uint32_t)f.page >= (uint32_t)p.n_pages) {
                    set_status(p.status, ST_INVALID_ARG);
                    f.page = f.tokens = 0;
                }
                const int row = f.page * p.page_size + f.offset;
#pragma unroll 1
                for (int i = 0; i < f.n; ++i) {
                    if (!my_turn()) {
                        advance();
                        continue;
                    }
                    const int from = (i << kPartsShift) + my_part;
                    const int my_row = __shfl_sync(0xFFFFFFFFu, row, from);
                    const int tokens = __shfl_sync(0xFFFFFFFFu, f.tokens, from);
                    const uint32_t there = __ballot_sync(0xFFFFFFFFu, lane < tw && tokens > 0);
                    acquire();
                    if (failed) break;
                    if (lane < tw) masks[stage][lane] = (1 << tokens) - 1;
                    __syncwarp();
                    if (lane == 0) {
                        armed[stage] = 1 + (int)(phase ^ 1u);
                        mbar_arrive_expect_tx(&full[stage], __popc(there) * bytes);
                    }
                    uint32_t to = ring + stage * plan.stage_bytes, scales = to + k_scales;
#pragma unroll 1
                    for (int n = 0; n < tw; ++n, to += part_codes, scales += part_scales) {
                        const int r = __shfl_sync(0xFFFFFFFFu, my_row, n);
                        if (lane == 0 && ((there >> n) & 1u)) {
                            tma_load_3d(to, &maps.kc, &full[stage], 0, r, head_first);
                            tma_load_3d(scales, &maps.ks, &full[stage], 0, r, group_first);
                            tma_load_3d(to + v_codes, &maps.vc, &full[stage], 0, r, head_first);
                            tma_load_3d(scales + (v_scales - k_scales), &maps.vs, &full[stage], 0, r, group_first);
                        }
                    }
                    __syncwarp();
                    advance();
                }
                if (failed) break;
                f = next;
            }
            // No copy may be under way when the CTA ends, whoever has given up
            // waiting for it: once neither warp arms a stage any more, the
            // phase that was last armed of each is awaited.
            unit_barrier(kProducerBarrier, 32 * kProducers);
#pragma unroll 1
            for (int n = 0; n < plan.stages; ++n)
                if (armed[n] != 0) bounded_wait(&full[n], (uint32_t)armed[n] - 1u, kDrainCycles);
        } else {
            // Pages that end inside of a tile, or rows that TMA cannot step
            // by: the rows of a stage's tokens are looked up one stage ahead,
            // and copied in 16-byte pieces of the codes and kScales of a
            // head's scales.
            const int tokens_stage = kTile << kPartsShift;
            int *rows = rows_sh[warp - kWarps];
            int pages[4], offsets[4];                                   // tokens lane, lane + 32, ...
            auto lookup = [&]() {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    pages[k] = -1;
                    offsets[k] = -1;
                    const int local = 32 * k + lane, t = (at.tile << (4 + kPartsShift)) + local;
                    if (left > 0 && local < tokens_stage && t < at.len) {
                        const uint32_t entry = quotient((uint32_t)t, p.page_div);
                        offsets[k] = t - (int)(entry * p.page_div.d);
                        pages[k] = __ldg(p.block_table + (int64_t)at.b * p.table_stride + entry);
                    }
                }
            };
            auto pass = [&](int n) {                                    // n tiles on
                for (; n > 0 && left > 0; --n) at.skip<4 + kPartsShift>(p, 1, --left > 0);
            };
            pass(turn);
            lookup();
#pragma unroll 1
            for (int i = 0; i < count; ++i) {
                if (!my_turn()) {
                    advance();
                    continue;
                }
                acquire();
                if (failed) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bool ok = offsets[k] >= 0;
                    if (ok && (uint32_t)pages[k] >= (uint32_t)p.n_pages) {
                        set_status(p.status, ST_INVALID_ARG);
                        ok = false;
                    }
                    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
                    const int local = 32 * k + lane;
                    if (local < tokens_stage) {
                        rows[local] = ok ? pages[k] * p.page_size + offsets[k] : -1;
                        if ((lane & 15) == 0) masks[stage][local >> 4] = (int)((mask >> (lane & 16)) & 0xFFFFu);
                    }
                }
                pass(kProducers);
                lookup();
                __syncwarp();
                const uint32_t to = ring + stage * plan.stage_bytes;
                if (plan.heads_shift == 0) copy_rows<kD, kPartsShift, 0>(p, rows, to, head_first);
                if constexpr (kPartsShift < 3)
                    if (plan.heads_shift == 1) copy_rows<kD, kPartsShift, 1>(p, rows, to, head_first);
                if constexpr (kPartsShift < 2)
                    if (plan.heads_shift == 2) copy_rows<kD, kPartsShift, 2>(p, rows, to, head_first);
                copies_arrive(&full[stage]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[stage]);               // the masks
                advance();
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        return;
    }

    // ================= computes =================
    const int g = lane >> 2, c = lane & 3;
    const int unit_cta = warp & ((1 << (plan.heads_shift + plan.subs_shift)) - 1);   // unit of this CTA, and part of its tokens
    const int part = warp >> (plan.heads_shift + plan.subs_shift);
    const int head_cta = unit_cta >> plan.subs_shift;
    const int hk = head_first + head_cta;
    const int sub = (((int)blockIdx.y - head_block * (int)p.sub_blocks.d) << plan.subs_shift) + (unit_cta & ((1 << plan.subs_shift) - 1));
    const int unit = hk * plan.units_head + sub;
    const int head0 = hk * p.group + sub * 8;
    const int heads = min(8, p.group - sub * 8);                        // query heads of this unit
    const float cscale = __fmul_rn(__fmul_rn(p.scale, kLog2e), __frcp_rn(gk));

    // ---- lane constants of the fragment reads, from the start of a stage
    const int tk = token_of<kD>(g >> 1, g & 1);                         // token of MMA row g (row g + 8: + 8)
    const int ta = token_of<kD>(c, 0), tb = token_of<kD>(c, 1);         // tokens of MMA rows 2c, 2c + 1
    constexpr int kVWords = kD / 64;                                    // words of V codes a lane takes per token
    constexpr int kKWords = kD == 64 ? 2 : 4;
    uint32_t k_at[2], va_at, vb_at, ks_at, vs_at;
    {
        const uint32_t tile = ((part << plan.heads_shift) + head_cta) * (kTile * S::kCodes);
        if (kD == 64) {
            k_at[0] = k_at[1] = tile + tk * S::kCodes + 8 * c;
            va_at = ta * S::kCodes + 4 * g;
            vb_at = tb * S::kCodes + 4 * g;
        } else if (kD == 128) {
            k_at[0] = k_at[1] = tile + tk * S::kCodes + 16 * swizzled<kD>(c, tk);
            va_at = ta * S::kCodes + 16 * swizzled<kD>(g >> 1, ta) + 8 * (g & 1);
            vb_at = tb * S::kCodes + 16 * swizzled<kD>(g >> 1, tb) + 8 * (g & 1);
        } else {
            k_at[0] = tile + tk * S::kCodes + 16 * swizzled<kD>(c, tk);
            k_at[1] = tile + tk * S::kCodes + 16 * swizzled<kD>(c + 4, tk);
            va_at = ta * S::kCodes + 16 * swizzled<kD>(g, ta);
            vb_at = tb * S::kCodes + 16 * swizzled<kD>(g, tb);
        }
        va_at += tile + v_codes;
        vb_at += tile + v_codes;
        const int x = hk * S::kScales;
        const uint32_t scales = (part * scale_groups + ((x - ((head_first * S::kScales) & ~15)) >> 4)) * (16 * kTile) + (x & 15);
        ks_at = k_scales + scales + tk * 16 + (kD == 64 ? c : 2 * c);
        vs_at = v_scales + scales + (kD == 64 ? g >> 1 : kD == 128 ? g : 2 * g);
    }

    // the warps' O, where several share a unit's tokens
    float4 *sums = reinterpret_cast<float4 *>(smem_raw + (ring - smem_u32(smem_raw)) + plan.stages * plan.stage_bytes);
    // B fragments of the query, kept where the warp's sums go later: registers
    // are what limits the warps of an SM here
    uint4 *q_frag = reinterpret_cast<uint4 *>(sums + warp * (2 * kD)) + lane;
    float oacc[S::kSteps][4];
    float lsum[2], mp[2], ck[2];
    int b = start.b, in_seq = start.tiles - start.tile;        // tiles to the end of the sequence
    bool starts_here = start.tile == 0;
    int left = count, stage = 0;
    uint32_t phase = 0;
    bool ready = false;
    const uint8_t *ring_at = smem_raw + (ring - smem_u32(smem_raw)), *at = ring_at;

    while (true) {
        {   // query of head g: lane c holds dims kD / 4 * c ... (kD = 256: 32c .. + 31 and 128 + 32c .. + 31)
            uint4 w[kD / 32];
            uint32_t amax = 0u;
            const uint16_t *q = p.q + (int64_t)b * p.qs_b + (int64_t)(head0 + g) * p.qs_h;
#pragma unroll
            for (int n = 0; n < kD / 32; ++n) {
                const int d = kD == 256 ? 32 * c + 8 * (n & 3) + 128 * (n >> 2) : (kD / 4) * c + 8 * n;
                // a plain load: o may be q, which the kernel then writes
                w[n] = g < heads ? *reinterpret_cast<const uint4 *>(q + d) : make_uint4(0u, 0u, 0u, 0u);
                amax = max_u16x2(amax, max_u16x2(max_u16x2(w[n].x & 0x7FFF7FFFu, w[n].y & 0x7FFF7FFFu),
                                                 max_u16x2(w[n].z & 0x7FFF7FFFu, w[n].w & 0x7FFF7FFFu)));
            }
            uint32_t e = max(amax & 0xFFFFu, amax >> 16) >> 7;          // exponent field of the largest value
            e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 1));
            e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 2));
            // times 2^(14 - (e - 127)), within FP32's exponents (so that a
            // query of subnormal values is held, exactly); one with infinities
            // or NaN stays as it is
            const int up = e == 255u ? 0 : min(141 - (int)e, 126);
            const float mult = __uint_as_float((uint32_t)(127 + up) << 23);
            const float undo = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int n = 0; n < kD / 32; ++n) {
                const uint32_t x[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
                uint32_t y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[k] = f16x2_from_f32(__fmul_rn(bf16_lo(x[k]), mult), __fmul_rn(bf16_hi(x[k]), mult));
                q_frag[32 * n] = make_uint4(y[0], y[1], y[2], y[3]);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                ck[n] = __fmul_rn(cscale, __shfl_sync(0xFFFFFFFFu, undo, 8 * c + 4 * n));
                lsum[n] = 0.0f;
                mp[n] = kLowest;
            }
#pragma unroll
            for (int j = 0; j < S::kSteps; ++j)
#pragma unroll
                for (int n = 0; n < 4; ++n) oacc[j][n] = 0.0f;
        }
        const bool ends = in_seq <= left;                               // the sequence ends in this range
        const int n_tiles = ends ? in_seq : left;
        left -= n_tiles;
#pragma unroll 1
        for (int tile = n_tiles; tile > 0; --tile) {
            // A wait that gives up leaves the unit in step: its tiles then
            // count as empty, every barrier of the unit is still met.
            if (!failed && !ready) {
                failed = !__all_sync(0xFFFFFFFFu, bounded_wait(&full[stage], phase, p.timeout));
                if (failed) set_status(p.status, ST_TIMEOUT);
            }
            const int next = stage + 1 == plan.stages ? 0 : stage + 1;
            const uint32_t mask = failed ? 0u : (uint32_t)masks[stage][part];

            // ---- S = K q^T
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int part_k = 0; part_k < (kD == 256 ? 2 : 1); ++part_k) {
                uint32_t w0[kKWords], w1[kKWords];
                lds_words<kKWords>(at + k_at[part_k], w0);
                lds_words<kKWords>(at + k_at[part_k] + 8 * S::kCodes, w1);
                uint32_t s0[2], s1[2];                                  // scales of rows g, g + 8 as (s, s)
                if (kD == 64) {
                    const uint32_t x = f16x2_from_e4m3x2(lds8(at + ks_at) | (lds8(at + ks_at + 128) << 8));
                    s0[0] = s0[1] = __byte_perm(x, x, 0x1010);
                    s1[0] = s1[1] = __byte_perm(x, x, 0x3232);
                } else {
                    const uint32_t x0 = f16x2_from_e4m3x2(lds16(at + ks_at + 8 * part_k));
                    const uint32_t x1 = f16x2_from_e4m3x2(lds16(at + ks_at + 8 * part_k + 128));
                    s0[0] = __byte_perm(x0, x0, 0x1010);
                    s0[1] = __byte_perm(x0, x0, 0x3232);
                    s1[0] = __byte_perm(x1, x1, 0x1010);
                    s1[1] = __byte_perm(x1, x1, 0x3232);
                }
#pragma unroll
                for (int n = 0; n < kKWords; ++n) {                     // two MMA steps a word
                    uint32_t x[4], y[4];
                    f16x2_from_word(w0[n], x);
                    f16x2_from_word(w1[n], y);
                    const int blk = n / 2;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[k] = mul_f16x2(x[k], s0[blk]);
                        y[k] = mul_f16x2(y[k], s1[blk]);
                    }
                    const uint4 f = q_frag[32 * (4 * part_k + n)];
                    mma_f16(s, x[0], y[0], x[1], y[1], f.x, f.y);
                    mma_f16(s, x[2], y[2], x[3], y[3], f.z, f.w);
                }
            }
            uint32_t wa[2][kVWords], wb[2][kVWords], sc[2][2];          // [rows 2c.. / 2c + 8 ..]
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                lds_words<kVWords>(at + va_at + 8 * n * S::kCodes, wa[n]);
                lds_words<kVWords>(at + vb_at + 8 * n * S::kCodes, wb[n]);
                if (kD == 256) {
                    const uint32_t x = lds16(at + vs_at + (ta + 8 * n) * 16);
                    const uint32_t y = lds16(at + vs_at + (tb + 8 * n) * 16);
                    sc[n][0] = f16x2_from_e4m3x2(__byte_perm(x, y, 0x0040));
                    sc[n][1] = f16x2_from_e4m3x2(__byte_perm(x, y, 0x0051));
                } else {
                    const uint32_t x = lds8(at + vs_at + (ta + 8 * n) * 16);
                    const uint32_t y = lds8(at + vs_at + (tb + 8 * n) * 16);
                    sc[n][0] = sc[n][1] = f16x2_from_e4m3x2(x | (y << 8));
                }
            }
            // whether the next tile is there: asked now, so that the answer is at hand
            ready = __all_sync(0xFFFFFFFFu, mbar_test_wait(&full[next], next == 0 ? phase ^ 1u : phase));
            // ---- weights: e = S c - m', rows tk and tk + 8, heads 2c and 2c + 1
            float e[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) e[n] = __fmaf_rn(s[n], ck[n & 1], -mp[n & 1]);
            if (mask != 0xFFFFu) {
                const bool r0 = (mask >> tk) & 1u, r1 = (mask >> (tk + 8)) & 1u;
                if (!r0) e[0] = e[1] = -__int_as_float(0x7F800000);
                if (!r1) e[2] = e[3] = -__int_as_float(0x7F800000);
            }
            if (__any_sync(0xFFFFFFFFu, fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])) > kSlack)) {
                const bool r0 = (mask >> tk) & 1u, r1 = (mask >> (tk + 8)) & 1u;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float x0 = __fmul_rn(s[n], ck[n]), x1 = __fmul_rn(s[n + 2], ck[n]);
                    float top = fmaxf(r0 ? x0 : kLowest, r1 ? x1 : kLowest);
#pragma unroll
                    for (int off = 4; off <= 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
                    const float mn = fmaxf(mp[n], top - kOffset);
                    const float alpha = exp2_fast(mp[n] - mn);
                    mp[n] = mn;
                    lsum[n] *= alpha;
#pragma unroll
                    for (int j = 0; j < S::kSteps; ++j) {
                        oacc[j][n] *= alpha;
                        oacc[j][n + 2] *= alpha;
                    }
                    // From the rounded x, as mn is: the exact product is off from
                    // x by 16 at 2^28, which would take the largest weight out of
                    // FP16's range on either side.  A score past FP32's range
                    // gives inf - inf, NaN in its head.
                    if (r0) e[n] = __fsub_rn(x0, mn);
                    if (r1) e[n + 2] = __fsub_rn(x1, mn);
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) e[n] = exp2_fast(e[n]);
            lsum[0] += e[0] + e[2];
            lsum[1] += e[1] + e[3];
            const uint32_t p0 = transpose_8x8(f16x2_from_f32(e[0], e[1]));
            const uint32_t p1 = transpose_8x8(f16x2_from_f32(e[2], e[3]));

            // ---- O^T += V^T P^T
            if (mask != 0xFFFFu) {
                // what lies in the rows of absent tokens is not theirs: with
                // a scale of 0 their values count 0 (any code is finite)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const uint32_t keep = (((mask >> (ta + 8 * n)) & 1u) ? 0xFFFFu : 0u) |
                                          (((mask >> (tb + 8 * n)) & 1u) ? 0xFFFF0000u : 0u);
                    sc[n][0] &= keep;
                    sc[n][1] &= keep;
                }
            }
#pragma unroll
            for (int n = 0; n < kVWords; ++n) {                         // four M-tiles a word
                uint32_t even[2][4], odd[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f16x2_from_word(nibbles(wa[h][n], wb[h][n] << 4), even[h]);
                    f16x2_from_word(nibbles(wa[h][n] >> 4, wb[h][n]), odd[h]);
                    const uint32_t x = sc[h][kD == 256 ? n / 2 : 0];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        even[h][k] = mul_f16x2(even[h][k], x);
                        odd[h][k] = mul_f16x2(odd[h][k], x);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_f16(oacc[4 * n + k], even[0][k], odd[0][k], even[1][k], odd[1][k], p0, p1);
            }
            // A warp that has given up hands no stage back, so that none is
            // armed again before all warps have seen its copies land; the
            // producers' own waits then run out.  (Leaving the loop instead
            // was 2 % slower at 64 x 8192.)
            warp_sync();
            if (lane == 0 && !failed) mbar_arrive(&empty[stage]);
            at += plan.stage_bytes;
            if (++stage == plan.stages) {
                stage = 0;
                phase ^= 1u;
                at = ring_at;
            }
        }

        // ---- end of this CTA's part of the sequence: the unit's warps meet
        // in shared memory, and each sums and stores its share of the M-tiles.
        // Rolled loops on purpose: with everything unrolled the kernel was
        // 131 KB, and fetching it made a one-token call 10.8 us, not 8.9.
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) lsum[n] += __shfl_xor_sync(0xFFFFFFFFu, lsum[n], off);
        float4 *mine = sums + warp * (2 * kD) + lane;
#pragma unroll
        for (int j = 0; j < S::kSteps; ++j) mine[32 * j] = make_float4(oacc[j][0], oacc[j][1], oacc[j][2], oacc[j][3]);
        if (g == 0) ml[warp][c] = make_float4(mp[0], lsum[0], mp[1], lsum[1]);
        int next_len = 0;
        if (left > 0) {                                             // length and query of the next sequence on their way
            next_len = length_of(p, b + 1);
            if (g < heads)
                prefetch_l1(p.q + (int64_t)(b + 1) * p.qs_b + (int64_t)(head0 + g) * p.qs_h + (kD == 256 ? 32 * c : (kD / 4) * c));
        }
        const int step = kWarps >> kPartsShift;                    // warps between two parts of a unit
        unit_barrier(1 + unit_cta, 32 * tw);
        float M[2] = {kLowest, kLowest}, L[2] = {0.0f, 0.0f};
#pragma unroll 1
        for (int w = unit_cta; w < kWarps; w += 2 * step) {
            const float4 v = ml[w][c], u = ml[w + step][c];
            M[0] = fmaxf(M[0], fmaxf(v.x, u.x));
            M[1] = fmaxf(M[1], fmaxf(v.z, u.z));
        }
#pragma unroll 1
        for (int w = unit_cta; w < kWarps; w += 2 * step) {
            const float4 v = ml[w][c], u = ml[w + step][c];
            L[0] += v.y * exp2_fast(v.x - M[0]) + u.y * exp2_fast(u.x - M[0]);
            L[1] += v.w * exp2_fast(v.z - M[1]) + u.w * exp2_fast(u.z - M[1]);
        }
        const bool whole = ends && starts_here;
        float f[2] = {1.0f, 1.0f}, post = 1.0f;
        if (whole) {
            const float gv = __ldg(p.gv);
            post = post_of(gv);
#pragma unroll
            for (int n = 0; n < 2; ++n) f[n] = share_of(L[n], gv, post);
        }
        const int h = head0 + 2 * c;
        const bool h0 = 2 * c < heads, h1 = 2 * c + 1 < heads;
        uint16_t *o = p.o + (int64_t)b * p.os_b + (int64_t)h * p.os_h + (kD / 8) * g;
        const int64_t slot = (int64_t)(2 * blockIdx.x + (starts_here ? 1 : 0)) * plan.units + unit;
        float4 *part_o = p.part_o + slot * (2 * kD) + lane;
#pragma unroll 1
        for (int j = part; j < S::kSteps; j += tw) {
            float r[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (int w = unit_cta; w < kWarps; w += 2 * step) {
                const float4 v = sums[w * (2 * kD) + 32 * j + lane], u = sums[(w + step) * (2 * kD) + 32 * j + lane];
                const float4 x = ml[w][c], y = ml[w + step][c];
                const float f0 = exp2_fast(x.x - M[0]), f1 = exp2_fast(x.z - M[1]);
                const float g0 = exp2_fast(y.x - M[0]), g1 = exp2_fast(y.z - M[1]);
                r[0] += v.x * f0 + u.x * g0;
                r[1] += v.y * f1 + u.y * g1;
                r[2] += v.z * f0 + u.z * g0;
                r[3] += v.w * f1 + u.w * g1;
            }
            if (whole) {
                if (h0) *reinterpret_cast<uint32_t *>(o + 2 * j) = bf16x2_from_f32(r[0] * f[0] * post, r[2] * f[0] * post);
                if (h1) *reinterpret_cast<uint32_t *>(o + p.os_h + 2 * j) = bf16x2_from_f32(r[1] * f[1] * post, r[3] * f[1] * post);
            } else {
                part_o[32 * j] = make_float4(r[0], r[1], r[2], r[3]);
            }
        }
        if (part == 0 && g == 0) {
            if (!whole) {
                p.part_ml[slot * 4 + c] = make_float4(M[0], L[0], M[1], L[1]);
            } else if (p.lse != nullptr) {
                float *lse = p.lse + (int64_t)b * p.heads_q + h;
                if (h0) lse[0] = lse_of(M[0], L[0]);
                if (h1) lse[1] = lse_of(M[1], L[1]);
            }
        }
        // what is read above is written again only behind the next barrier of the unit
        unit_barrier(1 + unit_cta, 32 * tw);
        if (left == 0) break;
        ++b;
        in_seq = tiles_of(next_len, (4 + kPartsShift));
        starts_here = true;
    }
}

// Joins the parts of the sequences that were cut: blockIdx.x is the sequence
// (or the range at whose end one is cut); its items are the M-tiles of O^T of
// each unit (128 values: 8 heads x 16 dims).  A warp takes four parts in one
// round of loads -- their maxima, sums and values -- with the running maximum
// and sum of the online softmax; 1 to 16 warps take an item by the number of
// its parts, and are joined in shared memory.
constexpr int kJoinWarps = 16;

__global__ void __launch_bounds__(32 * kJoinWarps) k_paged_combine(const __grid_constant__ PagedAttnParams p, int dim) {
    __shared__ float4 ml[kJoinWarps][4], sums[kJoinWarps][32];
    grid_dependents_launch();
    grid_dependency_wait();
    const int4 join = p.joins[blockIdx.x];
    const int b = join.x, x0 = join.y, pieces = join.z;
    if (pieces <= 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int tiles = dim / 16, units = p.plan.units, items = units * tiles;
    // log2 of the warps an item: enough for one round, or for two where that
    // would leave items for another pass
    int shift = 0;
    while (shift < 4 && (4 << shift) < pieces) ++shift;
    if (shift > 0 && (int)gridDim.y * (kJoinWarps >> shift) < items) --shift;
    const int mine = warp & ((1 << shift) - 1), first = warp - mine;    // place in the item's warps; the first of them
#pragma unroll 1
    for (int at = blockIdx.y * (kJoinWarps >> shift); at < items; at += gridDim.y * (kJoinWarps >> shift)) {
        const int item = at + (warp >> shift);
        const int unit = item / tiles, j = item - unit * tiles;
        // piece n: the first lies in the second slot of its range, the others in the first
        auto slot = [&](int n) { return (int64_t)(2 * (x0 + n) + (n == 0 ? 1 : 0)) * units + unit; };
        float m[2] = {kLowest, kLowest}, l[2] = {0.0f, 0.0f}, a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int n0 = 4 * mine; n0 < pieces && item < items; n0 += 4 << shift) {
            float4 o[4], v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = min(n0 + k, pieces - 1);
                o[k] = __ldcg(p.part_o + slot(n) * (2 * dim) + 32 * j + lane);
                v[k] = __ldcg(p.part_ml + slot(n) * 4 + c);
                if (n0 + k >= pieces) v[k] = make_float4(kLowest, 0.0f, kLowest, 0.0f), o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            const float t0 = fmaxf(fmaxf(fmaxf(m[0], v[0].x), fmaxf(v[1].x, v[2].x)), v[3].x);
            const float t1 = fmaxf(fmaxf(fmaxf(m[1], v[0].z), fmaxf(v[1].z, v[2].z)), v[3].z);
            const float f0 = exp2_fast(m[0] - t0), f1 = exp2_fast(m[1] - t1);
            m[0] = t0;
            m[1] = t1;
            l[0] *= f0;
            l[1] *= f1;
            a[0] *= f0;
            a[1] *= f1;
            a[2] *= f0;
            a[3] *= f1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float w0 = exp2_fast(v[k].x - t0), w1 = exp2_fast(v[k].z - t1);
                l[0] += v[k].y * w0;
                l[1] += v[k].w * w1;
                a[0] += o[k].x * w0;
                a[1] += o[k].y * w1;
                a[2] += o[k].z * w0;
                a[3] += o[k].w * w1;
            }
        }
        if (shift > 0) {
            sums[warp][lane] = make_float4(a[0], a[1], a[2], a[3]);
            if (g == 0) ml[warp][c] = make_float4(m[0], l[0], m[1], l[1]);
            __syncthreads();
            l[0] = l[1] = a[0] = a[1] = a[2] = a[3] = 0.0f;
#pragma unroll 1
            for (int w = first; w < first + (1 << shift) && mine == 0; ++w) {
                m[0] = fmaxf(m[0], ml[w][c].x);
                m[1] = fmaxf(m[1], ml[w][c].z);
            }
#pragma unroll 1
            for (int w = first; w < first + (1 << shift) && mine == 0; ++w) {
                const float4 v = ml[w][c], o = sums[w][lane];
                const float f0 = exp2_fast(v.x - m[0]), f1 = exp2_fast(v.z - m[1]);
                l[0] += v.y * f0;
                l[1] += v.w * f1;
                a[0] += o.x * f0;
                a[1] += o.y * f1;
                a[2] += o.z * f0;
                a[3] += o.w * f1;
            }
            __syncthreads();
        }
        if (mine == 0 && item < items) {
            const int hk = unit / p.plan.units_head, sub = unit - hk * p.plan.units_head;
            const int h = hk * p.group + sub * 8 + 2 * c, heads = min(8, p.group - sub * 8) - 2 * c;
            const float gv = __ldg(p.gv), post = post_of(gv);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                if (n < heads) {
                    const float f = share_of(l[n], gv, post);
                    *reinterpret_cast<uint32_t *>(p.o + (int64_t)b * p.os_b + (int64_t)(h + n) * p.os_h + (dim / 8) * g + 2 * j) =
                        bf16x2_from_f32(a[n] * f * post, a[n + 2] * f * post);
                    if (j == 0 && g == 0 && p.lse != nullptr) p.lse[(int64_t)b * p.heads_q + h + n] = lse_of(m[n], l[n]);
                }
            }
        }
    }
}

namespace {

cudaError_t launch_dependent(const void *kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, void **args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <int kD, bool kTma, int kPartsShift>
cudaError_t launch_main(const PagedAttnParams &p, const PagedMaps &maps, cudaStream_t s) {
    constexpr int kProducers = Producers<kD, kTma>::kCount;
    // with fewer stages a producer could take a barrier's phase for the one after
    if (p.plan.stages < kProducers) return cudaErrorInvalidConfiguration;
    static std::atomic<uint64_t> ready{0};               // devices (below 64) with the shared memory allowed
    const void *kernel = (const void *)k_paged_attention<kD, kTma, kPartsShift>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!((ready.load(std::memory_order_relaxed) >> dev) & 1u)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kD == 256 ? kPagedSmem256 : kPagedSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    void *args[] = {const_cast<PagedAttnParams *>(&p), const_cast<PagedMaps *>(&maps)};
    return launch_dependent(kernel, dim3((unsigned)p.plan.ranges, (unsigned)p.plan.blocks), 32 * (kWarps + kProducers),
                            (size_t)p.plan.smem, s, args);
}

// Parts that the plan can ask for: with TMA a row's scales are whole 16-byte
// groups, so that there are at least 4 heads of 64 or 2 of 128 values.
template <int kD>
cudaError_t launch_parts(const PagedAttnParams &p, const PagedMaps &maps, cudaStream_t s) {
    const int parts = p.plan.parts_shift;
    if (p.tma) {
        if (parts == 1) return launch_main<kD, true, 1>(p, maps, s);
        if constexpr (kD >= 128)
            if (parts == 2) return launch_main<kD, true, 2>(p, maps, s);
        if constexpr (kD == 256)
            if (parts == 3) return launch_main<kD, true, 3>(p, maps, s);
    } else {
        if (parts == 1) return launch_main<kD, false, 1>(p, maps, s);
        if (parts == 2) return launch_main<kD, false, 2>(p, maps, s);
        if (parts == 3) return launch_main<kD, false, 3>(p, maps, s);
    }
    return cudaErrorInvalidConfiguration;
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnParams &p, const PagedMaps &maps, int dim, cudaStream_t s) {
    cudaError_t e = dim == 64 ? launch_parts<64>(p, maps, s)
                    : dim == 128 ? launch_parts<128>(p, maps, s)
                                 : launch_parts<256>(p, maps, s);
    if (e != cudaSuccess) return e;
    // the sequences that can be cut; CTAs for a warp an item, and where the
    // sequences are few, up to a CTA an item, within about four an SM
    const int joins = std::min(p.sequences, p.plan.ranges);
    const int items = p.plan.units * (dim / 16);
    const int y = std::min(items, std::max((items + kJoinWarps - 1) / kJoinWarps, 592 / joins));
    void *args[] = {const_cast<PagedAttnParams *>(&p), &dim};
    return launch_dependent((const void *)k_paged_combine, dim3((unsigned)joins, (unsigned)y), 32 * kJoinWarps, 0, s, args);
}

}  // namespace nvfp4
