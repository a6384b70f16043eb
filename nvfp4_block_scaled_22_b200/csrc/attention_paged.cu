// Decode attention of a batch of sequences over a paged NVFP4 KV cache: one
// query token a sequence, grouped-query heads,
//   s_t = scale q . k_t,  o = sum_t exp(s_t) v_t / sum_t exp(s_t),
// t over the sequence's cached tokens; token t lives in pool row
// block_table[b][t / page_size] * page_size + t % page_size.
//
// Each cache byte is read once (0.5625 bytes a value) and restored in
// registers; the bound is that read, as long as a value costs no more than
// about three instructions of a lane (148 SMs hold 79 values a ns each at the
// measured copy rate).
//
// Units and warps.  A unit is a KV head with up to 8 of its query heads (the 8
// columns of an MMA); larger groups are several units.  A CTA has 8 warps
// over `units_cta` neighbouring units (so that it reads whole pieces of a
// cache row) and 8 / units_cta warps share the tokens of one unit.  Every
// warp runs on its own 16-token tiles through a ring of cp.async stages and
// keeps its own online softmax; nothing in the loop waits for another warp.
//
// Schedule.  The sequences' tiles (16 tokens times the warps of a unit; an
// empty sequence counts one) are one list, cut into equal ranges, one a CTA,
// on the device from seq_lens: no CTA has more than one tile above another
// whatever the lengths, and the host needs no length.  A sequence that ends
// inside of its CTA's range is written at once; one that is cut leaves a
// partial (m, l, O) per CTA, which k_paged_combine joins in CTA order.
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
//     2^14, and the largest p of a head is at least 2^6, so that rounding p
//     to FP16 for the product with V costs 2^-11 of each weight, or 2^-31 of
//     the largest for tiny ones.  The sum l takes the unrounded p in FP32.
//   O^T[dim x 8 heads] += V^T P^T, the same MMA: P goes from accumulator to
//     operand layout by movmatrix; the codes of two tokens are interleaved
//     by nibbles so that one conversion gives the two tokens of one dim.
//   Token r of an MMA is token tau(r) of the tile (r = 8h + 2c + j: tau = 8h
//   + 4j + (c ^ 3j)), and 16-byte pieces are stored xor-swizzled, so that
//   both the row-wise reads of K and the column-wise reads of V meet no
//   shared-memory bank twice.
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

constexpr int kWarps = 8;
constexpr int kStages = 4;
constexpr int kTile = 16;            // tokens a warp takes at once

template <int kD>
struct Shape {
    static constexpr int kCodes = kD / 2;                       // bytes of a token's codes
    static constexpr int kScales = kD / 16;
    static constexpr int kChunks = kD / 32;                     // 16-byte pieces of a token's codes
    static constexpr int kSteps = kD / 16;                      // MMA steps over the dims (and M-tiles of O^T)
    static constexpr int kStage = 2 * kTile * (kCodes + kScales);
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kSum = kWarps * 8 * kD * 4;            // the warps' O, for the join
    static constexpr int kSmem = kRing + kSum;
    static constexpr int kCtasPerSm = kD == 256 ? 1 : 2;
};

// Piece of token t where piece `ch` is stored.
template <int kD>
__device__ __forceinline__ int swizzled(int ch, int t) {
    if (kD == 64) return ch;
    if (kD == 128) return ch ^ (t & 2);
    return ch ^ (2 * (t & 3));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
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

// (a & m) | (b & ~m), m = 0x0F0F0F0F
__device__ __forceinline__ uint32_t nibbles(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(d) : "r"(0x0F0F0F0Fu), "r"(a), "r"(b));
    return d;
}

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool there) {
    const int n = there ? kBytes : 0;                           // 0: the destination is zero-filled
    if (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" :: "r"(dst), "l"(src), "n"(kBytes), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(kLeft) : "memory");
}

// __syncwarp as a statement that the reads below cannot move across
__device__ __forceinline__ void warp_sync() { asm volatile("bar.warp.sync 0xFFFFFFFF;" ::: "memory"); }

__device__ __forceinline__ void unit_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t d;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t d;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(d) : "r"(a));
    return d;
}
// kWords (1, 2 or 4) words
template <int kWords>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t *d) {
    if (kWords == 1)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(d[0]) : "r"(a));
    else if (kWords == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(d[0]), "=r"(d[1]) : "r"(a));
    else
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(a));
}

// Length of sequence b (its tokens' table entries exist), and the tiles it
// counts in the schedule.
__device__ __forceinline__ int length_of(const PagedAttnParams &p, int b) {
    const int len = p.seq_lens[b];
    return len < 0 ? 0 : min(len, p.capacity);
}
__device__ __forceinline__ int tiles_of(int len, int tile_shift) {
    return max(1, (int)(((uint32_t)len + (1u << tile_shift) - 1u) >> tile_shift));
}

// A position in the list of tiles.
struct Cursor {
    int b, tile, tiles, len;
    __device__ __forceinline__ void next(const PagedAttnParams &p, bool more) {
        if (++tile == tiles) {
            ++b;
            tile = 0;
            len = more ? length_of(p, b) : 0;
            tiles = tiles_of(len, p.tile_shift);
        }
    }
};

}  // namespace

template <int kD>
__global__ void __launch_bounds__(kWarps * 32, Shape<kD>::kCtasPerSm) k_paged_attention(PagedAttnParams p) {
    using S = Shape<kD>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int masks[kWarps][kStages];
    __shared__ float ml[kWarps][8][2];
    __shared__ int64_t warp_sums[kWarps];
    __shared__ Cursor start_sh;
    grid_dependents_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;

    // ---- schedule: this CTA's range [first, first + count) of the tiles
    int64_t first;
    int count;
    {
        const int per = (p.sequences + kWarps * 32 - 1) / (kWarps * 32);
        const int b0 = min(p.sequences, tid * per), b1 = min(p.sequences, b0 + per);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) {
            const int len = p.seq_lens[b];
            if ((len < 0 || len > p.capacity) && blockIdx.x == 0 && blockIdx.y == 0) set_status(p.status, ST_INVALID_ARG);
            mine += tiles_of(length_of(p, b), p.tile_shift);
        }
        int64_t upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, off);
            if (lane >= off) upto += v;
        }
        if (lane == 31) warp_sums[warp] = upto;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) upto += total;
            total += warp_sums[w];
        }
        const int64_t ranges = min((int64_t)gridDim.x, (total + p.min_tiles - 1) / p.min_tiles);
        const int64_t x = blockIdx.x;
        first = x < ranges ? x * total / ranges : total;
        const int64_t last = x < ranges ? (x + 1) * total / ranges : total;
        count = (int)(last - first);
        // the threads whose sequences hold the first tile of a range, or
        // start in it, write down what the joining kernel needs
        int64_t at = upto - mine;
        const bool by_sequence = p.sequences <= (int)gridDim.x;
        if (blockIdx.y == 0 && !by_sequence && tid == 0) p.joins[x] = make_int4(0, 0, 0, 0);
        if (blockIdx.y == 0 && !by_sequence) __syncthreads();
        for (int b = b0; b < b1; ++b) {
            const int len = length_of(p, b), n = tiles_of(len, p.tile_shift);
            if (at <= first && first < at + n && count > 0) {
                start_sh.b = b;
                start_sh.tile = (int)(first - at);
                start_sh.tiles = n;
                start_sh.len = len;
            }
            if (blockIdx.y == 0 && at >= first && at < last) {
                const int64_t end = ((at + n) * ranges - 1) / total;      // range of the sequence's last tile
                const int pieces = (int)(end - x) + 1;
                if (by_sequence) p.joins[b] = make_int4(b, (int)x, pieces, 0);
                else if (pieces > 1) p.joins[x] = make_int4(b, (int)x, pieces, 0);
            }
            at += n;
        }
        __syncthreads();
        if (count <= 0) return;
    }

    const int tw_shift = p.tile_shift - 4, tw = 1 << tw_shift;          // warps that share a unit's tokens
    const int unit_cta = warp >> tw_shift, part = warp & (tw - 1);
    const int unit = blockIdx.y * p.units_cta + unit_cta;
    const int hk = unit / p.units_head, head0 = hk * p.group + (unit - hk * p.units_head) * 8;
    const int heads = min(8, (hk + 1) * p.group - head0);               // query heads of this unit
    const float cscale = __fdiv_rn(__fmul_rn(p.scale, kLog2e), *p.gk);

    const uint32_t ring = smem_u32(smem) + warp * (kStages * S::kStage);
    const uint8_t *kc = p.kc + hk * S::kCodes, *vc = p.vc + hk * S::kCodes;
    const uint8_t *ks = p.ks + hk * S::kScales, *vs = p.vs + hk * S::kScales;

    // ---- producer side: the tile at `ahead`; its pages are looked up one
    // step before its copies are issued
    Cursor ahead = start_sh;
    int ahead_left = count;
    int page = 0, offset = 0;
    bool there = false;
    auto lookup = [&]() {
        there = false;
        page = offset = 0;
        if (ahead_left > 0) {
            const int t = (ahead.tile << p.tile_shift) + part * kTile + (lane & 15);
            if (t < ahead.len) {
                const uint32_t entry = quotient((uint32_t)t, p.page_div);
                offset = t - (int)(entry * p.page_div.d);
                page = __ldg(p.block_table + (int64_t)ahead.b * p.table_stride + entry);
                there = true;
            }
            --ahead_left;
            ahead.next(p, ahead_left > 0);
        }
    };
    auto issue = [&](int stage) {
        bool ok = there;
        if (ok && (page < 0 || page >= p.n_pages)) {
            set_status(p.status, ST_INVALID_ARG);
            ok = false;
        }
        const int row = ok ? page * p.page_size + offset : -1;
        const uint32_t dst = ring + stage * S::kStage;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok) & 0xFFFFu;
        if (lane == 0) masks[warp][stage] = (int)mask;
        if (mask == 0u) return;                                         // no token: nothing will be read
#pragma unroll
        for (int i = 0; i < S::kChunks / 2; ++i) {
            const int n = i * 32 + lane, t = n / S::kChunks, ch = n % S::kChunks;
            const int r = __shfl_sync(0xFFFFFFFFu, row, t);
            const int64_t src = r < 0 ? 0 : (int64_t)r * p.row_codes + 16 * ch;
            const uint32_t to = dst + t * S::kCodes + 16 * swizzled<kD>(ch, t);
            copy_async<16>(to, kc + src, r >= 0);
            copy_async<16>(to + kTile * S::kCodes, vc + src, r >= 0);
        }
        {   // lanes 0 .. 15: K scales of token `lane`; 16 .. 31: V scales
            const int64_t src = row < 0 ? 0 : (int64_t)row * p.row_scales;
            copy_async<S::kScales>(dst + 2 * kTile * S::kCodes + lane * S::kScales,
                                   (lane < 16 ? ks : vs) + src, row >= 0);
        }
    };
    lookup();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        issue(s);
        copies_commit();
        lookup();
    }

    // ---- lane constants of the fragment reads
    const int tk = 4 * (g & 1) + ((g >> 1) ^ (3 * (g & 1)));            // token of MMA row g (row g + 8: + 8)
    const int ta = c, tb = 4 + (c ^ 3);                                 // tokens of MMA rows 2c, 2c + 1
    constexpr int kVWords = kD / 64;                                    // words of V codes a lane takes per token
    constexpr int kKWords = kD == 64 ? 2 : 4;
    uint32_t k_at[2], va_at, vb_at;
    if (kD == 64) {
        k_at[0] = k_at[1] = tk * S::kCodes + 8 * c;
        va_at = ta * S::kCodes + 4 * g;
        vb_at = tb * S::kCodes + 4 * g;
    } else if (kD == 128) {
        k_at[0] = k_at[1] = tk * S::kCodes + 16 * swizzled<kD>(c, tk);
        va_at = ta * S::kCodes + 16 * swizzled<kD>(g >> 1, ta) + 8 * (g & 1);
        vb_at = tb * S::kCodes + 16 * swizzled<kD>(g >> 1, tb) + 8 * (g & 1);
    } else {
        k_at[0] = tk * S::kCodes + 16 * swizzled<kD>(c, tk);
        k_at[1] = tk * S::kCodes + 16 * swizzled<kD>(c + 4, tk);
        va_at = ta * S::kCodes + 16 * swizzled<kD>(g, ta);
        vb_at = tb * S::kCodes + 16 * swizzled<kD>(g, tb);
    }
    va_at += kTile * S::kCodes;
    vb_at += kTile * S::kCodes;
    constexpr uint32_t kScaleAt = 2 * kTile * S::kCodes;
    const uint32_t ks_at = kScaleAt + tk * S::kScales + (kD == 64 ? c : 2 * c);
    const uint32_t vs_at = kScaleAt + kTile * S::kScales + (kD == 64 ? g >> 1 : kD == 128 ? g : 2 * g);

    // ---- consumer side
    Cursor now = start_sh;
    uint32_t qb[2 * S::kSteps];          // B fragments of the query
    float oacc[S::kSteps][4];
    float lsum[2] = {0.0f, 0.0f}, mp[2] = {kLowest, kLowest}, ck[2] = {0.0f, 0.0f};
    bool fresh = true, starts_here = now.tile == 0;

    for (int i = 0; i < count; ++i) {
        if (fresh) {
            fresh = false;
            // query of head g: lane c holds dims kD / 4 * c ... (kD = 256: 32c .. + 31 and 128 + 32c .. + 31)
            uint4 w[kD / 32];
            uint32_t amax = 0u;
            const uint16_t *q = p.q + (int64_t)now.b * p.qs_b + (int64_t)(head0 + g) * p.qs_h;
#pragma unroll
            for (int n = 0; n < kD / 32; ++n) {
                const int d = kD == 256 ? 32 * c + 8 * (n & 3) + 128 * (n >> 2) : (kD / 4) * c + 8 * n;
                w[n] = g < heads ? __ldg(reinterpret_cast<const uint4 *>(q + d)) : make_uint4(0u, 0u, 0u, 0u);
                amax = max_u16x2(amax, max_u16x2(max_u16x2(w[n].x & 0x7FFF7FFFu, w[n].y & 0x7FFF7FFFu),
                                                 max_u16x2(w[n].z & 0x7FFF7FFFu, w[n].w & 0x7FFF7FFFu)));
            }
            uint32_t e = max(amax & 0xFFFFu, amax >> 16) >> 7;          // exponent field of the largest value
            e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 1));
            e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 2));
            // times 2^(14 - (e - 127)), within FP32's exponents; a query of
            // zeros, infinities or NaN stays as it is
            const int up = e == 0u || e == 255u ? 0 : min(141 - (int)e, 126);
            const float mult = __uint_as_float((uint32_t)(127 + up) << 23);
            const float undo = __uint_as_float(up > 126 ? 0u : (uint32_t)(127 - up) << 23);
#pragma unroll
            for (int n = 0; n < kD / 32; ++n) {
                const uint32_t x[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    qb[4 * n + k] = f16x2_from_f32(__fmul_rn(bf16_lo(x[k]), mult), __fmul_rn(bf16_hi(x[k]), mult));
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
        const int stage = i % kStages;
        copies_wait<kStages - 2>();
        warp_sync();
        issue((i + kStages - 1) % kStages);
        copies_commit();
        lookup();
        const uint32_t at = ring + stage * S::kStage;
        const uint32_t mask = (uint32_t)masks[warp][stage];

        if (mask != 0u) {
            // ---- S = K q^T
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int half = 0; half < (kD == 256 ? 2 : 1); ++half) {
                uint32_t w0[kKWords], w1[kKWords];
                lds_words<kKWords>(at + k_at[half], w0);
                lds_words<kKWords>(at + k_at[half] + 8 * S::kCodes, w1);
                uint32_t s0[2], s1[2];                                  // scales of rows g, g + 8 as (s, s)
                if (kD == 64) {
                    const uint32_t x = f16x2_from_e4m3x2(lds8(at + ks_at) | (lds8(at + ks_at + 8 * S::kScales) << 8));
                    s0[0] = s0[1] = __byte_perm(x, x, 0x1010);
                    s1[0] = s1[1] = __byte_perm(x, x, 0x3232);
                } else {
                    const uint32_t x0 = f16x2_from_e4m3x2(lds16(at + ks_at + 8 * half));
                    const uint32_t x1 = f16x2_from_e4m3x2(lds16(at + ks_at + 8 * half + 8 * S::kScales));
                    s0[0] = __byte_perm(x0, x0, 0x1010);
                    s0[1] = __byte_perm(x0, x0, 0x3232);
                    s1[0] = __byte_perm(x1, x1, 0x1010);
                    s1[1] = __byte_perm(x1, x1, 0x3232);
                }
#pragma unroll
                for (int n = 0; n < kKWords; ++n) {                     // two MMA steps a word
                    uint32_t a[4], b[4];
                    f16x2_from_word(w0[n], a);
                    f16x2_from_word(w1[n], b);
                    const int blk = n / 2;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        a[k] = mul_f16x2(a[k], s0[blk]);
                        b[k] = mul_f16x2(b[k], s1[blk]);
                    }
                    const int step = 8 * half + 2 * n;
                    mma_f16(s, a[0], b[0], a[1], b[1], qb[2 * step], qb[2 * step + 1]);
                    mma_f16(s, a[2], b[2], a[3], b[3], qb[2 * step + 2], qb[2 * step + 3]);
                }
            }
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
                    if (r0) e[n] = __fmaf_rn(s[n], ck[n], -mn);
                    if (r1) e[n + 2] = __fmaf_rn(s[n + 2], ck[n], -mn);
                }
            }
            float w[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) w[n] = exp2_fast(e[n]);
            lsum[0] += w[0] + w[2];
            lsum[1] += w[1] + w[3];
            const uint32_t p0 = transpose_8x8(f16x2_from_f32(w[0], w[1]));
            const uint32_t p1 = transpose_8x8(f16x2_from_f32(w[2], w[3]));

            // ---- O^T += V^T P^T
            uint32_t wa[2][kVWords], wb[2][kVWords], sc[2][2];          // [rows 2c.. / 2c + 8 ..]
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                lds_words<kVWords>(at + va_at + 8 * n * S::kCodes, wa[n]);
                lds_words<kVWords>(at + vb_at + 8 * n * S::kCodes, wb[n]);
                if (kD == 256) {
                    const uint32_t a = lds16(at + vs_at + (ta + 8 * n) * S::kScales);
                    const uint32_t b = lds16(at + vs_at + (tb + 8 * n) * S::kScales);
                    sc[n][0] = f16x2_from_e4m3x2(__byte_perm(a, b, 0x0040));
                    sc[n][1] = f16x2_from_e4m3x2(__byte_perm(a, b, 0x0051));
                } else {
                    const uint32_t a = lds8(at + vs_at + (ta + 8 * n) * S::kScales);
                    const uint32_t b = lds8(at + vs_at + (tb + 8 * n) * S::kScales);
                    sc[n][0] = sc[n][1] = f16x2_from_e4m3x2(a | (b << 8));
                }
            }
#pragma unroll
            for (int n = 0; n < kVWords; ++n) {                         // four M-tiles a word
                uint32_t even[2][4], odd[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f16x2_from_word(nibbles(wa[h][n], wb[h][n] << 4), even[h]);
                    f16x2_from_word(nibbles(wa[h][n] >> 4, wb[h][n]), odd[h]);
                    const uint32_t x = sc[h][n / 2 < 2 ? (kD == 256 ? n / 2 : 0) : 0];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        even[h][k] = mul_f16x2(even[h][k], x);
                        odd[h][k] = mul_f16x2(odd[h][k], x);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_f16(oacc[4 * n + k], even[0][k], odd[0][k], even[1][k], odd[1][k], p0, p1);
            }
        }

        // ---- end of this CTA's part of a sequence
        const bool ends = now.tile + 1 == now.tiles;
        if (ends || i + 1 == count) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) lsum[n] += __shfl_xor_sync(0xFFFFFFFFu, lsum[n], off);
            float M[2] = {mp[0], mp[1]}, L[2] = {lsum[0], lsum[1]};
            if (tw > 1) {
                if (g == 0) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        ml[warp][2 * c + n][0] = mp[n];
                        ml[warp][2 * c + n][1] = lsum[n];
                    }
                }
                unit_barrier(1 + unit_cta, 32 * tw);
                const int w0 = warp - part;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    for (int w = 0; w < tw; ++w) M[n] = fmaxf(M[n], ml[w0 + w][2 * c + n][0]);
                    L[n] = 0.0f;
                    for (int w = 0; w < tw; ++w) L[n] += ml[w0 + w][2 * c + n][1] * exp2_fast(ml[w0 + w][2 * c + n][0] - M[n]);
                }
                const float f0 = exp2_fast(mp[0] - M[0]), f1 = exp2_fast(mp[1] - M[1]);
                float *mine = reinterpret_cast<float *>(smem + S::kRing) + warp * (8 * kD) + lane;
#pragma unroll
                for (int j = 0; j < S::kSteps; ++j)
#pragma unroll
                    for (int n = 0; n < 4; ++n) mine[(4 * j + n) * 32] = oacc[j][n] * (n & 1 ? f1 : f0);
                unit_barrier(1 + unit_cta, 32 * tw);
            }
            const bool whole = ends && starts_here;
            const float *from = reinterpret_cast<const float *>(smem + S::kRing) + (warp - part) * (8 * kD) + lane;
            const int64_t slot = ((int64_t)(2 * blockIdx.x + (starts_here ? 1 : 0)) * gridDim.y + blockIdx.y) * p.units_cta + unit_cta;
            float *part_o = p.part_o + slot * (8 * kD) + lane;
            const float inv_gv = *p.gv;
#pragma unroll
            for (int j = 0; j < S::kSteps; ++j) {
                if ((j & (tw - 1)) != part) continue;
                float r[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    r[n] = oacc[j][n];
                    if (tw > 1) {
                        r[n] = 0.0f;
                        for (int w = 0; w < tw; ++w) r[n] += from[w * (8 * kD) + (4 * j + n) * 32];
                    }
                }
                if (whole) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        if (2 * c + n < heads) {
                            const bool none = L[n] == 0.0f;
                            const float lo = none ? 0.0f : __fdiv_rn(__fdiv_rn(r[n], L[n]), inv_gv);
                            const float hi = none ? 0.0f : __fdiv_rn(__fdiv_rn(r[n + 2], L[n]), inv_gv);
                            *reinterpret_cast<uint32_t *>(p.o + (int64_t)now.b * p.os_b + (int64_t)(head0 + 2 * c + n) * p.os_h +
                                                          (kD / 8) * g + 2 * j) = bf16x2_from_f32(lo, hi);
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n) part_o[(4 * j + n) * 32] = r[n];
                }
            }
            if (part == 0 && g == 0) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    if (whole) {
                        if (p.lse != nullptr && 2 * c + n < heads)
                            p.lse[(int64_t)now.b * p.heads_q + head0 + 2 * c + n] =
                                L[n] == 0.0f ? -__int_as_float(0x7F800000) : (M[n] + log2f(L[n])) * kLn2;
                    } else {
                        p.part_ml[slot * 8 + 2 * c + n] = make_float2(M[n], L[n]);
                    }
                }
            }
            fresh = true;
            starts_here = true;
        }
        now.next(p, i + 1 < count);
    }
}

// Joins the parts of the sequences that were cut: one sequence (or the one
// that is cut at the end of a range) per blockIdx.x, M-tiles of O^T (128
// values) in turn per blockIdx.y.  The parts of a tile are dealt to 8 groups
// of 32 threads, whose sums are added in order.
__global__ void __launch_bounds__(256) k_paged_combine(PagedAttnParams p, int dim, int ranges_x, int blocks_y) {
    __shared__ float weight[kPagedMaxRanges][8];
    __shared__ float red[32][8];
    __shared__ float4 sums[8][32];
    __shared__ float M_sh[8], L_sh[8];
    grid_dependency_wait();
    const int4 join = p.joins[blockIdx.x];
    const int b = join.x, x0 = join.y, pieces = join.z;
    if (pieces <= 1) return;
    const int tid = threadIdx.x, tiles = dim / 16, units = blocks_y * p.units_cta;
    const int total = units * tiles;
    int done = -1;
    for (int item = blockIdx.y; item < total; item += gridDim.y) {
        const int unit = item / tiles, j = item - unit * tiles;
        const int hk = unit / p.units_head, head0 = hk * p.group + (unit - hk * p.units_head) * 8;
        const int heads = min(8, (hk + 1) * p.group - head0);
        // piece n: the first lies in the second slot of its CTA, the others in the first
        auto slot = [&](int n) { return (int64_t)(2 * (x0 + n) + (n == 0 ? 1 : 0)) * units + unit; };
        if (unit != done) {
            done = unit;
            const int h = tid & 7, group = tid >> 3;
            float m = kLowest;
            for (int n = group; n < pieces; n += 32) m = fmaxf(m, p.part_ml[slot(n) * 8 + h].x);
            __syncthreads();
            red[group][h] = m;
            __syncthreads();
            if (tid < 8) {
                for (int n = 1; n < 32; ++n) m = fmaxf(m, red[n][tid]);
                M_sh[tid] = m;
            }
            __syncthreads();
            m = M_sh[h];
            float l = 0.0f;
            for (int n = group; n < pieces; n += 32) {
                const float2 v = p.part_ml[slot(n) * 8 + h];
                const float w = exp2_fast(v.x - m);
                weight[n][h] = w;
                l += w * v.y;
            }
            red[group][h] = l;
            __syncthreads();
            if (tid < 8) {
                l = 0.0f;
                for (int n = 0; n < 32; ++n) l += red[n][tid];
                L_sh[tid] = l;
                if (j == 0 && p.lse != nullptr && tid < heads)
                    p.lse[(int64_t)b * p.heads_q + head0 + tid] =
                        l == 0.0f ? -__int_as_float(0x7F800000) : (M_sh[tid] + log2f(l)) * kLn2;
            }
            __syncthreads();
        }
        // 128 values: [n = 0 .. 3][lane], four neighbouring lanes (c = 0 .. 3)
        // a thread: heads 0, 2, 4, 6 (n even) or 1, 3, 5, 7 (n odd)
        const int v = tid & 31, group = tid >> 5, n4 = v >> 3, odd = n4 & 1;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int n = group; n < pieces; n += 8) {
            const float4 o = *reinterpret_cast<const float4 *>(p.part_o + slot(n) * (8 * dim) + 128 * j + 4 * v);
            a.x += o.x * weight[n][odd];
            a.y += o.y * weight[n][2 + odd];
            a.z += o.z * weight[n][4 + odd];
            a.w += o.w * weight[n][6 + odd];
        }
        sums[group][v] = a;
        __syncthreads();
        if (tid < 64) {
            // one head and lane row g: values n = e and n = e + 2 (dims 2j, 2j + 1)
            const int h = tid & 7, gg = tid >> 3, e = h & 1, cc = h >> 1;
            const float *f = reinterpret_cast<const float *>(&sums[0][0]);
            float lo = 0.0f, hi = 0.0f;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                lo += f[n * 128 + e * 32 + gg * 4 + cc];
                hi += f[n * 128 + (e + 2) * 32 + gg * 4 + cc];
            }
            if (h < heads) {
                const float L = L_sh[h], gv = *p.gv;
                lo = L == 0.0f ? 0.0f : __fdiv_rn(__fdiv_rn(lo, L), gv);
                hi = L == 0.0f ? 0.0f : __fdiv_rn(__fdiv_rn(hi, L), gv);
                *reinterpret_cast<uint32_t *>(p.o + (int64_t)b * p.os_b + (int64_t)(head0 + h) * p.os_h +
                                              (dim / 8) * gg + 2 * j) = bf16x2_from_f32(lo, hi);
            }
        }
        __syncthreads();
    }
}

namespace {

template <int kD>
cudaError_t launch_main(const PagedAttnParams &p, dim3 grid, cudaStream_t s) {
    static std::atomic<uint64_t> ready{0};               // devices (below 64) with the shared memory allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!((ready.load(std::memory_order_relaxed) >> dev) & 1u)) {
        e = cudaFuncSetAttribute(k_paged_attention<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<kD>::kSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    k_paged_attention<kD><<<grid, kWarps * 32, Shape<kD>::kSmem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnParams &p, int dim, const PagedPlan &plan, cudaStream_t s) {
    const dim3 grid((unsigned)plan.ranges, (unsigned)plan.blocks);
    cudaError_t e = dim == 64 ? launch_main<64>(p, grid, s)
                    : dim == 128 ? launch_main<128>(p, grid, s)
                                 : launch_main<256>(p, grid, s);
    if (e != cudaSuccess) return e;
    // the sequences that can be cut, and CTAs for about one wave of the device
    const int joins = std::min(p.sequences, plan.ranges);
    const int tiles = plan.blocks * p.units_cta * (dim / 16);
    const int per = std::max(1, (int)(((int64_t)joins * tiles + 1183) / 1184));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)joins, (unsigned)((tiles + per - 1) / per));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_paged_combine, p, dim, plan.ranges, plan.blocks);
}

}  // namespace nvfp4
