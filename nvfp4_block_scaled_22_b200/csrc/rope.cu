// Rotary positions: the first 2 * pairs values of each head are rotated in
// pairs by angles position * f_i,
//   y1 = x1 c - x2 s,   y2 = x2 c + x1 s,   (c, s) = table[position][i],
// pair i being values (i, i + pairs) ("half") or (2i, 2i + 1)
// ("interleaved"); the rest of the head is copied.  The inverse (s -> -s) is
// the transposed map, so it turns the gradient of y into the gradient of x.
// Each product and the sum is one FP32 operation rounded to nearest, then
// BF16: the same bits for the same table, whatever the kernel variant.
//
// The table holds (cos, sin) in FP32, rounded once from angles formed in
// FP64: a position times a frequency needs about 24 + 20 bits before it is
// reduced to a turn, so an FP32 angle is off by 0.06 at position 2^20.
//
// Bound by memory: 4 bytes a value against 3 FP32 operations (8192 x 72 x 128
// in 47.6 us, 6.4 TB/s; interleaved 46.4; 4099 x 40 x 128 interleaved, half
// rotated, in 14.5 us).  The table, made once, is bound by its arithmetic: 125
// instructions an entry of FP64 sine and cosine and a division (131072
// positions x 64 pairs in 36.4 us, 80 % of the issue slots; its bytes: 10.2 us).
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"
#include "paged.cuh"

namespace nvfp4 {

__global__ void __launch_bounds__(256) k_rope_table(const double *__restrict__ inv_freq, int32_t pairs,
                                                    int64_t first, int64_t n, double magnitude,
                                                    float2 *__restrict__ table) {
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
        const int64_t row = e / pairs;
        double s, c;
        sincos((double)(first + row) * inv_freq[e - row * pairs], &s, &c);
        table[e] = make_float2((float)(c * magnitude), (float)(s * magnitude));
    }
}

// Half layout: an item is 8 pairs (two 16-byte pieces) of kRopeHeads heads
// of a token, which share 64 bytes of the table; then the 8-value pieces
// behind the rotated part.  With an item a head, the table took twice the
// L1 traffic of the values (55.6 us against 47.8 at 8192 x 72 x 128).  All heads
// are loaded before one is stored (y may be x, so that the compiler would
// not).
__global__ void __launch_bounds__(256) k_rope_half(RopeParams p) {
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    if (item >= p.items) return;
    const uint32_t t = quotient(item, p.per_token), in_t = item - t * p.per_token.d;
    const uint32_t group = quotient(in_t, p.per_head), piece = in_t - group * p.per_head.d;
    const uint32_t pair_items = (uint32_t)p.pairs >> 3;
    const int h0 = (int)group * kRopeHeads;
    const bool turned = piece < pair_items;
    const uint32_t at = turned ? 8 * piece : 2 * p.pairs + 8 * (piece - pair_items);
    const uint16_t *x = p.x + (int64_t)t * p.xs_t + (int64_t)h0 * p.xs_h + at;
    uint16_t *y = p.y + (int64_t)t * p.ys_t + (int64_t)h0 * p.ys_h + at;
    const int32_t position = p.positions[t];
    uint4 a[kRopeHeads], b[kRopeHeads];
#pragma unroll
    for (int h = 0; h < kRopeHeads; ++h) {
        a[h] = b[h] = make_uint4(0u, 0u, 0u, 0u);
        if (h0 + h < p.heads) {
            a[h] = *reinterpret_cast<const uint4 *>(x + (int64_t)h * p.xs_h);
            if (turned) b[h] = *reinterpret_cast<const uint4 *>(x + (int64_t)h * p.xs_h + p.pairs);
        }
    }
    const int64_t row = rope_row(position, p.table_rows, p.status);
    if (row < 0) return;
    if (turned) {
        const float4 *cs = reinterpret_cast<const float4 *>(p.table + row * p.pairs + 8 * piece);
        float4 f[4];                                     // cos, sin of two pairs
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __ldg(cs + i);
            f[i].y *= p.sign;
            f[i].w *= p.sign;
        }
#pragma unroll
        for (int h = 0; h < kRopeHeads; ++h) {
            const uint32_t aw[4] = {a[h].x, a[h].y, a[h].z, a[h].w}, bw[4] = {b[h].x, b[h].y, b[h].z, b[h].w};
            uint32_t ya[4], yb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo1, lo2, hi1, hi2;
                rotate(bf16_lo(aw[i]), bf16_lo(bw[i]), f[i].x, f[i].y, lo1, lo2);
                rotate(bf16_hi(aw[i]), bf16_hi(bw[i]), f[i].z, f[i].w, hi1, hi2);
                ya[i] = bf16x2_from_f32(lo1, hi1);
                yb[i] = bf16x2_from_f32(lo2, hi2);
            }
            if (h0 + h < p.heads) {
                *reinterpret_cast<uint4 *>(y + (int64_t)h * p.ys_h) = make_uint4(ya[0], ya[1], ya[2], ya[3]);
                *reinterpret_cast<uint4 *>(y + (int64_t)h * p.ys_h + p.pairs) = make_uint4(yb[0], yb[1], yb[2], yb[3]);
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < kRopeHeads; ++h)
            if (h0 + h < p.heads) *reinterpret_cast<uint4 *>(y + (int64_t)h * p.ys_h) = a[h];
    }
}

// Values o .. o + 7 of the two 16-byte pieces (a, b), in bits.
__device__ __forceinline__ uint4 window(const uint4 &a, const uint4 &b, uint32_t o) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (o & 4u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (o & 2u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (o & 1u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Half layout with any pair count, y apart from x: an item is a 16-byte piece
// of kRopeHeads heads of the output, whose partners lie in two neighbouring
// pieces of x; each value is rotated by itself, x c + partner (-s, or s in
// the second half), the same steps.  The pieces that a border of the rotated
// part cuts go value by value, as items behind a token's others: among them,
// each warp had waited for a few such lanes (8192 x 72 x 128 with 63 pairs: 175
// us, so 95; with 31 pairs 85, with one 55; pair by pair in k_rope_any 177, 260
// and 306.  8 heads an item, fewer warps: 138 with 63 pairs).
__global__ void __launch_bounds__(256) k_rope_half_pieces(RopeParams p) {
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    if (item >= p.items) return;
    const uint32_t pairs = (uint32_t)p.pairs;
    const uint32_t t = quotient(item, p.per_token), in_t = item - t * p.per_token.d;
    const bool cut = in_t >= p.uncut;
    const uint32_t border = (in_t - p.uncut) & (p.cuts - 1);            // of a cut item
    const uint32_t group = cut ? (in_t - p.uncut) >> (p.cuts - 1) : quotient(in_t, p.per_head);
    // the borders are at pairs (pairs % 8 != 0 here) and 2 * pairs (in the same piece, or between two, with one cut)
    const uint32_t at = cut ? ((border == 0u ? pairs : 2 * pairs) & ~7u) : 8 * (in_t - group * p.per_head.d);
    const bool first = at + 8 <= pairs, second = at >= pairs && at + 8 <= 2 * pairs;
    if (!cut && !first && !second && at < 2 * pairs) return;
    const int h0 = (int)group * kRopeHeads;
    const uint16_t *x = p.x + (int64_t)t * p.xs_t + (int64_t)h0 * p.xs_h;
    uint16_t *y = p.y + (int64_t)t * p.ys_t + (int64_t)h0 * p.ys_h + at;
    const int64_t row = rope_row(p.positions[t], p.table_rows, p.status);
    if (row < 0) return;
    const float2 *table = p.table + row * pairs;
    uint4 a[kRopeHeads];
#pragma unroll
    for (int h = 0; h < kRopeHeads; ++h)
        a[h] = h0 + h < p.heads ? __ldg(reinterpret_cast<const uint4 *>(x + (int64_t)h * p.xs_h + at)) : make_uint4(0u, 0u, 0u, 0u);
    if (!cut && (first || second)) {
        const uint32_t from = first ? at + pairs : at - pairs, o = from & 7u;
        uint4 b[kRopeHeads];
#pragma unroll
        for (int h = 0; h < kRopeHeads; ++h) {
            if (h0 + h < p.heads) {
                const uint4 *q = reinterpret_cast<const uint4 *>(x + (int64_t)h * p.xs_h + (from - o));
                const uint4 b0 = __ldg(q);
                b[h] = o != 0u ? window(b0, __ldg(q + 1), o) : b0;
            }
        }
        const float2 *cs = table + (first ? at : at - pairs);
        const float sign = first ? -p.sign : p.sign;
        float2 f[8];
        if ((pairs & 1u) == 0u) {                       // 16-byte aligned rows, and half of the loads
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 two = __ldg(reinterpret_cast<const float4 *>(cs) + i);
                f[2 * i] = make_float2(two.x, two.y);
                f[2 * i + 1] = make_float2(two.z, two.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __ldg(cs + i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i].y *= sign;
#pragma unroll
        for (int h = 0; h < kRopeHeads; ++h) {
            if (h0 + h < p.heads) {
                const uint32_t aw[4] = {a[h].x, a[h].y, a[h].z, a[h].w}, bw[4] = {b[h].x, b[h].y, b[h].z, b[h].w};
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = bf16x2_from_f32(
                        __fadd_rn(__fmul_rn(bf16_lo(aw[i]), f[2 * i].x), __fmul_rn(bf16_lo(bw[i]), f[2 * i].y)),
                        __fadd_rn(__fmul_rn(bf16_hi(aw[i]), f[2 * i + 1].x), __fmul_rn(bf16_hi(bw[i]), f[2 * i + 1].y)));
                a[h] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    } else if (cut) {
#pragma unroll
        for (uint32_t n = 0; n < 8; ++n) {
            const uint32_t i = at + n;
            if (i < 2 * pairs) {
                const uint32_t other = i < pairs ? i + pairs : i - pairs;
                const float2 f = __ldg(table + min(i, other));
                const float s = i < pairs ? -p.sign * f.y : p.sign * f.y;
#pragma unroll
                for (int h = 0; h < kRopeHeads; ++h) {
                    if (h0 + h < p.heads) {
                        uint32_t w[4] = {a[h].x, a[h].y, a[h].z, a[h].w};
                        const float v = (n & 1u) ? bf16_hi(w[n >> 1]) : bf16_lo(w[n >> 1]);
                        const float r = __fadd_rn(__fmul_rn(v, f.x), __fmul_rn(bf16_lo(__ldg(x + (int64_t)h * p.xs_h + other)), s));
                        const uint32_t bits = bf16x2_from_f32(r, r);
                        w[n >> 1] = (n & 1u) ? (w[n >> 1] & 0xFFFFu) | (bits & 0xFFFF0000u) : (w[n >> 1] & 0xFFFF0000u) | (bits & 0xFFFFu);
                        a[h] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int h = 0; h < kRopeHeads; ++h)
        if (h0 + h < p.heads) *reinterpret_cast<uint4 *>(y + (int64_t)h * p.ys_h) = a[h];
}

// Interleaved layout: an item is 8 values (4 pairs) of kRopeHeads heads of a
// token, which share 32 bytes of the table; kWhole: pairs % 4 == 0.  (An item
// a head took the table once a head: 8192 x 72 x 128 in 51.0 us, so 46.4; with
// 63 pairs 59.5 and 47.3.)
template <bool kWhole>
__device__ __forceinline__ void rope_interleaved(const RopeParams &p) {
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    if (item >= p.items) return;
    const uint32_t t = quotient(item, p.per_token), in_t = item - t * p.per_token.d;
    const uint32_t group = quotient(in_t, p.per_head), piece = in_t - group * p.per_head.d;
    const int h0 = (int)group * kRopeHeads;
    const uint16_t *x = p.x + (int64_t)t * p.xs_t + (int64_t)h0 * p.xs_h + 8 * piece;
    uint16_t *y = p.y + (int64_t)t * p.ys_t + (int64_t)h0 * p.ys_h + 8 * piece;
    const int32_t position = p.positions[t];
    uint4 a[kRopeHeads];
#pragma unroll
    for (int h = 0; h < kRopeHeads; ++h)
        a[h] = h0 + h < p.heads ? *reinterpret_cast<const uint4 *>(x + (int64_t)h * p.xs_h) : make_uint4(0u, 0u, 0u, 0u);
    const int64_t row = rope_row(position, p.table_rows, p.status);
    if (row < 0) return;
    const uint32_t pair = 4 * piece;
    float2 f[4];
    if (pair < (uint32_t)p.pairs) {
        const float2 *cs = p.table + row * p.pairs + pair;
        if (kWhole) {
            const float4 f0 = __ldg(reinterpret_cast<const float4 *>(cs)), f1 = __ldg(reinterpret_cast<const float4 *>(cs) + 1);
            f[0] = make_float2(f0.x, f0.y), f[1] = make_float2(f0.z, f0.w);
            f[2] = make_float2(f1.x, f1.y), f[3] = make_float2(f1.z, f1.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = pair + i < (uint32_t)p.pairs ? __ldg(cs + i) : make_float2(0.0f, 0.0f);
        }
    }
#pragma unroll
    for (int h = 0; h < kRopeHeads; ++h) {
        if (h0 + h >= p.heads) continue;
        uint32_t w[4] = {a[h].x, a[h].y, a[h].z, a[h].w};
        if (pair < (uint32_t)p.pairs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                rotate(bf16_lo(w[i]), bf16_hi(w[i]), f[i].x, p.sign * f[i].y, lo, hi);
                if (kWhole || pair + i < (uint32_t)p.pairs) w[i] = bf16x2_from_f32(lo, hi);
            }
        }
        *reinterpret_cast<uint4 *>(y + (int64_t)h * p.ys_h) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__global__ void __launch_bounds__(256) k_rope_interleaved(RopeParams p) { rope_interleaved<true>(p); }
__global__ void __launch_bounds__(256) k_rope_interleaved_pieces(RopeParams p) { rope_interleaved<false>(p); }

// Any pair count, head size and alignment: one pair an item, then one value
// an item behind the rotated part.  Taken where heads are not 16-byte aligned
// pieces, and for the half layout in place with pairs % 8 != 0 (the pieces'
// partners would have been overwritten).
__global__ void __launch_bounds__(256) k_rope_any(RopeParams p, int interleaved, int with_rest) {
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    if (item >= p.items) return;
    const uint32_t t = quotient(item, p.per_token), in_t = item - t * p.per_token.d;
    const uint32_t h = quotient(in_t, p.per_head), c = in_t - h * p.per_head.d;
    const int64_t pos = rope_row(p.positions[t], p.table_rows, p.status);
    if (pos < 0) return;
    const uint16_t *x = p.x + (int64_t)t * p.xs_t + (int64_t)h * p.xs_h;
    uint16_t *y = p.y + (int64_t)t * p.ys_t + (int64_t)h * p.ys_h;
    if (c < (uint32_t)p.pairs) {
        const uint32_t i1 = interleaved ? 2 * c : c, i2 = interleaved ? 2 * c + 1 : c + p.pairs;
        const float2 f = p.table[pos * p.pairs + c];
        float y1, y2;
        rotate(bf16_lo(x[i1]), bf16_lo(x[i2]), f.x, p.sign * f.y, y1, y2);
        const uint32_t w = bf16x2_from_f32(y1, y2);
        y[i1] = (uint16_t)w;
        y[i2] = (uint16_t)(w >> 16);
    } else if (with_rest) {
        y[c + p.pairs] = x[c + p.pairs];
    }
}

}  // namespace nvfp4
