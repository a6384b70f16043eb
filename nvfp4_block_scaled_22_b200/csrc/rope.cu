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
// in 47.8 us, 6.4 TB/s; 4099 x 40 x 128 interleaved, half rotated, in 13.9 us).
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

// Where an item lies: a token's position row (-1: left alone), and the item's
// piece of a head.
struct RopeItem {
    int64_t row;
    const uint16_t *x;
    uint16_t *y;
    uint32_t piece;
};

__device__ __forceinline__ RopeItem rope_item(const RopeParams &p, uint32_t item) {
    const uint32_t t = quotient(item, p.per_token), in_t = item - t * p.per_token.d;
    const uint32_t h = quotient(in_t, p.per_head);
    RopeItem r;
    r.row = rope_row(p.positions[t], p.table_rows, p.status);
    r.x = p.x + (int64_t)t * p.xs_t + (int64_t)h * p.xs_h;
    r.y = p.y + (int64_t)t * p.ys_t + (int64_t)h * p.ys_h;
    r.piece = in_t - h * p.per_head.d;
    return r;
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

// Interleaved layout, 8 values (4 pairs) an item.
__global__ void __launch_bounds__(256) k_rope_interleaved(RopeParams p) {
    const uint32_t base = blockIdx.x * (256u * kRopeItems) + threadIdx.x;
    RopeItem it[kRopeItems];
    uint4 a[kRopeItems];
#pragma unroll
    for (int n = 0; n < kRopeItems; ++n) {
        it[n].row = -1;
        if (base + 256u * n < p.items) it[n] = rope_item(p, base + 256u * n);
        if (it[n].row >= 0) a[n] = *reinterpret_cast<const uint4 *>(it[n].x + 8 * it[n].piece);
    }
#pragma unroll
    for (int n = 0; n < kRopeItems; ++n) {
        if (it[n].row < 0) continue;
        uint4 y = a[n];
        if (4 * it[n].piece < (uint32_t)p.pairs) {
            const float4 *cs = reinterpret_cast<const float4 *>(p.table + it[n].row * p.pairs + 4 * it[n].piece);
            const float4 f0 = __ldg(cs), f1 = __ldg(cs + 1);
            float lo, hi;
            rotate(bf16_lo(a[n].x), bf16_hi(a[n].x), f0.x, p.sign * f0.y, lo, hi);
            y.x = bf16x2_from_f32(lo, hi);
            rotate(bf16_lo(a[n].y), bf16_hi(a[n].y), f0.z, p.sign * f0.w, lo, hi);
            y.y = bf16x2_from_f32(lo, hi);
            rotate(bf16_lo(a[n].z), bf16_hi(a[n].z), f1.x, p.sign * f1.y, lo, hi);
            y.z = bf16x2_from_f32(lo, hi);
            rotate(bf16_lo(a[n].w), bf16_hi(a[n].w), f1.z, p.sign * f1.w, lo, hi);
            y.w = bf16x2_from_f32(lo, hi);
        }
        *reinterpret_cast<uint4 *>(it[n].y + 8 * it[n].piece) = y;
    }
}

// Any pair count, head size and alignment: one pair an item, then one value
// an item behind the rotated part.  Taken where the pieces above do not come
// out whole or 16-byte aligned.
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
