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
// Bound by memory: 4 bytes a value against 3 FP32 operations.
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

// Half layout, 8 pairs an item (two 16-byte pieces of a head, one table
// row's 64 bytes), then the 8-value pieces behind the rotated part.
__global__ void __launch_bounds__(256) k_rope_half(RopeParams p) {
    const uint32_t base = blockIdx.x * (256u * kRopeItems) + threadIdx.x;
    const uint32_t pair_items = (uint32_t)p.pairs >> 3;
#pragma unroll
    for (int n = 0; n < kRopeItems; ++n) {
        const uint32_t item = base + 256u * n;
        if (item >= p.items) return;
        const uint32_t t = quotient(item, p.per_token), in_t = item - t * p.per_token.d;
        const uint32_t h = quotient(in_t, p.per_head), c = in_t - h * p.per_head.d;
        const int64_t pos = rope_row(p.positions[t], p.table_rows, p.status);
        if (pos < 0) continue;
        const uint16_t *x = p.x + (int64_t)t * p.xs_t + (int64_t)h * p.xs_h;
        uint16_t *y = p.y + (int64_t)t * p.ys_t + (int64_t)h * p.ys_h;
        if (c < pair_items) {
            const uint4 a = *reinterpret_cast<const uint4 *>(x + 8 * c);
            const uint4 b = *reinterpret_cast<const uint4 *>(x + p.pairs + 8 * c);
            const float4 *cs = reinterpret_cast<const float4 *>(p.table + pos * p.pairs + 8 * c);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
            uint32_t ya[4], yb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = __ldg(cs + i);          // cos, sin of two pairs
                float lo1, lo2, hi1, hi2;
                rotate(bf16_lo(aw[i]), bf16_lo(bw[i]), f.x, p.sign * f.y, lo1, lo2);
                rotate(bf16_hi(aw[i]), bf16_hi(bw[i]), f.z, p.sign * f.w, hi1, hi2);
                ya[i] = bf16x2_from_f32(lo1, hi1);
                yb[i] = bf16x2_from_f32(lo2, hi2);
            }
            *reinterpret_cast<uint4 *>(y + 8 * c) = make_uint4(ya[0], ya[1], ya[2], ya[3]);
            *reinterpret_cast<uint4 *>(y + p.pairs + 8 * c) = make_uint4(yb[0], yb[1], yb[2], yb[3]);
        } else {
            const uint32_t at = 2 * p.pairs + 8 * (c - pair_items);
            *reinterpret_cast<uint4 *>(y + at) = *reinterpret_cast<const uint4 *>(x + at);
        }
    }
}

// Interleaved layout, 8 values (4 pairs) an item.
__global__ void __launch_bounds__(256) k_rope_interleaved(RopeParams p) {
    const uint32_t base = blockIdx.x * (256u * kRopeItems) + threadIdx.x;
#pragma unroll
    for (int n = 0; n < kRopeItems; ++n) {
        const uint32_t item = base + 256u * n;
        if (item >= p.items) return;
        const uint32_t t = quotient(item, p.per_token), in_t = item - t * p.per_token.d;
        const uint32_t h = quotient(in_t, p.per_head), c = in_t - h * p.per_head.d;
        const int64_t pos = rope_row(p.positions[t], p.table_rows, p.status);
        if (pos < 0) continue;
        const uint4 a = *reinterpret_cast<const uint4 *>(p.x + (int64_t)t * p.xs_t + (int64_t)h * p.xs_h + 8 * c);
        uint4 *y = reinterpret_cast<uint4 *>(p.y + (int64_t)t * p.ys_t + (int64_t)h * p.ys_h + 8 * c);
        if (4 * c < (uint32_t)p.pairs) {
            const float4 *cs = reinterpret_cast<const float4 *>(p.table + pos * p.pairs + 4 * c);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = __ldg(cs + (i >> 1));
                float y1, y2;
                rotate(bf16_lo(aw[i]), bf16_hi(aw[i]), (i & 1) ? f.z : f.x,
                       p.sign * ((i & 1) ? f.w : f.y), y1, y2);
                o[i] = bf16x2_from_f32(y1, y2);
            }
            *y = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
            *y = a;
        }
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
