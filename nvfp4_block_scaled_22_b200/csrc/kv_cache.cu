// The paged NVFP4 KV cache: a pool of token rows (an nvfp4_tensor with the
// LINEAR scale layout), written row by row as tokens arrive and read back
// row by row.
//
// k_kv_write*: row slots[t] of the K pool receives the NVFP4 of k[t] (rotated
// first when a table is given, and rounded to BF16 as k_rope_* rounds it),
// row slots[t] of the V pool that of v[t], under the pools' own tensor
// scales; per 16-value block the steps of nvfp4_quantize with a supplied g,
//   s = e4m3(RN(RN(amax / 6) g)),  e = s ? RN(g / s) : 0,
//   code = e2m1(RN(x e)),
// so the bytes are those of nvfp4_quantize of the (rotated) rows.  One thread
// takes one block: 32 bytes in, 8 + 1 bytes out; neighbouring threads take
// neighbouring blocks of a row.
// k_kv_read: y = bf16(RN(e2m1 RN(s / g))), the steps of nvfp4_dequantize.
//
// Both are bound by memory (2.56 bytes a value; two IEEE divisions a block
// are 2 to 3 instructions a value of the 14 that fit beside the copy).
#include <cstdint>
#include <cuda_runtime.h>

#include "encode_common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

// The rotated block of 16 values of a key: `own` holds values 16b .. 16b + 15
// of the head, x is the head.
// kWhole: half layout and pairs % 16 == 0, so that the partners of a block
// are one block; otherwise the partners are fetched one by one.
template <bool kWhole>
__device__ __forceinline__ void rotate_block(uint4 &a, uint4 &b, const uint16_t *x, int blk,
                                             const KvWriteParams &p, int64_t pos) {
    const int j0 = 16 * blk;
    if (j0 >= 2 * p.pairs) return;
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const float2 *row = p.table + pos * p.pairs;
    if (kWhole) {
        const bool first = j0 < p.pairs;
        const uint4 *partner = reinterpret_cast<const uint4 *>(x + (first ? j0 + p.pairs : j0 - p.pairs));
        const uint4 c = partner[0], d = partner[1];
        const uint32_t u[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
        const float4 *cs = reinterpret_cast<const float4 *>(row + (first ? j0 : j0 - p.pairs));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 f = __ldg(cs + i);
            // first: y1 of (own, partner); second: y2 of (partner, own)
            const float lo = first ? __fsub_rn(__fmul_rn(bf16_lo(w[i]), f.x), __fmul_rn(bf16_lo(u[i]), f.y))
                                   : __fadd_rn(__fmul_rn(bf16_lo(w[i]), f.x), __fmul_rn(bf16_lo(u[i]), f.y));
            const float hi = first ? __fsub_rn(__fmul_rn(bf16_hi(w[i]), f.z), __fmul_rn(bf16_hi(u[i]), f.w))
                                   : __fadd_rn(__fmul_rn(bf16_hi(w[i]), f.z), __fmul_rn(bf16_hi(u[i]), f.w));
            w[i] = bf16x2_from_f32(lo, hi);
        }
    } else if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int pair = (j0 >> 1) + i;
            if (pair < p.pairs) {
                const float2 f = __ldg(row + pair);
                float y1, y2;
                rotate(bf16_lo(w[i]), bf16_hi(w[i]), f.x, f.y, y1, y2);
                w[i] = bf16x2_from_f32(y1, y2);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float y[2] = {bf16_lo(w[i]), bf16_hi(w[i])};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = j0 + 2 * i + e;
                if (j < 2 * p.pairs) {
                    const bool first = j < p.pairs;
                    const int pair = first ? j : j - p.pairs;
                    const float2 f = __ldg(row + pair);
                    const float other = bf16_lo(x[first ? j + p.pairs : pair]);
                    y[e] = first ? __fsub_rn(__fmul_rn(y[e], f.x), __fmul_rn(other, f.y))
                                 : __fadd_rn(__fmul_rn(y[e], f.x), __fmul_rn(other, f.y));
                }
            }
            w[i] = bf16x2_from_f32(y[0], y[1]);
        }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

// kRope: 0 no rotation, 1 whole partner blocks, 2 any.
template <int kRope>
__device__ __forceinline__ void kv_write_body(const KvWriteParams &p) {
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    if (item >= p.items) return;
    const uint32_t t = quotient(item, p.per_token);
    uint32_t blk = item - t * p.per_token.d;               // block of the K row, then of the V row
    const int64_t row = pool_row(p.slots[t], p.pool_rows, p.status);
    if (row < 0) return;
    const uint32_t row_blocks = p.per_token.d >> 1;
    const bool is_v = blk >= row_blocks;
    if (is_v) blk -= row_blocks;
    const uint32_t h = quotient(blk, p.per_head), b = blk - h * p.per_head.d;
    int64_t pos = 0;
    if (kRope != 0) {
        // a token whose position has no table row is not written at all
        pos = rope_row(p.positions[t], p.table_rows, p.status);
        if (pos < 0) return;
    }
    const uint16_t *x = is_v ? p.v + (int64_t)t * p.vs_t + (int64_t)h * p.vs_h
                             : p.k + (int64_t)t * p.ks_t + (int64_t)h * p.ks_h;
    uint4 w0 = reinterpret_cast<const uint4 *>(x + 16 * b)[0];
    uint4 w1 = reinterpret_cast<const uint4 *>(x + 16 * b)[1];
    if (kRope != 0 && !is_v) rotate_block<kRope == 1>(w0, w1, x, (int)b, p, pos);
    const uint32_t bits = block_amax_bits(w0, w1);
    if (bits > 0x7F7FFFFFu) set_status(p.status, ST_NONFINITE);
    const float g = is_v ? *p.gv : *p.gk;
    const uint32_t s = e4m3_from_f32(__fmul_rn(__fdiv_rn(__uint_as_float(bits), 6.0f), g));
    const float e = (s & 0x7Fu) == 0u ? 0.0f : __fdiv_rn(g, f32_from_e4m3(s & 0x7Fu));
    uint2 codes;
    codes.x = encode8(w0.x, w0.y, w0.z, w0.w, e);
    codes.y = encode8(w1.x, w1.y, w1.z, w1.w, e);
    uint8_t *c = (is_v ? p.vc : p.kc) + row * p.row_codes;
    uint8_t *sc = (is_v ? p.vs : p.ks) + row * p.row_scales;
    reinterpret_cast<uint2 *>(c)[blk] = codes;
    sc[blk] = (uint8_t)s;
}

}  // namespace

__global__ void __launch_bounds__(256) k_kv_write(KvWriteParams p) { kv_write_body<0>(p); }
__global__ void __launch_bounds__(256) k_kv_write_half(KvWriteParams p) { kv_write_body<1>(p); }
__global__ void __launch_bounds__(256) k_kv_write_any(KvWriteParams p) { kv_write_body<2>(p); }

__global__ void __launch_bounds__(256) k_kv_read(KvReadParams p) {
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    if (item >= p.items) return;
    const uint32_t r = quotient(item, p.per_row);
    uint32_t blk = item - r * p.per_row.d;
    const bool is_v = blk >= p.row_blocks;
    if (is_v) blk -= p.row_blocks;
    const int64_t row = pool_row(p.slots[r], p.pool_rows, p.status);
    uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (row >= 0) {
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>((is_v ? p.vc : p.kc) + row * p.row_codes) + blk);
        const uint32_t s = __ldg((is_v ? p.vs : p.ks) + row * p.row_scales + blk);
        const float d = __fdiv_rn(f32_from_e4m3(s), is_v ? *p.gv : *p.gk);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t byte = ((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu;
            const float2 f = f32x2_from_f16x2(f16x2_from_e2m1x2(byte));
            o[i] = bf16x2_from_f32(__fmul_rn(f.x, d), __fmul_rn(f.y, d));
        }
    }
    uint16_t *y = (is_v ? p.yv + (int64_t)r * p.ldv : p.yk + (int64_t)r * p.ldk) + 16 * (int64_t)blk;
    store_32b(y, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]), p.vec32 != 0);
}

}  // namespace nvfp4
