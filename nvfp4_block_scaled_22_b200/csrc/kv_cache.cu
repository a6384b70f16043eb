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
// so the bytes are those of nvfp4_quantize of the (rotated) rows.  A thread
// takes two blocks at a time: a pair that the half layout rotates into each
// other, or two neighbours.
// k_kv_read: y = bf16(RN(e2m1 RN(s / g))), the steps of nvfp4_dequantize.
//
// Both are bound by memory (2.56 bytes a value): 131072 rows of 2 x 1024
// values are read back in 108 us (6.4 TB/s), 16384 tokens of 2 x 8 x 128
// written in 17.8 us (4.8 TB/s, launch included), with rotated keys in 24.3
// us (interleaved 27.3): the table rows are loaded behind slot and position,
// outside of the one item that a thread fetches ahead, and 19 warps an SM do
// not hide that (a warp waits for loads 3.7 cycles an instruction issued; 57 %
// of the issue slots are used).  Tried for the write: a half
// block a thread (30 us: the scale's arithmetic twice), two heads a thread
// that share table entries (27.6 us: registers), tables for the divisions
// (26.5 us).
#include <cstdint>
#include <cuda_runtime.h>

#include "encode_common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

struct Block {
    uint4 lo, hi;            // 16 BF16 values
};

__device__ __forceinline__ Block load_block(const uint16_t *x) {
    Block b;
    b.lo = reinterpret_cast<const uint4 *>(x)[0];
    b.hi = reinterpret_cast<const uint4 *>(x)[1];
    return b;
}

// Values i .. i + 15 (a) and their partners (b), rotated by 16 table entries.
__device__ __forceinline__ void rotate_blocks(Block &a, Block &b, const float2 *table) {
    uint32_t w[8] = {a.lo.x, a.lo.y, a.lo.z, a.lo.w, a.hi.x, a.hi.y, a.hi.z, a.hi.w};
    uint32_t u[8] = {b.lo.x, b.lo.y, b.lo.z, b.lo.w, b.hi.x, b.hi.y, b.hi.z, b.hi.w};
    const float4 *cs = reinterpret_cast<const float4 *>(table);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 f = __ldg(cs + i);
        float lo1, lo2, hi1, hi2;
        rotate(bf16_lo(w[i]), bf16_lo(u[i]), f.x, f.y, lo1, lo2);
        rotate(bf16_hi(w[i]), bf16_hi(u[i]), f.z, f.w, hi1, hi2);
        w[i] = bf16x2_from_f32(lo1, hi1);
        u[i] = bf16x2_from_f32(lo2, hi2);
    }
    a.lo = make_uint4(w[0], w[1], w[2], w[3]);
    a.hi = make_uint4(w[4], w[5], w[6], w[7]);
    b.lo = make_uint4(u[0], u[1], u[2], u[3]);
    b.hi = make_uint4(u[4], u[5], u[6], u[7]);
}

// Block `blk` of head x rotated by itself: neighbouring pairs, or partners
// fetched by 8 (pairs % 8 == 0: 16384 x 16 x 64 with 8 pairs in 24.9 us, one by
// one 35.7) or one by one (any pair count).
__device__ __forceinline__ void rotate_alone(Block &a, const uint16_t *x, int blk, const KvWriteParams &p,
                                             int64_t pos) {
    const int j0 = 16 * blk;
    if (j0 >= 2 * p.pairs) return;
    uint32_t w[8] = {a.lo.x, a.lo.y, a.lo.z, a.lo.w, a.hi.x, a.hi.y, a.hi.z, a.hi.w};
    const float2 *row = p.table + pos * p.pairs;
    if (p.interleaved) {
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
    } else if (p.pairs % 8 == 0) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int j = j0 + 8 * n;
            if (j < 2 * p.pairs) {
                const bool first = j < p.pairs;
                const int pair = first ? j : j - p.pairs;
                const uint4 q = *reinterpret_cast<const uint4 *>(first ? x + j + p.pairs : x + pair);
                const uint32_t u[4] = {q.x, q.y, q.z, q.w};
                const float4 *cs = reinterpret_cast<const float4 *>(row + pair);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 f = __ldg(cs + i);
                    const uint32_t a1 = first ? w[4 * n + i] : u[i], a2 = first ? u[i] : w[4 * n + i];
                    float lo1, lo2, hi1, hi2;
                    rotate(bf16_lo(a1), bf16_lo(a2), f.x, f.y, lo1, lo2);
                    rotate(bf16_hi(a1), bf16_hi(a2), f.z, f.w, hi1, hi2);
                    w[4 * n + i] = first ? bf16x2_from_f32(lo1, hi1) : bf16x2_from_f32(lo2, hi2);
                }
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
                    float y1, y2;
                    if (first) {
                        rotate(y[e], bf16_lo(x[j + p.pairs]), f.x, f.y, y1, y2);
                        y[e] = y1;
                    } else {
                        rotate(bf16_lo(x[pair]), y[e], f.x, f.y, y1, y2);
                        y[e] = y2;
                    }
                }
            }
            w[i] = bf16x2_from_f32(y[0], y[1]);
        }
    }
    a.lo = make_uint4(w[0], w[1], w[2], w[3]);
    a.hi = make_uint4(w[4], w[5], w[6], w[7]);
}

// One block under the tensor scale g (div6_f32 is RN(amax / 6)).
__device__ __forceinline__ EncodeBlockOut encode(const Block &x, float g) {
    const uint32_t bits = block_amax_bits(x.lo, x.hi);
    EncodeBlockOut o;
    o.scale = e4m3_from_f32(__fmul_rn(div6_f32(__uint_as_float(bits)), g));
    const uint32_t s = o.scale & 0x7Fu;
    const float e = s == 0u || s == 0x7Fu ? 0.0f : __fdiv_rn(g, f32_from_e4m3(s));
    o.codes.x = encode8(x.lo.x, x.lo.y, x.lo.z, x.lo.w, e);
    o.codes.y = encode8(x.hi.x, x.hi.y, x.hi.z, x.hi.w, e);
    o.finite = bits <= 0x7F7FFFFFu;
    return o;
}

// One or two blocks of a head, with what their writing needs.
struct WriteItem {
    Block a, b;
    const uint16_t *x;
    int32_t slot, position;
    int b0, b1, h;           // blocks (b1: -1 if there is one), head
    bool is_v, turns;        // the blocks are rotated into each other
};

// kRope: 0 no rotation, 1 half layout with whole partner blocks (pairs % 16
// == 0), 2 any other.
template <int kRope>
__device__ __forceinline__ WriteItem fetch_item(const KvWriteParams &p, uint32_t item) {
    WriteItem w;
    const uint32_t t = quotient(item, p.per_token);
    uint32_t rest = item - t * p.per_token.d;                       // of the K row, then of the V row
    w.is_v = rest >= p.k_items;
    if (w.is_v) rest -= p.k_items;
    w.h = (int)quotient(rest, w.is_v ? p.per_head_v : p.per_head_k);
    const int i = (int)rest - w.h * (int)(w.is_v ? p.per_head_v.d : p.per_head_k.d);
    w.slot = p.slots[t];
    w.position = kRope != 0 ? p.positions[t] : 0;
    w.x = w.is_v ? p.v + (int64_t)t * p.vs_t + w.h * p.vs_h : p.k + (int64_t)t * p.ks_t + w.h * p.ks_h;
    // items of a head: pairs of rotated blocks (kRope 1), then two neighbours at a time
    const int turned = kRope == 1 && !w.is_v ? p.pairs >> 4 : 0;
    w.turns = i < turned;
    w.b0 = w.turns ? i : 2 * turned + 2 * (i - turned);
    w.b1 = w.turns ? i + turned : w.b0 + 1 < (int)p.head_blocks ? w.b0 + 1 : -1;
    w.a = load_block(w.x + 16 * w.b0);
    w.b = load_block(w.x + 16 * (w.b1 >= 0 ? w.b1 : w.b0));
    return w;
}

template <int kRope>
__device__ __forceinline__ void write_item(const KvWriteParams &p, WriteItem &w) {
    const int64_t row = pool_row(w.slot, p.pool_rows, p.status);
    if (row < 0) return;
    if (kRope != 0) {
        // a token whose position has no table row is not written at all
        const int64_t pos = rope_row(w.position, p.table_rows, p.status);
        if (pos < 0) return;
        if (kRope == 1 && w.turns) rotate_blocks(w.a, w.b, p.table + pos * p.pairs + 16 * w.b0);
        if (kRope == 2 && !w.is_v) {
            rotate_alone(w.a, w.x, w.b0, p, pos);
            if (w.b1 >= 0) rotate_alone(w.b, w.x, w.b1, p, pos);
        }
    }
    const float g = __ldg(w.is_v ? p.gv : p.gk);
    uint8_t *codes = (w.is_v ? p.vc : p.kc) + row * p.row_codes + (int64_t)w.h * p.head_blocks * 8;
    uint8_t *scales = (w.is_v ? p.vs : p.ks) + row * p.row_scales + (int64_t)w.h * p.head_blocks;
    const EncodeBlockOut ea = encode(w.a, g), eb = encode(w.b, g);
    if (!ea.finite || !eb.finite) set_status(p.status, ST_NONFINITE);
    *reinterpret_cast<uint2 *>(codes + 8 * w.b0) = ea.codes;
    scales[w.b0] = (uint8_t)ea.scale;
    if (w.b1 >= 0) {
        *reinterpret_cast<uint2 *>(codes + 8 * w.b1) = eb.codes;
        scales[w.b1] = (uint8_t)eb.scale;
    }
}

// Each thread fetches its next item before it works on the one it has.
template <int kRope>
__device__ __forceinline__ void kv_write_body(const KvWriteParams &p) {
    const uint32_t step = gridDim.x * 256u;
    uint32_t item = blockIdx.x * 256u + threadIdx.x;
    if (item >= p.items) return;
    WriteItem now = fetch_item<kRope>(p, item);
#pragma unroll 1
    for (; item + step < p.items; item += step) {
        const WriteItem next = fetch_item<kRope>(p, item + step);
        write_item<kRope>(p, now);
        now = next;
    }
    write_item<kRope>(p, now);
}

}  // namespace

__global__ void __launch_bounds__(256, kWriteCtasPerSm) k_kv_write(KvWriteParams p) { kv_write_body<0>(p); }
__global__ void __launch_bounds__(256, kWriteCtasPerSm) k_kv_write_half(KvWriteParams p) { kv_write_body<1>(p); }
__global__ void __launch_bounds__(256, kWriteCtasPerSm) k_kv_write_any(KvWriteParams p) { kv_write_body<2>(p); }

// Four blocks a thread, 256 apart, loaded before the first is stored.
__global__ void __launch_bounds__(256) k_kv_read(KvReadParams p) {
    const uint32_t base = blockIdx.x * (256u * kReadItems) + threadIdx.x;
    uint2 c[kReadItems];
    uint32_t s[kReadItems];
    uint16_t *y[kReadItems];
    bool is_v[kReadItems];
#pragma unroll
    for (int n = 0; n < kReadItems; ++n) {
        const uint32_t item = base + 256u * n;
        y[n] = nullptr;
        c[n] = make_uint2(0u, 0u);
        s[n] = 0u;
        is_v[n] = false;
        if (item < p.items) {
            const uint32_t r = quotient(item, p.per_row);
            uint32_t blk = item - r * p.per_row.d;
            is_v[n] = blk >= p.row_blocks;
            if (is_v[n]) blk -= p.row_blocks;
            const int64_t row = pool_row(p.slots[r], p.pool_rows, p.status);
            y[n] = (is_v[n] ? p.yv + (int64_t)r * p.ldv : p.yk + (int64_t)r * p.ldk) + 16 * (int64_t)blk;
            if (row >= 0) {
                c[n] = __ldg(reinterpret_cast<const uint2 *>((is_v[n] ? p.vc : p.kc) + row * p.row_codes) + blk);
                s[n] = __ldg((is_v[n] ? p.vs : p.ks) + row * p.row_scales + blk);
            }
        }
    }
    const float gk = *p.gk, gv = *p.gv;
#pragma unroll
    for (int n = 0; n < kReadItems; ++n) {
        if (y[n] == nullptr) continue;
        // codes and scale 0 (no row): zeros
        const float d = __fdiv_rn(f32_from_e4m3(s[n]), is_v[n] ? gv : gk);
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t byte = ((i < 4 ? c[n].x : c[n].y) >> (8 * (i & 3))) & 0xFFu;
            const float2 f = f32x2_from_f16x2(f16x2_from_e2m1x2(byte));
            o[i] = bf16x2_from_f32(__fmul_rn(f.x, d), __fmul_rn(f.y, d));
        }
        store_32b(y[n], make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]), p.vec32 != 0);
    }
}

}  // namespace nvfp4
