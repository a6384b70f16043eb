// Kernel parameter blocks and launch entry points shared by the host API
// (api.cu) and the kernel files.  Internal to libnvfp4.so.
#pragma once
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "gemm.h"

namespace nvfp4 {

struct EncodeParams {
    const uint16_t *x;      // BF16 source, row pitch ld elements
    int64_t ld;
    int64_t rows, cols;     // output (gathered) shape
    const int32_t *gather;  // optional row map (output row -> source row, -1 = zero row)
    int64_t src_rows;       // rows of x (gathered indices must lie below)
    uint8_t *codes;
    uint8_t *scales;
    int32_t layout;         // 0 swizzled 128x4, 1 linear
    float *global;
    int32_t global_supplied;
    const uint32_t *partials;
    int32_t n_partials;
    uint32_t *status;
    uint32_t rht_mask = 0;  // random Hadamard transform: sign bit j negates value j of a block
    uint64_t sr_seed = 0;   // stochastic rounding: Philox key
};

// Quantize / dequantize work unit: one row and kChunkBlocks consecutive
// 16-value blocks of it per warp task.
constexpr int kChunkBlocks = 128;

// Warp tasks of the encode kernel (rows padded to 128 in the swizzled
// layout; scale columns padded to a multiple of 4): rows of at least
// kChunkBlocks blocks split into chunks of kChunkBlocks, narrower rows into
// 32-block groups.
inline int64_t encode_tasks(int64_t rows, int64_t cols, int32_t layout) {
    const int64_t rows_out = (layout == 0) ? (rows + 127) / 128 * 128 : rows;
    const int64_t groups = ((cols / 16 + 3) / 4 * 4 + 31) / 32;
    return rows_out * (groups >= kChunkBlocks / 32 ? (groups + 3) / 4 : groups);
}

// True when rows are split into 32-block groups (a warp then takes four
// tasks per pass) rather than chunks.
inline bool tasks_are_groups(int64_t cols) {
    return ((cols / 16 + 3) / 4 * 4 + 31) / 32 < kChunkBlocks / 32;
}

// Warp tasks of the dequantize kernel (same split, unpadded).
inline int64_t decode_tasks(int64_t rows, int64_t cols) {
    const int64_t groups = (cols / 16 + 31) / 32;
    return rows * (groups >= kChunkBlocks / 32 ? (groups + 3) / 4 : groups);
}

struct DequantParams {
    const uint8_t *codes;
    const uint8_t *scales;
    int32_t layout;
    const float *global;
    int64_t rows, cols;
    uint16_t *y;
    int64_t ld;
    int32_t y_vec32 = 0;    // 1: y and ld * 2 bytes are 32-byte aligned (one 256-bit store per block)
};

// Row gather of an NVFP4 tensor (gather.cu).
struct GatherParams {
    const uint8_t *src_codes, *src_scales;
    const float *src_global;
    int32_t src_layout;
    int64_t src_rows;
    uint8_t *dst_codes, *dst_scales;
    float *dst_global;
    int32_t dst_layout;
    int64_t rows, cols;      // output rows, columns (values per row)
    const int32_t *map;      // output row -> source row, -1 = zero row
    uint32_t *status;
};
constexpr int kGatherSplit = 2;   // CTAs per 128-row output band (grid.y of k_gather_rows)
__global__ void k_gather_rows(GatherParams p);

__global__ void k_amax(const uint16_t *x, int64_t ld, int64_t rows, int64_t cols,
                       const int32_t *gather, int64_t src_rows, uint32_t *partials,
                       uint32_t *status);
__global__ void k_amax_rht(const uint16_t *x, int64_t ld, int64_t rows, int64_t cols,
                           uint32_t rht_mask, uint32_t *partials);
__global__ void k_finalize_g(const uint32_t *partials, int n, float *global, uint32_t *status);
__global__ void k_encode(EncodeParams p);
__global__ void k_encode_narrow(EncodeParams p);
__global__ void k_encode_rht(EncodeParams p);
__global__ void k_encode_rht_narrow(EncodeParams p);
__global__ void k_encode_sr(EncodeParams p);
__global__ void k_encode_sr_narrow(EncodeParams p);
__global__ void k_encode_rht_sr(EncodeParams p);
__global__ void k_encode_rht_sr_narrow(EncodeParams p);
// Column-wise quantization (out = NVFP4 of x^T): p.rows = columns of x,
// p.cols = rows of x (a multiple of 16), x is p.cols x p.rows with pitch
// p.ld; 128 threads per CTA.
constexpr int kTransposeThreads = 128;
constexpr int kTransposeSmemBytes = (kTransposeThreads / 32) * 2 * 64 * 64 * 2;   // 64 KiB
cudaError_t launch_transpose_kernel(const void *kernel, int grid, void **args, cudaStream_t stream);
__global__ void k_amax_t_rht(const uint16_t *x, int64_t ld, int64_t R, int64_t C, uint32_t rht_mask,
                             uint32_t *partials);
__global__ void k_encode_t(EncodeParams p);
__global__ void k_encode_t_rht(EncodeParams p);
__global__ void k_encode_t_2d(EncodeParams p);
__global__ void k_encode_t_sr(EncodeParams p);
__global__ void k_encode_t_rht_sr(EncodeParams p);
// 2D (16x16 block) row-wise encode: 256 threads; tasks of 16 rows x 256 columns.
__global__ void k_encode_2d(EncodeParams p);
inline int64_t transpose_tasks(int64_t x_rows, int64_t out_rows_padded) {
    return ((x_rows + 63) / 64) * ((out_rows_padded + 63) / 64);
}

// Consumers.  MoE combine: one CTA of 256 threads per token.
constexpr int kMaxTopk = 32;
struct CombineParams {
    const uint16_t *out;     // expert outputs, BF16, pitch ld
    int64_t ld;
    int64_t out_rows;        // rows of out: slots at or past it are skipped
    const int32_t *slots;    // [tokens x topk] rows of out (-1 = none)
    const float *weights;    // [tokens x topk]
    int32_t topk;
    int64_t hidden;
    uint16_t *y;             // [tokens x hidden] BF16, pitch ldy
    int64_t ldy;
};
__global__ void k_moe_combine(CombineParams p);

// NVFP4 -> E4M3 bytes (pitch ld) and the per-tensor factor RN(8 / g).
struct Fp8Params {
    const uint8_t *codes;
    const uint8_t *scales;
    int32_t layout;
    const float *global;
    int64_t rows, cols;
    uint8_t *y;
    int64_t ld;
    float *fp8_scale;
};
__global__ void k_dequantize_fp8(Fp8Params p);

// SiLU-gated activation + quantize: gu = [gate | up] BF16 rows x 2*inter.
struct SwigluParams {
    const uint16_t *gu;
    int64_t ld;
    int64_t rows, inter;
    uint8_t *codes;
    uint8_t *scales;
    int32_t layout;
    float *global;
    uint32_t *partials;
    int32_t n_partials;
    uint32_t *status;
};
__global__ void k_amax_swiglu(SwigluParams p);
__global__ void k_encode_swiglu(SwigluParams p);

// MXFP4 (block 32, UE8M0 scales, no tensor scale); 256 threads.
__global__ void k_encode_mx(EncodeParams p);
__global__ void k_dequantize_mx(DequantParams p);

__global__ void k_dequantize(DequantParams p);
__global__ void k_dequantize_narrow(DequantParams p);

// Decode attention over an NVFP4 KV cache: one query token, grouped query
// heads, head_dim 128, K and V [tokens x heads_kv * 128] in the linear
// scale layout.  Pass 1 (grid chunks x heads_kv, kAttnThreads threads):
// per chunk of tokens and KV head, the running score maximum m, the weight
// sum l and the unnormalised output O of each of the group's query heads.
// Pass 2 (grid heads_q, 128 threads): merge the chunks, o = O / l / g_V.
constexpr int kAttnDim = 128;        // head_dim
constexpr int kAttnMaxGroup = 8;     // query heads per KV head
constexpr int kAttnThreads = 256;
constexpr int kAttnSub = 256;        // tokens per sub-tile (one per thread)
struct AttnParams {
    const uint16_t *q;               // BF16 [heads_q x 128], pitch ldq
    int64_t ldq;
    const uint8_t *kc, *ks;          // K codes [tokens x cols/2], scales [tokens x cols/16]
    const uint8_t *vc, *vs;
    const float *gk, *gv;            // tensor scales
    int64_t tokens, cols;            // cols = heads_kv * 128
    int32_t heads_kv, group;         // heads_q = group * heads_kv
    float scale;                     // softmax scale
    int64_t chunk;                   // tokens per pass-1 CTA, a multiple of kAttnSub
    int32_t n_chunks;
    float *part_o;                   // [n_chunks][heads_q][128]
    float *part_ml;                  // [n_chunks][heads_q][2]: m (log2 units), l
    uint16_t *o;                     // BF16 [heads_q x 128], pitch ldo
    int64_t ldo;
};
__global__ void k_attn_partial(AttnParams p);
__global__ void k_attn_combine(AttnParams p);

// Division of n < 2^31 by a launch constant d >= 1: n / d =
// (hi32(n m) + n) >> s with s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994; for n < 2^31 the sum stays below 2^32).
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f;
    f.d = d;
    f.s = 0;
    while (f.s < 31 && (1u << f.s) < d) ++f.s;
    f.m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.s) - d)) / d + 1);
    return f;
}

// Rotary positions (rope.cu).
struct RopeParams {
    const uint16_t *x;       // BF16, strides in elements
    int64_t xs_t, xs_h;
    uint16_t *y;
    int64_t ys_t, ys_h;
    const int32_t *positions;
    const float2 *table;     // [table_rows][pairs] (cos, sin)
    int64_t table_rows;
    int32_t pairs, heads;
    float sign;              // +1, or -1 for the inverse
    uint32_t items;          // work items (tokens x heads x items of a head)
    FastDiv per_token, per_head;
    // half layout in pieces that the rotated part's borders cut: a token's
    // items but for those of the cut pieces, and cut pieces of a head (1 or 2)
    uint32_t uncut, cuts;
    uint32_t *status;
};
constexpr int kRopeHeads = 4;   // heads that an item of 16-byte pieces takes
__global__ void k_rope_table(const double *inv_freq, int32_t pairs, int64_t first, int64_t n,
                             double magnitude, float2 *table);
__global__ void k_rope_half(RopeParams p);
__global__ void k_rope_half_pieces(RopeParams p);
__global__ void k_rope_interleaved(RopeParams p);
__global__ void k_rope_interleaved_pieces(RopeParams p);
__global__ void k_rope_any(RopeParams p, int interleaved, int with_rest);

// Paged cache write and read (kv_cache.cu).
struct KvWriteParams {
    const uint16_t *k, *v;   // BF16 [tokens][heads][dim], strides in elements
    int64_t ks_t, ks_h, vs_t, vs_h;
    const int32_t *slots;    // [tokens] pool rows, -1 = none
    int64_t pool_rows;
    uint8_t *kc, *ks, *vc, *vs;
    const float *gk, *gv;
    int64_t row_codes, row_scales;
    const int32_t *positions;
    const float2 *table;     // nullptr: keys are not rotated
    int64_t table_rows;
    int32_t pairs;
    int32_t interleaved;
    // items of one or two blocks
    uint32_t items, k_items; // tokens x (items of a K row + items of a V row); of a K row
    FastDiv per_token;
    FastDiv per_head_k, per_head_v;
    uint32_t head_blocks;
    uint32_t *status;
};
constexpr int kWriteCtasPerSm = 3;   // one wave of CTAs, each thread an item ahead
__global__ void k_kv_write(KvWriteParams p);
__global__ void k_kv_write_half(KvWriteParams p);
__global__ void k_kv_write_any(KvWriteParams p);

struct KvReadParams {
    const uint8_t *kc, *ks, *vc, *vs;
    const float *gk, *gv;
    int64_t pool_rows, row_codes, row_scales;
    const int32_t *slots;
    uint16_t *yk, *yv;       // BF16 [rows][cols], pitches in elements
    int64_t ldk, ldv;
    int32_t vec32;           // both outputs allow 32-byte stores
    uint32_t items;          // rows x (blocks of a K row + blocks of a V row)
    FastDiv per_row;
    uint32_t row_blocks;
    uint32_t *status;
};
constexpr int kReadItems = 4;   // blocks a thread takes
__global__ void k_kv_read(KvReadParams p);

// Decode attention over a paged cache (attention_paged.cu).
//
// The launch plan, by the head counts alone (so that the scratch does not
// depend on lengths or device).  A unit is a KV head with up to 8 of its query
// heads.  The 8 computing warps of a CTA are heads_cta x subs x parts (powers
// of two): neighbouring KV heads, units of one head, and 16-token parts of
// the tile of 16 x parts tokens that a stage of the ring holds.
// Four units a CTA: whole 256-byte pieces of a cache row of 128-value heads;
// 8 units were 2 to 6 % slower (twice the parts to join), 2 units 6 to 12 %
// (each row in more pieces).
constexpr int kPagedUnitsCta = 4;
constexpr int kPagedMaxStages = 8;
constexpr int kPagedMaxHeads = 65535;        // of queries: no more CTAs over the units than a grid's second axis has
constexpr int kPagedSmem = 112 * 1024;       // two CTAs an SM
constexpr int kPagedSmem256 = 223 * 1024;    // one CTA an SM, with some 3 KB of barriers and the like
struct PagedPlan {
    int units_head, units;                   // units of a KV head, of all
    int heads_shift, subs_shift, parts_shift;
    int blocks, ranges;                      // CTAs over the units; ranges of the tile list
    int stages, stage_bytes, smem;
};
inline PagedPlan paged_plan(int heads_q, int heads_kv, int dim) {
    PagedPlan n;
    n.units_head = (heads_q / heads_kv + 7) / 8;
    n.units = heads_kv * n.units_head;
    n.subs_shift = n.units_head % 4 == 0 ? 2 : n.units_head % 2 == 0 ? 1 : 0;
    n.heads_shift = 0;
    while ((2 << (n.heads_shift + n.subs_shift)) <= kPagedUnitsCta && heads_kv % (2 << n.heads_shift) == 0) ++n.heads_shift;
    n.parts_shift = 3 - n.subs_shift - n.heads_shift;
    n.blocks = (heads_kv >> n.heads_shift) * (n.units_head >> n.subs_shift);
    const int ctas = dim == 256 ? 148 : 296;                          // one wave of 148 SMs
    n.ranges = ctas / n.blocks > 1 ? ctas / n.blocks : 1;
    const int heads = 1 << n.heads_shift, parts = 1 << n.parts_shift;
    const int groups = heads * (dim / 16) / 16 > 1 ? heads * (dim / 16) / 16 : 1;
    n.stage_bytes = (2 * parts * 16 * (heads * (dim / 2) + groups * 16) + 1023) / 1024 * 1024;
    const int sums = 8 * 8 * dim * 4;                                  // the warps' O
    const int room = (dim == 256 ? kPagedSmem256 : kPagedSmem) - 1024 - sums;
    n.stages = room / n.stage_bytes < kPagedMaxStages ? room / n.stage_bytes : kPagedMaxStages;
    n.smem = 1024 + n.stages * n.stage_bytes + sums;
    return n;
}
// Scratch: per range two parts (a sequence cut at its start, one cut at its
// end) of each unit: 8 x dim values and 8 (m, l) pairs; then the joins.
inline size_t paged_scratch_bytes(const PagedPlan &n, int dim) {
    return (size_t)2 * n.ranges * n.units * (8 * dim + 16) * 4 + (size_t)n.ranges * 16;
}

// Codes as (byte of a head, row, head), boxes of one head's bytes x 16 rows x
// the CTA's heads; scales as (byte of 16, row, group of 16 bytes).
struct PagedMaps {
    CUtensorMap kc, ks, vc, vs;
};

struct PagedAttnParams {
    const uint16_t *q;       // BF16 [sequences][heads_q][dim], strides in elements
    int64_t qs_b, qs_h;
    const uint8_t *kc, *ks, *vc, *vs;
    const float *gk, *gv;
    int64_t row_codes, row_scales;
    const int32_t *block_table;
    int64_t table_stride;
    int32_t capacity;        // tokens that a sequence's table entries hold
    int32_t n_pages;         // pages of the pool
    const int32_t *seq_lens;
    int32_t sequences, heads_q, group, page_size;
    FastDiv page_div;
    PagedPlan plan;
    FastDiv sub_blocks;      // CTAs over the units of a head
    int32_t tma;             // page_size % 16 == 0 (16 tokens share a page) and 16-byte scale rows: tiles by TMA
    long long timeout;       // clock bound of a wait
    float scale;
    uint16_t *o;
    int64_t os_b, os_h;
    float *lse;              // nullptr, or [sequences][heads_q]
    // [2 ranges][units][dim / 16][lane]: values of an M-tile of O^T in a lane
    float4 *part_o;
    float4 *part_ml;         // [2 ranges][units][4]: (m, l) of heads 2c and 2c + 1
    int4 *joins;             // (sequence, first range, parts): by sequence, or by range if there are more sequences
    uint32_t *status;
};
cudaError_t launch_paged_attention(const PagedAttnParams &p, const PagedMaps &maps, int dim, cudaStream_t s);

}  // namespace nvfp4
