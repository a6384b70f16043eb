// Decode attention of a batch of sequences over a paged NVFP4 KV cache: one
// query token a sequence, grouped-query heads,
//   s_t = scale q . k_t,  o = sum_t exp(s_t) v_t / sum_t exp(s_t),
// t over the sequence's cached tokens; token t lives in pool row
// block_table[b][t / page_size] * page_size + t % page_size.
//
// One CTA of four warps takes one query head of one sequence; warp w takes
// tokens w, w + 4, ... with the online softmax of the running maximum and
// sum, all in FP32, and the four states are joined at the end.
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

// kD / 32 values a lane, from kD / 64 code bytes.
template <int kD>
__device__ __forceinline__ void restore(const uint8_t *codes, const uint8_t *scales, int lane,
                                        float (&x)[kD / 32]) {
    constexpr int kPer = kD / 32;
    const float s = f32_from_e4m3(scales[lane * kPer / 16]);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
        const float2 f = f32x2_from_f16x2(f16x2_from_e2m1x2(codes[lane * (kPer / 2) + i]));
        x[2 * i] = __fmul_rn(f.x, s);
        x[2 * i + 1] = __fmul_rn(f.y, s);
    }
}

}  // namespace

template <int kD>
__global__ void __launch_bounds__(128) k_paged_attention(PagedAttnParams p) {
    constexpr int kPer = kD / 32;
    __shared__ float sm_m[4], sm_l[4], sm_o[4][kD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x, b = blockIdx.y, hk = h / p.group;
    const int64_t capacity = (int64_t)p.table_pages * p.page_size;
    int64_t len = p.seq_lens[b];
    if (len < 0 || len > capacity) {
        set_status(p.status, ST_INVALID_ARG);
        len = len < 0 ? 0 : capacity;
    }
    const float ck = __fdiv_rn(__fmul_rn(p.scale, kLog2e), *p.gk);
    const uint16_t *q = p.q + (int64_t)b * p.qs_b + (int64_t)h * p.qs_h;
    float qf[kPer], o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        qf[i] = bf16_lo(q[lane * kPer + i]);
        o[i] = 0.0f;
    }
    float m = __uint_as_float(0xFF7FFFFFu), l = 0.0f;      // the lowest finite value
    const int32_t *table = p.block_table + (int64_t)b * p.table_stride;
    for (int64_t t = warp; t < len; t += 4) {
        const int32_t page = table[t / p.page_size];
        if (page < 0 || page >= p.n_pages) {
            set_status(p.status, ST_INVALID_ARG);
            continue;
        }
        const int64_t row = (int64_t)page * p.page_size + t % p.page_size;
        float x[kPer], s = 0.0f;
        restore<kD>(p.kc + row * p.row_codes + hk * (kD / 2), p.ks + row * p.row_scales + hk * (kD / 16), lane, x);
#pragma unroll
        for (int i = 0; i < kPer; ++i) s = __fmaf_rn(x[i], qf[i], s);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
        s *= ck;
        const float mn = fmaxf(m, s), alpha = exp2f(m - mn), w = exp2f(s - mn);
        m = mn;
        l = l * alpha + w;
        restore<kD>(p.vc + row * p.row_codes + hk * (kD / 2), p.vs + row * p.row_scales + hk * (kD / 16), lane, x);
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = o[i] * alpha + w * x[i];
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) sm_o[warp][lane * kPer + i] = o[i];
    __syncthreads();
    const float M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    float L = 0.0f;
    for (int w = 0; w < 4; ++w) L += exp2f(sm_m[w] - M) * sm_l[w];
    for (int d = threadIdx.x; d < kD; d += 128) {
        float r = 0.0f;
        for (int w = 0; w < 4; ++w) r += exp2f(sm_m[w] - M) * sm_o[w][d];
        r = L > 0.0f || L != L ? __fdiv_rn(__fdiv_rn(r, L), *p.gv) : 0.0f;
        p.o[(int64_t)b * p.os_b + (int64_t)h * p.os_h + d] = (uint16_t)bf16x2_from_f32(r, 0.0f);
    }
    if (p.lse != nullptr && threadIdx.x == 0)
        p.lse[(int64_t)b * p.heads_q + h] = L == 0.0f ? __uint_as_float(0xFF800000u) : (M + log2f(L)) * kLn2;
}

cudaError_t launch_paged_attention(const PagedAttnParams &p, int dim, cudaStream_t s) {
    const dim3 grid((unsigned)p.heads_q, (unsigned)p.sequences);
    if (dim == 64) k_paged_attention<64><<<grid, 128, 0, s>>>(p);
    else if (dim == 128) k_paged_attention<128><<<grid, 128, 0, s>>>(p);
    else k_paged_attention<256><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace nvfp4
