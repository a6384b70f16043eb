// Device helpers shared by the rotary, cache and paged attention kernels.
// Internal to libnvfp4.so.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

__device__ __forceinline__ uint32_t quotient(uint32_t n, const FastDiv &f) {
    return (__umulhi(n, f.m) + n) >> f.s;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// One pair: each product and the sum rounded to nearest (no contraction).
__device__ __forceinline__ void rotate(float x1, float x2, float c, float s, float &y1, float &y2) {
    y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
    y2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
}

// Table row of a position, or -1 for a row that is left alone: position -1
// (padding), or a position outside of the table, which is recorded.
__device__ __forceinline__ int64_t rope_row(int32_t position, int64_t table_rows, uint32_t *status) {
    if (position >= 0 && position < table_rows) return position;
    if (position != -1) set_status(status, ST_INVALID_ARG);
    return -1;
}

// Pool row of a slot in the same manner.
__device__ __forceinline__ int64_t pool_row(int32_t slot, int64_t rows, uint32_t *status) {
    if (slot >= 0 && slot < rows) return slot;
    if (slot != -1) set_status(status, ST_INVALID_ARG);
    return -1;
}

}  // namespace

}  // namespace nvfp4
