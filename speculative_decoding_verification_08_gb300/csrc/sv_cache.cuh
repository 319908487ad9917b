// sv_cache.cuh -- what the paged-cache kernels share: the batch as the device
// sees it, element types, and a sequence's checked lengths.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "specverify.h"

namespace sv {

// Division of 0 <= n < 2^31 by a fixed d >= 1: the high word of n m, shifted;
// m = ceil(2^(31 + s) / d) with 2^s >= d, whose excess over the exact factor
// is too small to reach the next integer for these n.
struct FastDiv {
    uint32_t d, m, s;
    __host__ void set(uint32_t by) {
        d = by;
        s = 0;
        while ((1ull << s) < by) ++s;
        m = (uint32_t)(((1ull << (31 + s)) + by - 1) / by);
    }
    __device__ __forceinline__ int div(int n) const {
        return d == 1 ? n : (int)(__umulhi((uint32_t)n, m) >> (s - 1));
    }
};

struct Batch {
    const int32_t *pages;
    int64_t pages_stride;
    const int32_t *q_start;
    const int32_t *kv_len;
    int32_t B, tokens, num_pages, page_size, max_pages;
    uint32_t *status;
};

struct Sequence {
    int32_t row0, n, len;  // first token row, new tokens, length with them
    bool bad;
};

// Sequence b's lengths; one that does not fit is left out (n = 0).
__device__ __forceinline__ Sequence load_sequence(const Batch &A, int32_t b) {
    Sequence s;
    const int32_t r0 = __ldg(A.q_start + b), r1 = __ldg(A.q_start + b + 1);
    s.len = __ldg(A.kv_len + b);
    s.row0 = r0;
    s.n = r1 - r0;
    s.bad = r0 < 0 || r1 < r0 || r1 > A.tokens || s.len < 0 ||
            (int64_t)s.len > (int64_t)A.max_pages * A.page_size;
    if (s.bad) s.n = 0;
    return s;
}

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(float x) {
    return x;
}
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) {
    return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_f32(__half x) {
    return __half2float(x);
}
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32(float x) {
    return __float2half_rn(x);
}

}  // namespace sv
