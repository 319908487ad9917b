// sv_attend.cuh -- attention of new tokens over the paged cache.
#pragma once

#include "sv_append.cuh"
#include "sv_cache.cuh"

namespace sv {

struct AttendParams {
    Batch batch;
    const void *q, *k_cache, *v_cache;
    void *out;
    int64_t q_st[2], o_st[2], kc_st[3], vc_st[3];
    int32_t q_heads, kv_heads, head_dim, window;
    float scale;
};

// One warp per (token, query head): the running maximum and sum of the
// softmax over one key at a time, lanes over the head's values.
template <class T>
__global__ void __launch_bounds__(256) attend_kernel(const __grid_constant__ AttendParams A) {
    const int lane = threadIdx.x % 32;
    const int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (w >= (int64_t)A.batch.tokens * A.q_heads) return;
    const int32_t t = (int32_t)(w / A.q_heads), h = (int32_t)(w - (int64_t)t * A.q_heads);
    const int32_t b = find_sequence(A.batch.q_start, A.batch.B, t, lane);
    if (b < 0) return;
    const Sequence s = load_sequence(A.batch, b);
    if (s.bad) {
        if (lane == 0) atomicOr(A.batch.status, SV_STATUS_BAD_LENGTH);
        return;
    }
    const int32_t j = t - s.row0;
    if (j < 0 || j >= s.n) return;
    const int32_t g = h / (A.q_heads / A.kv_heads);
    const T *q = static_cast<const T *>(A.q) + t * A.q_st[0] + h * A.q_st[1];
    float qv[4], o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < 4; ++i)
        qv[i] = lane + 32 * i < A.head_dim ? to_f32<T>(q[lane + 32 * i]) * A.scale : 0.f;
    const int32_t last = s.len - s.n + j;
    const int32_t first = A.window > 0 ? max(0, last - A.window + 1) : 0;
    float m = -INFINITY, l = 0.f;
    for (int32_t x = first; x <= last; ++x) {
        const int32_t pg = x / A.batch.page_size, at = x - pg * A.batch.page_size;
        const int32_t id = __ldg(A.batch.pages + b * A.batch.pages_stride + pg);
        const bool ok = id >= 0 && id < A.batch.num_pages;
        if (!ok && lane == 0) atomicOr(A.batch.status, SV_STATUS_BAD_PAGE);
        const T *k = static_cast<const T *>(A.k_cache) + id * A.kc_st[0] + at * A.kc_st[1] +
                     g * A.kc_st[2];
        const T *v = static_cast<const T *>(A.v_cache) + id * A.vc_st[0] + at * A.vc_st[1] +
                     g * A.vc_st[2];
        float dot = 0.f;
        for (int i = 0; i < 4; ++i)
            if (ok && lane + 32 * i < A.head_dim) dot += qv[i] * to_f32<T>(k[lane + 32 * i]);
        for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        const float mn = fmaxf(m, dot), keep = __expf(m - mn), p = __expf(dot - mn);
        m = mn;
        l = l * keep + p;
        for (int i = 0; i < 4; ++i) {
            o[i] *= keep;
            if (ok && lane + 32 * i < A.head_dim) o[i] += p * to_f32<T>(v[lane + 32 * i]);
        }
    }
    T *out = static_cast<T *>(A.out) + t * A.o_st[0] + h * A.o_st[1];
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < A.head_dim) out[lane + 32 * i] = from_f32<T>(l > 0.f ? o[i] / l : 0.f);
}

}  // namespace sv
