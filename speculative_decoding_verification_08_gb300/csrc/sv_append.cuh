// sv_append.cuh -- rotation of new queries and keys, and the append of keys
// and values to the paged cache.
//
// Pair (a, c) of a head turns by the angle position * inv_freq[i]:
// (a cos - c sin, a sin + c cos) in fp32, rounded once to the cache's type.
// The angle is formed in fp64 and reduced to a fraction of a turn before it
// drops to fp32, so cos and sin are good to ~1e-7 at any position (in fp32 a
// position of 2^20 would leave an angle error of 0.06).
//
// Bound by memory: every value is read once and written once and the
// arithmetic is a few operations each.  A block takes kAppendTokens tokens (or
// one, when there are few): a warp per token finds its sequence (32-way
// search of q_start), slot, page and its rot_dim / 2 cosines and sines, then
// all threads stream the tokens' heads with 16-byte accesses.
#pragma once

#include "sv_cache.cuh"

namespace sv {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;
constexpr int kMaxHeadDim = 128;

struct AppendParams {
    Batch batch;
    const void *k, *v, *q;
    void *q_out, *k_cache, *v_cache;
    int64_t k_st[2], v_st[2], q_st[2], o_st[2];  // token and head strides, elements
    int64_t kc_st[3], vc_st[3];                  // page, slot and head strides
    const double *inv_freq;
    const int32_t *positions;
    int32_t q_heads, kv_heads, head_dim, rot_dim;
};

// The largest b with q_start[b] <= t, by a whole warp (q_start ascending).
__device__ __forceinline__ int32_t find_sequence(const int32_t *q_start, int32_t B, int32_t t,
                                                 int lane) {
    int32_t lo = 0, hi = B;  // q_start[lo] <= t is assumed, the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 31) / 32;
        const int32_t at = lo + lane * step;
        const bool le = at < hi && __ldg(q_start + at) <= t;
        const int got = 32 - __clz(__ballot_sync(0xffffffffu, le));  // lanes 0..got-1 hold
        if (got == 0) return -1;
        lo += (got - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

template <int N>
struct alignas(2 * N) Pack {
    uint16_t x[N];
};

template <class T>
__device__ __forceinline__ float f32_of(uint16_t x) {
    T y;
    *reinterpret_cast<uint16_t *>(&y) = x;
    return to_f32<T>(y);
}

template <class T>
__device__ __forceinline__ uint16_t bits_of(float x) {
    const T y = from_f32<T>(x);
    return *reinterpret_cast<const uint16_t *>(&y);
}

// One head's work item i: a pair of packs of the rotated part, or one pack of
// the rest.  kVec values per pack.
template <class T, int kVec, bool kInterleaved>
__device__ __forceinline__ void rotate_item(const uint16_t *src, uint16_t *dst, int i, int half,
                                            const float2 *cs) {
    typedef Pack<kVec> P;
    const int pairs = half / kVec;
    if (i < pairs) {
        P a, c;
        int ia, ic;
        if (kInterleaved) {
            ia = 2 * i * kVec;
            ic = ia + kVec;
        } else {
            ia = i * kVec;
            ic = ia + half;
        }
        a = *reinterpret_cast<const P *>(src + ia);
        c = *reinterpret_cast<const P *>(src + ic);
        const float2 *t = cs + i * kVec;
        if (kInterleaved) {
#pragma unroll
            for (int e = 0; e < kVec; e += 2) {
                const float2 u = t[e / 2], w = t[(kVec + e) / 2];
                const float a0 = f32_of<T>(a.x[e]), a1 = f32_of<T>(a.x[e + 1]);
                a.x[e] = bits_of<T>(a0 * u.x - a1 * u.y);
                a.x[e + 1] = bits_of<T>(a0 * u.y + a1 * u.x);
                const float c0 = f32_of<T>(c.x[e]), c1 = f32_of<T>(c.x[e + 1]);
                c.x[e] = bits_of<T>(c0 * w.x - c1 * w.y);
                c.x[e + 1] = bits_of<T>(c0 * w.y + c1 * w.x);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float2 u = t[e];
                const float x = f32_of<T>(a.x[e]), y = f32_of<T>(c.x[e]);
                a.x[e] = bits_of<T>(x * u.x - y * u.y);
                c.x[e] = bits_of<T>(x * u.y + y * u.x);
            }
        }
        *reinterpret_cast<P *>(dst + ia) = a;
        *reinterpret_cast<P *>(dst + ic) = c;
    } else {
        const int at = 2 * half + (i - pairs) * kVec;
        *reinterpret_cast<P *>(dst + at) = *reinterpret_cast<const P *>(src + at);
    }
}

struct TokenPlace {
    int32_t token;      // -1: no sequence takes this row
    int32_t page, at;   // page -1: not written to the cache
};

template <class T, int kVec, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(const __grid_constant__ AppendParams A, int per_block) {
    __shared__ TokenPlace place[kAppendTokens];
    __shared__ float2 cs[kAppendTokens][kMaxHeadDim / 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t t0 = (int32_t)blockIdx.x * per_block;
    const int here = min(per_block, A.batch.tokens - t0);
    const int half = A.rot_dim / 2;

    for (int w = warp; w < here; w += kAppendThreads / 32) {
        const int32_t t = t0 + w;
        TokenPlace p = {-1, -1, 0};
        int64_t pos = 0;
        const int32_t b = find_sequence(A.batch.q_start, A.batch.B, t, lane);
        if (b >= 0) {
            const Sequence s = load_sequence(A.batch, b);
            const int32_t j = t - s.row0;
            if (s.bad) {
                if (lane == 0) atomicOr(A.batch.status, SV_STATUS_BAD_LENGTH);
            } else if (j >= 0 && j < s.n) {
                p.token = t;
                const int64_t slot = (int64_t)s.len - s.n + j;
                pos = A.positions ? (int64_t)__ldg(A.positions + t) : slot;
                if (slot < 0) {
                    if (lane == 0) atomicOr(A.batch.status, SV_STATUS_BAD_LENGTH);
                } else {
                    const int32_t pg = (int32_t)slot / A.batch.page_size;
                    const int32_t id = __ldg(A.batch.pages + b * A.batch.pages_stride + pg);
                    if (id < 0 || id >= A.batch.num_pages) {
                        if (lane == 0) atomicOr(A.batch.status, SV_STATUS_BAD_PAGE);
                    } else {
                        p.page = id;
                        p.at = (int32_t)slot - pg * A.batch.page_size;
                    }
                }
            }
        }
        if (lane == 0) place[w] = p;
        if (p.token >= 0)
            for (int i = lane; i < half; i += 32) {
                const double turns = (double)pos * __ldg(A.inv_freq + i) * 0.15915494309189535;
                float s, c;
                sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
                cs[w][i] = make_float2(c, s);
            }
    }
    __syncthreads();

    const uint16_t *q = static_cast<const uint16_t *>(A.q);
    const uint16_t *k = static_cast<const uint16_t *>(A.k);
    const uint16_t *v = static_cast<const uint16_t *>(A.v);
    const int turned = half / kVec + (A.head_dim - A.rot_dim) / kVec;  // items per rotated head
    const int per_head_v = A.head_dim / 8;
    const int rot_items = (A.q_heads + A.kv_heads) * turned;
    const int items = rot_items + A.kv_heads * per_head_v;
    for (int w = 0; w < here; ++w) {
        const TokenPlace p = place[w];
        if (p.token < 0) continue;
        const int64_t t = p.token;
        for (int i = threadIdx.x; i < items; i += kAppendThreads) {
            if (i < rot_items) {
                const int h = i / turned, x = i - h * turned;
                if (h < A.q_heads) {
                    rotate_item<T, kVec, kInterleaved>(
                        q + t * A.q_st[0] + h * A.q_st[1],
                        static_cast<uint16_t *>(A.q_out) + t * A.o_st[0] + h * A.o_st[1], x, half,
                        cs[w]);
                } else if (p.page >= 0) {
                    const int g = h - A.q_heads;
                    rotate_item<T, kVec, kInterleaved>(
                        k + t * A.k_st[0] + g * A.k_st[1],
                        static_cast<uint16_t *>(A.k_cache) + p.page * A.kc_st[0] +
                            p.at * A.kc_st[1] + g * A.kc_st[2],
                        x, half, cs[w]);
                }
            } else if (p.page >= 0) {
                const int r = i - rot_items, g = r / per_head_v, x = (r - g * per_head_v) * 8;
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(A.v_cache) +
                                           p.page * A.vc_st[0] + p.at * A.vc_st[1] +
                                           g * A.vc_st[2] + x) =
                    *reinterpret_cast<const uint4 *>(v + t * A.v_st[0] + g * A.v_st[1] + x);
            }
        }
    }
}

}  // namespace sv
