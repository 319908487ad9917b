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
// arithmetic is a few operations each.  A block takes up to kAppendTokens
// tokens: a warp per token finds its sequence (32-way search of q_start), slot,
// page and its rot_dim / 2 cosines and sines, while every thread's first loads
// are on their way; then the threads, a pair of packs of a rotated head (or one
// pack of what is copied) to each, go through the tokens.
//
// 25400 tokens of 16 + 16 + 16 heads of 64 (fp16, half of a head rotated, pages
// of 16): 67 us, 4.7 TB/s, half of the issue slots taken: 6354 blocks of four tokens
// pay the lookup, the angles and a barrier each before their first store, 16-byte
// packs of 40 registers spill a little (24 bytes; 44 with adjacent pairs), and those
// of adjacent pairs leave in half sectors.  1536 tokens of 32 + 8 + 8 heads of 128: 11.8 us, 3.2
// TB/s, 3 us of it launch and lookup; one token 4.5 us.
#pragma once

#include "sv_barrier.cuh"
#include "sv_cache.cuh"

namespace sv {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 4;

struct AppendParams {
    Batch batch;
    FastDiv by_page;
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
    uint32_t x[N / 2];  // two values each
};

__device__ __forceinline__ float2 pair_of(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_of(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ uint32_t bits_of(float lo, float hi, __nv_bfloat16) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&y);
}
__device__ __forceinline__ uint32_t bits_of(float lo, float hi, __half) {
    const __half2 y = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&y);
}

// Turns a pair of packs.  cs: cosines and sines of pairs 2 e and 2 e + 1 of the
// item, `step` apart (so that neighbouring items' lie side by side).
template <class T, int kVec, bool kInterleaved>
__device__ __forceinline__ void turn(Pack<kVec> &a, Pack<kVec> &c, const float4 *cs, int step) {
    if (kInterleaved) {
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e) {   // pair e of a, pair kVec / 2 + e of c
            const float2 x = pair_of(a.x[e], T()), y = pair_of(c.x[e], T());
            const float4 p = cs[e / 2 * step], q = cs[(kVec / 2 + e) / 2 * step];
            const float2 u = e % 2 ? make_float2(p.z, p.w) : make_float2(p.x, p.y);
            const float2 w = (kVec / 2 + e) % 2 ? make_float2(q.z, q.w) : make_float2(q.x, q.y);
            a.x[e] = bits_of(x.x * u.x - x.y * u.y, x.x * u.y + x.y * u.x, T());
            c.x[e] = bits_of(y.x * w.x - y.y * w.y, y.x * w.y + y.y * w.x, T());
        }
    } else {
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e) {   // pairs 2 e and 2 e + 1
            const float2 x = pair_of(a.x[e], T()), y = pair_of(c.x[e], T());
            const float4 u = cs[e * step];
            a.x[e] = bits_of(x.x * u.x - y.x * u.y, x.y * u.z - y.y * u.w, T());
            c.x[e] = bits_of(x.x * u.y + y.x * u.x, x.y * u.w + y.y * u.z, T());
        }
    }
}

// Where a block's token goes: offsets into q_out, the key and the value cache;
// -1: nowhere.
struct TokenPlace {
    int64_t to[3];
};

template <class T, int kVec, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads, 6)
    append_kernel(const __grid_constant__ AppendParams A, int per_block) {
    __shared__ TokenPlace place[kAppendTokens];
    __shared__ float4 cs[kAppendTokens][kMaxHeadDim / 4];
    typedef Pack<kVec> P;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t t0 = (int32_t)blockIdx.x * per_block;
    const int here = min(per_block, A.batch.tokens - t0);
    const int half = A.rot_dim / 2;
    const int pairs = half / kVec;
    const int turned = pairs + (A.head_dim - A.rot_dim) / kVec;  // items of a rotated head
    const int per_value = A.head_dim / kVec;
    const int rot_items = (A.q_heads + A.kv_heads) * turned;
    const int items = rot_items + A.kv_heads * per_value;

    // item i of a token: a pair of packs of a head's rotated part, or one pack of
    // what is copied (its rest, or a value)
    int kind, second, x;   // kind 0 query, 1 key, 2 value
    int64_t step;
    const uint16_t *src;
    uint16_t *dst;
    P a, c, a1, c1;
    auto fetch = [&](int i) {
        int head, at;
        second = 0;
        if (i < rot_items) {
            head = i / turned;
            x = i - head * turned;
            kind = head < A.q_heads ? 0 : 1;
            if (kind) head -= A.q_heads;
            if (x < pairs) {
                at = kInterleaved ? 2 * x * kVec : x * kVec;
                second = kInterleaved ? kVec : half;
            } else {
                at = A.rot_dim + (x - pairs) * kVec;
            }
        } else {
            x = i - rot_items;
            kind = 2;
            head = x / per_value;
            at = (x - head * per_value) * kVec;
        }
        const int64_t *st = kind == 0 ? A.q_st : kind == 1 ? A.k_st : A.v_st;
        step = st[0];
        src = static_cast<const uint16_t *>(kind == 0 ? A.q : kind == 1 ? A.k : A.v) + t0 * step +
              head * st[1] + at;
        dst = static_cast<uint16_t *>(kind == 0 ? A.q_out : kind == 1 ? A.k_cache : A.v_cache) +
              head * (kind == 0 ? A.o_st[1] : kind == 1 ? A.kc_st[2] : A.vc_st[2]) + at;
        a = *reinterpret_cast<const P *>(src);
        if (second) c = *reinterpret_cast<const P *>(src + second);
    };

    wait_for_primary_grid();
    // the first loads are on their way while the tokens' places are found
    if ((int)threadIdx.x < items) fetch(threadIdx.x);
    for (int w = warp; w < here; w += (int)blockDim.x / 32) {
        const int32_t t = t0 + w;
        TokenPlace p = {{-1, -1, -1}};
        int64_t pos = 0;
        const int32_t b = find_sequence(A.batch.q_start, A.batch.B, t, lane);
        if (b >= 0) {
            const Sequence s = load_sequence(A.batch, b);
            const int32_t j = t - s.row0;
            if (s.bad) {
                if (lane == 0) atomicOr(A.batch.status, SV_STATUS_BAD_LENGTH);
            } else if (j >= 0 && j < s.n) {
                p.to[0] = t * A.o_st[0];
                const int64_t slot = (int64_t)s.len - s.n + j;
                pos = A.positions ? (int64_t)__ldg(A.positions + t) : slot;
                if (slot < 0) {
                    if (lane == 0) atomicOr(A.batch.status, SV_STATUS_BAD_LENGTH);
                } else {
                    const int32_t pg = A.by_page.div((int)slot);
                    const int32_t id = __ldg(A.batch.pages + b * A.batch.pages_stride + pg);
                    if (id < 0 || id >= A.batch.num_pages) {
                        if (lane == 0) atomicOr(A.batch.status, SV_STATUS_BAD_PAGE);
                    } else {
                        const int64_t in = (int32_t)slot - pg * A.batch.page_size;
                        p.to[1] = id * A.kc_st[0] + in * A.kc_st[1];
                        p.to[2] = id * A.vc_st[0] + in * A.vc_st[1];
                    }
                }
            }
        }
        if (lane == 0) place[w] = p;
        if (p.to[0] >= 0)
            for (int e = lane; e < half; e += 32) {
                const double turns = (double)pos * __ldg(A.inv_freq + e) * 0.15915494309189535;
                float s, co;
                sincospif((float)(2.0 * (turns - rint(turns))), &s, &co);
                // pair e: item e / kVec's, its e % kVec
                float2 *to = reinterpret_cast<float2 *>(&cs[w][e % kVec / 2 * pairs + e / kVec]);
                to[e % 2] = make_float2(co, s);
            }
    }
    __syncthreads();

    for (int i = threadIdx.x; i < items; i += blockDim.x) {
        if (i != (int)threadIdx.x) fetch(i);
#pragma unroll 1
        for (int w = 0; w < here; ++w) {
            const bool more = w + 1 < here;
            src += step;
            if (more) {
                a1 = *reinterpret_cast<const P *>(src);
                if (second) c1 = *reinterpret_cast<const P *>(src + second);
            }
            const int64_t to = place[w].to[kind];
            if (to >= 0) {
                if (second) {
                    turn<T, kVec, kInterleaved>(a, c, &cs[w][x], pairs);
                    *reinterpret_cast<P *>(dst + to + second) = c;
                }
                *reinterpret_cast<P *>(dst + to) = a;
            }
            a = a1;
            c = c1;
        }
    }
}

}  // namespace sv
