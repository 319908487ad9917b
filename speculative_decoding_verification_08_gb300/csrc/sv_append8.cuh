// sv_append8.cuh -- the append with norms of queries and keys for each head, to
// a cache of 16-bit or of 8-bit values, and the way back: cached rows to 16 bits.
//
// A head's vector x: y = x * rsqrt(mean x^2 + eps) * w (where a norm is given),
// its pairs turned as in sv_append.cuh, all in fp32.  16-bit: rounded once.
// 8-bit: the smallest power of two 2^e, -100 <= e <= 100, with max |y| <= 448 *
// 2^e; codes are y * 2^-e (exact) rounded once to e4m3 (what lies beyond 448 *
// 2^100 saturates), the scale is e + 127 in a byte (e8m0).  A power of two costs
// e4m3 nothing but range: its relative step does not depend on the scale, and
// code times scale is exact in bf16 and fp32.  A vector with a NaN or an infinity
// has the scale NaN (255) and codes of zero.
//
// Bound by memory: a group of lanes (a power of two, 8 values each) holds a
// head's vector in registers, so that sums and maxima are a few shuffles and the
// turn's other half is a second load of the same lines.
#pragma once

#include "sv_append.cuh"

namespace sv {

struct Scales {
    uint8_t *k, *v;
    int64_t k_st[3], v_st[3];  // page, slot and head strides, bytes
};

struct AppendNormParams {
    AppendParams a;       // (cache strides in elements of the cache)
    Scales scales;        // 8-bit caches
    const void *q_norm, *k_norm;
    int32_t norm_f32;     // weights in fp32, else in the tokens' type
    float eps;
};

// ---- the 8-bit coding --------------------------------------------------------

constexpr int kMinScale = -100, kMaxScale = 100;
constexpr uint32_t kScaleNan = 255;

// The exponent for vectors whose largest magnitude has these bits (finite).
__device__ __forceinline__ int scale_exponent(uint32_t top) {
    const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kMinScale), kMaxScale);
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// What an e8m0 byte stands for.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    if (byte == 0) return __uint_as_float(0x00400000u);
    return byte == kScaleNan ? __uint_as_float(0x7fffffffu) : __uint_as_float(byte << 23);
}

// Two floats to e4m3 codes, lo in the low byte.
__device__ __forceinline__ uint32_t codes_of(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two codes to floats.
__device__ __forceinline__ float2 values_of(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// ---- the places of a block's rows ----------------------------------------------

struct RowPlace {
    int64_t k, v;     // offsets into the caches; -1: nowhere
    int64_t ks, vs;   // into the scales
    int32_t known;    // the row is one of a sequence that fits
};

// Row t of the token arrays: its slot's places, by a whole warp.  pos: its slot.
__device__ __forceinline__ RowPlace place_of(const Batch &A, const FastDiv &by_page, const int64_t *kc_st,
                                             const int64_t *vc_st, const Scales &S, int32_t t, int64_t &pos,
                                             int lane) {
    RowPlace p = {-1, -1, -1, -1, 0};
    pos = 0;
    const int32_t b = find_sequence(A.q_start, A.B, t, lane);
    if (b < 0) return p;
    const Sequence s = load_sequence(A, b);
    const int32_t j = t - s.row0;
    if (s.bad) {
        if (lane == 0) atomicOr(A.status, SV_STATUS_BAD_LENGTH);
        return p;
    }
    if (j < 0 || j >= s.n) return p;
    p.known = 1;
    pos = (int64_t)s.len - s.n + j;
    if (pos < 0) {
        if (lane == 0) atomicOr(A.status, SV_STATUS_BAD_LENGTH);
        return p;
    }
    const int32_t pg = by_page.div((int)pos);
    const int32_t id = __ldg(A.pages + b * A.pages_stride + pg);
    if (id < 0 || id >= A.num_pages) {
        if (lane == 0) atomicOr(A.status, SV_STATUS_BAD_PAGE);
        return p;
    }
    const int64_t in = (int32_t)pos - pg * A.page_size;
    p.k = id * kc_st[0] + in * kc_st[1];
    p.v = id * vc_st[0] + in * vc_st[1];
    p.ks = id * S.k_st[0] + in * S.k_st[1];
    p.vs = id * S.v_st[0] + in * S.v_st[1];
    return p;
}

// ---- append ----------------------------------------------------------------------

enum Turning { kPackTurn, kPairTurn, kAdjacentTurn };

template <class T>
__device__ __forceinline__ void unpack(const Pack<8> &p, float (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = pair_of(p.x[e], T());
        y[2 * e] = f.x;
        y[2 * e + 1] = f.y;
    }
}

// Weights of the eight values at `at`.
template <class T>
__device__ __forceinline__ void weights_at(const void *w, bool f32, int at, float (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        y[e] = f32 ? __ldg(static_cast<const float *>(w) + at + e) : to_f32<T>(static_cast<const T *>(w)[at + e]);
}

// kTurn: how a pair's other value comes.  kPackTurn: both halves of the pairs start
// on a pack (rot_dim a multiple of 16): one 16-byte load; kPairTurn: four loads of
// two; kAdjacentTurn: it lies in the same pack (also where nothing turns).
template <class T, bool kEight, Turning kTurn>
__global__ void __launch_bounds__(kAppendThreads, 2)
    append_norm_kernel(const __grid_constant__ AppendNormParams A, int per_block, int lanes) {
    __shared__ RowPlace place[kAppendTokens];
    __shared__ __align__(16) float2 cs[kAppendTokens][kMaxHeadDim / 2];
    typedef Pack<8> P;
    const AppendParams &a = A.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t t0 = (int32_t)blockIdx.x * per_block;
    const int here = min(per_block, a.batch.tokens - t0);
    const int half = a.rot_dim / 2;

    wait_for_primary_grid();
    for (int w = warp; w < here; w += (int)blockDim.x / 32) {
        int64_t pos;
        const RowPlace p = place_of(a.batch, a.by_page, a.kc_st, a.vc_st, A.scales, t0 + w, pos, lane);
        if (lane == 0) place[w] = p;
        if (p.known) {
            if (a.positions) pos = (int64_t)__ldg(a.positions + t0 + w);
            for (int e = lane; e < half; e += 32) {
                const double turns = (double)pos * __ldg(a.inv_freq + e) * 0.15915494309189535;
                float s, co;
                sincospif((float)(2.0 * (turns - rint(turns))), &s, &co);
                cs[w][e] = make_float2(co, s);
            }
        }
    }
    __syncthreads();

    // `lanes` lanes to a vector; a warp's vectors side by side
    const int sub = lane % lanes, at = sub * 8;
    const bool inside = at < a.head_dim;
    const int per_warp = 32 / lanes;
    const int vectors = a.q_heads + 2 * a.kv_heads;
    for (int first = warp * per_warp; first < vectors; first += (int)blockDim.x / 32 * per_warp) {
        const int i = first + lane / lanes;
        const bool active = i < vectors && inside;
        const int kind = i < a.q_heads ? 0 : i < a.q_heads + a.kv_heads ? 1 : 2;
        const int head = i - (kind == 0 ? 0 : kind == 1 ? a.q_heads : a.q_heads + a.kv_heads);
        const int64_t *st = kind == 0 ? a.q_st : kind == 1 ? a.k_st : a.v_st;
        const uint16_t *src = static_cast<const uint16_t *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                              t0 * st[0] + head * st[1];
        // where a value's other one lies (kind 2 does not turn)
        const bool turns = kind != 2 && at < a.rot_dim;
        P own[kAppendTokens], other[kAppendTokens];
        auto other_at = [&](int x) { return x < half ? x + half : x < a.rot_dim ? x - half : x; };
#pragma unroll
        for (int w = 0; w < kAppendTokens; ++w) {
            own[w] = other[w] = P{};
            if (!active || w >= here) continue;
            const uint16_t *from = src + w * st[0];
            own[w] = *reinterpret_cast<const P *>(from + at);
            if (kTurn == kPackTurn && turns) other[w] = *reinterpret_cast<const P *>(from + other_at(at));
            if (kTurn == kPairTurn && turns)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    other[w].x[e] = *reinterpret_cast<const uint32_t *>(from + other_at(at + 2 * e));
        }
        __syncwarp();  // q_out may be q: a head's loads come before its stores
        const void *norm = kind == 0 ? A.q_norm : kind == 1 ? A.k_norm : nullptr;
        const bool any_norm = A.q_norm || A.k_norm;
        float wo[8], wx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) wo[e] = wx[e] = 1.f;
        if (norm && active) {
            weights_at<T>(norm, A.norm_f32, at, wo);
            if (kTurn == kPackTurn && turns) weights_at<T>(norm, A.norm_f32, other_at(at), wx);
            if (kTurn == kPairTurn && turns)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int x = other_at(at + (e & ~1)) + (e & 1);
                    wx[e] = A.norm_f32 ? __ldg(static_cast<const float *>(norm) + x)
                                       : to_f32<T>(static_cast<const T *>(norm)[x]);
                }
        }
#pragma unroll
        for (int w = 0; w < kAppendTokens; ++w) {
            if (w >= here) break;
            float y[8], z[8];
            unpack<T>(own[w], y);
            unpack<T>(other[w], z);
            if (any_norm) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(y[e], y[e], sum);
                for (int d = lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float f = norm ? rsqrtf(sum / (float)a.head_dim + A.eps) : 1.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] *= f * wo[e];
                    z[e] *= f * wx[e];
                }
            }
            if (turns) {
                if (kTurn == kAdjacentTurn) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        if (at + e < a.rot_dim) {
                            const float2 c = cs[w][(at + e) / 2];
                            const float u = y[e] * c.x - y[e + 1] * c.y, v = y[e] * c.y + y[e + 1] * c.x;
                            y[e] = u;
                            y[e + 1] = v;
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int x = at + e;
                        if (x < half) {
                            const float2 c = cs[w][x];
                            y[e] = y[e] * c.x - z[e] * c.y;
                        } else if (x < a.rot_dim) {
                            const float2 c = cs[w][x - half];
                            y[e] = z[e] * c.y + y[e] * c.x;
                        }
                    }
                }
            }
            const RowPlace &p = place[w];
            if (kind == 0 || !kEight) {
                if (active && p.known) {
                    P o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o.x[e] = bits_of(y[2 * e], y[2 * e + 1], T());
                    if (kind == 0)
                        *reinterpret_cast<P *>(static_cast<uint16_t *>(a.q_out) + (t0 + w) * a.o_st[0] +
                                               head * a.o_st[1] + at) = o;
                    else if (p.k >= 0)
                        *reinterpret_cast<P *>(static_cast<uint16_t *>(kind == 1 ? a.k_cache : a.v_cache) +
                                               (kind == 1 ? p.k + head * a.kc_st[2] : p.v + head * a.vc_st[2]) +
                                               at) = o;
                }
            }
            if (kEight) {
                // the bits of magnitudes order as they do; NaN and infinity lie above
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
                for (int d = lanes / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                if (kind != 0 && active && p.k >= 0) {
                    const bool finite = top < 0x7f800000u;
                    const int e8 = scale_exponent(top);
                    const float f = power_of_two(-e8);
                    uint2 o = make_uint2(0, 0);
                    if (finite) {
                        o.x = codes_of(y[0] * f, y[1] * f) | codes_of(y[2] * f, y[3] * f) << 16;
                        o.y = codes_of(y[4] * f, y[5] * f) | codes_of(y[6] * f, y[7] * f) << 16;
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(kind == 1 ? a.k_cache : a.v_cache) +
                                               (kind == 1 ? p.k + head * a.kc_st[2] : p.v + head * a.vc_st[2]) +
                                               at) = o;
                    if (sub == 0) {
                        uint8_t *to = kind == 1 ? A.scales.k + p.ks + head * A.scales.k_st[2]
                                                : A.scales.v + p.vs + head * A.scales.v_st[2];
                        *to = (uint8_t)(finite ? e8 + 127 : kScaleNan);
                    }
                }
            }
        }
    }
}

// ---- the way back -----------------------------------------------------------------

constexpr int kReadThreads = 256;
constexpr int kReadRows = 16;  // rows per block at most

struct ReadParams {
    Batch batch;
    FastDiv by_page, by_chunks, by_heads;  // 16-value chunks of a head; kv heads
    const void *k_cache, *v_cache;
    int64_t kc_st[3], vc_st[3];
    Scales scales;
    void *k, *v;
    int64_t k_st[2], v_st[2];   // row and head strides of the outputs, elements
    int32_t kv_heads, head_dim, chunks;
    // Whole sequences into pages of their own (page i of sequence b is page b *
    // max_pages + i, slots in order) for the 16-bit attention: `table` is that page
    // table; slots before every row's window are left out.
    int32_t *table;
    int32_t window;
};

// Sixteen codes times a scale, in 16 bits.
template <class T, bool kSaturate>
__device__ __forceinline__ void expand(uint4 c, float f, uint4 &lo, uint4 &hi) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float2 a = values_of(w[e] & 0xffffu), b = values_of(w[e] >> 16);
        a.x *= f, a.y *= f, b.x *= f, b.y *= f;
        if (kSaturate) {  // fp16: a vector's largest may have been rounded past 65504
            a.x = fminf(fmaxf(a.x, -65504.f), 65504.f), a.y = fminf(fmaxf(a.y, -65504.f), 65504.f);
            b.x = fminf(fmaxf(b.x, -65504.f), 65504.f), b.y = fminf(fmaxf(b.y, -65504.f), 65504.f);
        }
        o[2 * e] = bits_of(a.x, a.y, T());
        o[2 * e + 1] = bits_of(b.x, b.y, T());
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

template <class T, bool kEight, bool kPages>
__global__ void __launch_bounds__(kReadThreads)
    read_kernel(const __grid_constant__ ReadParams A, int per_block) {
    __shared__ RowPlace place[kReadRows];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t r0 = (int64_t)blockIdx.x * per_block;
    wait_for_primary_grid();
    int here;
    if (kPages) {
        // a block's rows lie in one sequence's pages (per_block divides page_size)
        const int64_t per_sequence = (int64_t)A.batch.max_pages * A.batch.page_size;
        const int32_t b = (int32_t)(r0 / per_sequence);
        const int32_t slot0 = (int32_t)(r0 - b * per_sequence);
        const Sequence s = load_sequence(A.batch, b);
        here = per_block;
        if (s.bad || s.n == 0 || slot0 >= s.len) return;
        const int32_t first = A.window > 0 ? s.len - s.n - A.window + 1 : 0;
        const int32_t pg = A.by_page.div(slot0);
        if (threadIdx.x == 0 && slot0 - pg * A.batch.page_size == 0)
            A.table[(int64_t)b * A.batch.max_pages + pg] = b * A.batch.max_pages + pg;
        if ((pg + 1) * A.batch.page_size <= first) return;  // (the attention skips whole pages only)
        if (warp == 0) {
            const int32_t id = __ldg(A.batch.pages + b * A.batch.pages_stride + pg);
            const bool ok = id >= 0 && id < A.batch.num_pages;
            if (!ok && lane == 0) atomicOr(A.batch.status, SV_STATUS_BAD_PAGE);
            for (int w = lane; w < here; w += 32) {
                const int64_t in = slot0 + w - pg * A.batch.page_size;
                RowPlace p = {-1, -1, -1, -1, slot0 + w < s.len};
                if (ok && p.known) {
                    p.k = id * A.kc_st[0] + in * A.kc_st[1];
                    p.v = id * A.vc_st[0] + in * A.vc_st[1];
                    p.ks = id * A.scales.k_st[0] + in * A.scales.k_st[1];
                    p.vs = id * A.scales.v_st[0] + in * A.scales.v_st[1];
                }
                place[w] = p;
            }
        }
    } else {
        here = (int)min((int64_t)per_block, A.batch.tokens - r0);
        for (int w = warp; w < here; w += kReadThreads / 32) {
            int64_t pos;
            const RowPlace p = place_of(A.batch, A.by_page, A.kc_st, A.vc_st, A.scales, (int32_t)(r0 + w), pos, lane);
            if (lane == 0) place[w] = p;
        }
    }
    __syncthreads();

    // items: (row, key or value, head, chunk of 16 values), four loads in flight
    const int per_row = 2 * A.kv_heads * A.chunks;
    const int items = here * per_row;
    constexpr int kAhead = 4;
    for (int i0 = threadIdx.x; i0 < items; i0 += kAhead * kReadThreads) {
        uint4 x[kAhead], x2[kAhead];
        uint32_t scale[kAhead];
        uint16_t *to[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int i = i0 + e * kReadThreads;
            to[e] = nullptr;
            x[e] = x2[e] = make_uint4(0, 0, 0, 0);
            scale[e] = 127;
            if (i >= items) continue;
            const int head_of_all = A.by_chunks.div(i), ch = i - head_of_all * A.chunks;
            const int row_and_kind = A.by_heads.div(head_of_all), h = head_of_all - row_and_kind * A.kv_heads;
            const int w = row_and_kind >> 1, kind = row_and_kind & 1;
            const RowPlace &p = place[w];
            if (!p.known) continue;
            to[e] = static_cast<uint16_t *>(kind ? A.v : A.k) + (r0 + w) * (kind ? A.v_st[0] : A.k_st[0]) +
                    h * (kind ? A.v_st[1] : A.k_st[1]) + ch * 16;
            if (p.k < 0) continue;  // no such slot or page: zeros
            const int64_t from = (kind ? p.v + h * A.vc_st[2] : p.k + h * A.kc_st[2]) + ch * 16;
            if (kEight) {
                x[e] = __ldg(reinterpret_cast<const uint4 *>(
                    static_cast<const uint8_t *>(kind ? A.v_cache : A.k_cache) + from));
                scale[e] = __ldg(kind ? A.scales.v + p.vs + h * A.scales.v_st[2]
                                      : A.scales.k + p.ks + h * A.scales.k_st[2]);
            } else {
                const uint4 *at = reinterpret_cast<const uint4 *>(
                    static_cast<const uint16_t *>(kind ? A.v_cache : A.k_cache) + from);
                x[e] = __ldg(at);
                // (head_dim a multiple of 8: a head's last chunk may be half a one)
                if (ch * 16 + 8 < A.head_dim) x2[e] = __ldg(at + 1);
            }
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            if (!to[e]) continue;
            if (kEight) expand<T, kPages && __is_same(T, __half)>(x[e], scale_of(scale[e]), x[e], x2[e]);
            reinterpret_cast<uint4 *>(to[e])[0] = x[e];
            if (kEight) {
                reinterpret_cast<uint4 *>(to[e])[1] = x2[e];
            } else {
                const int i = i0 + e * kReadThreads;
                const int ch = i - A.by_chunks.div(i) * A.chunks;
                if (ch * 16 + 8 < A.head_dim) reinterpret_cast<uint4 *>(to[e])[1] = x2[e];
            }
        }
    }
}

}  // namespace sv
