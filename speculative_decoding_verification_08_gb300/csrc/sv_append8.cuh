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
// Bound by memory: a group of lanes (a power of two, 16 values each) holds a head's
// vector in registers, a pair's two values in one lane wherever pairs start on packs of
// 8, so that sums and maxima are a few shuffles and nothing is loaded twice.  Angles
// are fixed-point: a frequency in turns as a 64-bit fraction, once a block (fp64 runs at
// 1/64 of fp32 here), so that position times frequency modulo a turn is one integer
// product.  They are good to 2^-26 of a turn (the conversion to fp32) and position times
// frequency (in turns) times 2^-52 (the frequency's own rounding in fp64).
//
// Measured (32 query heads over 8 of 128, bf16, unless said otherwise):
//   18,157 tokens of prompts into 8 bits, half of each head turned: 81 us, 5.1 TB/s (90
//     without the next token's loads ahead and with 8 tokens a block; 258 with 8 values to
//     a lane, each pair's other value loaded beside it, and fp64 angles); 63 % of the issue
//     slots are taken, a third of the warps fit (80 registers; 93 with 64);
//   24,425 tokens normed, 16 over 4 heads of 96 in fp16, adjacent pairs: 60 us, 3.8 TB/s:
//     6 of 8 lanes have values, and the same;
//   rounds of 256 x 6 tokens: 12 to 14 us normed, 13 normed to 8 bits, 3 of it launch and
//     lookup; one token 9 to 11, all of it the call's host time.
#pragma once

#include "sv_append.cuh"
#include "sv_pairs.cuh"

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
    int32_t position;
};

// Row t of the token arrays: its slot's places, by a whole warp.  pos: its slot.
__device__ __forceinline__ RowPlace place_of(const Batch &A, const FastDiv &by_page, const int64_t *kc_st,
                                             const int64_t *vc_st, const Scales &S, int32_t t, int64_t &pos,
                                             int lane) {
    RowPlace p = {-1, -1, -1, -1, 0, 0};
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

constexpr int kNormTokens = 16;  // tokens per block at most

// How pairs lie.  kPackTurn: both halves start on a pack (rot_dim a multiple of 16) and
// lane l < rot_dim / 16 has packs l of both; kAdjacentTurn: within a pack (or nothing
// turns); kPairTurn: a pair's other value is loaded beside the lane's own.
enum Turning { kPackTurn, kPairTurn, kAdjacentTurn };

// A pack's eight values as four pairs of floats.
template <class T>
__device__ __forceinline__ void unpack(const Pack<8> &p, uint64_t (&y)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = pair_of(p.x[e], T());
        y[e] = pair2(f.x, f.y);
    }
}

// Weights i and i + 1.
template <class T>
__device__ __forceinline__ uint64_t weights_at(const void *w, bool f32, int i) {
    return f32 ? pair2(__ldg(static_cast<const float *>(w) + i), __ldg(static_cast<const float *>(w) + i + 1))
               : pair2(to_f32<T>(static_cast<const T *>(w)[i]), to_f32<T>(static_cast<const T *>(w)[i + 1]));
}

template <class T, bool kEight, Turning kTurn>
__global__ void __launch_bounds__(kAppendThreads, kTurn == kPairTurn ? 2 : 3)
    append_norm_kernel(const __grid_constant__ AppendNormParams A, int per_block, int lanes) {
    __shared__ RowPlace place[kNormTokens];
    __shared__ __align__(16) float cosines[kNormTokens][kMaxHeadDim / 2], sines[kNormTokens][kMaxHeadDim / 2];
    __shared__ uint64_t turn_of[kMaxHeadDim / 2];
    typedef Pack<8> P;
    const AppendParams &a = A.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t t0 = (int32_t)blockIdx.x * per_block;
    const int here = min(per_block, a.batch.tokens - t0);
    const int half = a.rot_dim / 2;

    // `lanes` lanes to a vector, a warp's vectors side by side; each lane's two packs
    const int sub = lane % lanes;
    const bool pairs = kTurn == kPackTurn && sub * 16 < a.rot_dim;
    const int at0 = pairs ? sub * 8 : sub * 16, at1 = pairs ? half + at0 : at0 + 8;
    const bool in0 = at0 < a.head_dim, in1 = at1 < a.head_dim;
    const int per_warp = 32 / lanes, stride = (int)blockDim.x / 32 * per_warp;
    const int vectors = a.q_heads + 2 * a.kv_heads;

    wait_for_primary_grid();
    for (int e = threadIdx.x; e < half; e += (int)blockDim.x) {
        const double turns = __ldg(a.inv_freq + e) * 0.15915494309189535;
        turn_of[e] = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
    }
    for (int w = warp; w < here; w += (int)blockDim.x / 32) {
        int64_t slot;
        RowPlace p = place_of(a.batch, a.by_page, a.kc_st, a.vc_st, A.scales, t0 + w, slot, lane);
        p.position = a.positions ? __ldg(a.positions + t0 + w) : (int32_t)slot;
        if (lane == 0) place[w] = p;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < here * half; i += (int)blockDim.x) {
        const int w = i / half, e = i - w * half;
        const uint64_t turns = (uint64_t)(int64_t)place[w].position * turn_of[e];
        float s, c;
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
        cosines[w][e] = c;
        sines[w][e] = s;
    }
    __syncthreads();

    const bool any_norm = A.q_norm || A.k_norm;
    const float inv_dim = 1.f / (float)a.head_dim;
    int weights_of = -1;
    uint64_t w0[4], w1[4], z0[4], z1[4];  // norms of the lane's values, and of their others
    for (int first = warp * per_warp; first < vectors; first += stride) {
        const int i = first + lane / lanes;
        const bool active = i < vectors;
        const int kind = i < a.q_heads ? 0 : i < a.q_heads + a.kv_heads ? 1 : 2;
        const int head = i - (kind == 0 ? 0 : kind == 1 ? a.q_heads : a.q_heads + a.kv_heads);
        const int64_t step = kind == 0 ? a.q_st[0] : kind == 1 ? a.k_st[0] : a.v_st[0];
        const uint16_t *src = static_cast<const uint16_t *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + t0 * step +
                              head * (kind == 0 ? a.q_st[1] : kind == 1 ? a.k_st[1] : a.v_st[1]);
        const void *norm = kind == 0 ? A.q_norm : kind == 1 ? A.k_norm : nullptr;
        const bool turns = kind != 2 && a.rot_dim > 0;
        auto other_at = [&](int x) { return x < half ? x + half : x < a.rot_dim ? x - half : x; };
        if (any_norm && weights_of != kind) {
            weights_of = kind;
#pragma unroll
            for (int e = 0; e < 4; ++e) w0[e] = w1[e] = z0[e] = z1[e] = pair2(1.f, 1.f);
            if (norm)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (in0) w0[e] = weights_at<T>(norm, A.norm_f32, at0 + 2 * e);
                    if (in1) w1[e] = weights_at<T>(norm, A.norm_f32, at1 + 2 * e);
                    if (kTurn == kPairTurn) {
                        if (in0) z0[e] = weights_at<T>(norm, A.norm_f32, other_at(at0 + 2 * e));
                        if (in1) z1[e] = weights_at<T>(norm, A.norm_f32, other_at(at1 + 2 * e));
                    }
                }
        }
        // the next token's values are on their way while one is worked on
        struct Values {
            P own[2], other[2];
        };
        auto load = [&](int w) -> Values {
            Values v{};
            if (!active || w >= here) return v;
            const uint16_t *from = src + w * step;
            if (in0) v.own[0] = *reinterpret_cast<const P *>(from + at0);
            if (in1) v.own[1] = *reinterpret_cast<const P *>(from + at1);
            if (kTurn == kPairTurn && turns)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (in0) v.other[0].x[e] = *reinterpret_cast<const uint32_t *>(from + other_at(at0 + 2 * e));
                    if (in1) v.other[1].x[e] = *reinterpret_cast<const uint32_t *>(from + other_at(at1 + 2 * e));
                }
            return v;
        };
        Values now = load(0);
#pragma unroll 1
        for (int w = 0; w < here; ++w) {
            const Values next = load(w + 1);
            __syncwarp();  // q_out may be q: a head's loads come before its stores
            {
                uint64_t y0[4], y1[4], o0[4], o1[4];
                unpack<T>(now.own[0], y0);
                unpack<T>(now.own[1], y1);
                if (kTurn == kPairTurn) {
                    unpack<T>(now.other[0], o0);
                    unpack<T>(now.other[1], o1);
                }
                if (any_norm) {
                    uint64_t sum2 = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum2 = fma2(y1[e], y1[e], fma2(y0[e], y0[e], sum2));
                    float u, v;
                    unpair2(sum2, u, v);
                    float sum = u + v;
                    for (int d = lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    const float f = norm ? rsqrtf(fmaf(sum, inv_dim, A.eps)) : 1.f;
                    const uint64_t f2 = pair2(f, f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y0[e] = mul2(y0[e], mul2(f2, w0[e]));
                        y1[e] = mul2(y1[e], mul2(f2, w1[e]));
                        if (kTurn == kPairTurn) {
                            o0[e] = mul2(o0[e], mul2(f2, z0[e]));
                            o1[e] = mul2(o1[e], mul2(f2, z1[e]));
                        }
                    }
                }
                if (kTurn == kPackTurn && turns && pairs) {
                    // (a, c) -> (a cos - c sin, a sin + c cos)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float4 co = *reinterpret_cast<const float4 *>(&cosines[w][at0 + 2 * e]);
                        const float4 si = *reinterpret_cast<const float4 *>(&sines[w][at0 + 2 * e]);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint64_t c2 = x ? pair2(co.z, co.w) : pair2(co.x, co.y);
                            const uint64_t s2 = x ? pair2(si.z, si.w) : pair2(si.x, si.y);
                            const uint64_t m2 = x ? pair2(-si.z, -si.w) : pair2(-si.x, -si.y);
                            const uint64_t p = y0[e + x], q = y1[e + x];
                            y0[e + x] = fma2(p, c2, mul2(q, m2));
                            y1[e + x] = fma2(p, s2, mul2(q, c2));
                        }
                    }
                }
                if (kTurn == kAdjacentTurn && turns) {
#pragma unroll
                    for (int pack = 0; pack < 2; ++pack) {
                        const int at = pack ? at1 : at0;
                        if (at >= a.rot_dim) continue;
                        uint64_t(&y)[4] = pack ? y1 : y0;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (at + 2 * e < a.rot_dim) {
                                const float c = cosines[w][at / 2 + e], s = sines[w][at / 2 + e];
                                float p, q;
                                unpair2(y[e], p, q);
                                y[e] = pair2(p * c - q * s, p * s + q * c);
                            }
                    }
                }
                if (kTurn == kPairTurn && turns) {
#pragma unroll
                    for (int pack = 0; pack < 2; ++pack)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int x = (pack ? at1 : at0) + 2 * e;  // x and x + 1 lie in one half
                            if (x >= a.rot_dim) continue;
                            uint64_t &y = pack ? y1[e] : y0[e];
                            const uint64_t z = pack ? o1[e] : o0[e];
                            const int j = x < half ? x : x - half;
                            const uint64_t c2 = pair2(cosines[w][j], cosines[w][j + 1]);
                            const float sign = x < half ? -1.f : 1.f;
                            y = fma2(y, c2, mul2(z, pair2(sign * sines[w][j], sign * sines[w][j + 1])));
                        }
                }
                const RowPlace &p = place[w];
                if (kind == 0 || !kEight) {
                    if (active && p.known) {
                        uint16_t *to = kind == 0 ? static_cast<uint16_t *>(a.q_out) + (t0 + w) * a.o_st[0] + head * a.o_st[1]
                                       : kind == 1 ? static_cast<uint16_t *>(a.k_cache) + p.k + head * a.kc_st[2]
                                                   : static_cast<uint16_t *>(a.v_cache) + p.v + head * a.vc_st[2];
                        if (kind == 0 || p.k >= 0) {
                            P o;
#pragma unroll
                            for (int pack = 0; pack < 2; ++pack) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float u, v;
                                    unpair2(pack ? y1[e] : y0[e], u, v);
                                    o.x[e] = bits_of(u, v, T());
                                }
                                if (pack ? in1 : in0) *reinterpret_cast<P *>(to + (pack ? at1 : at0)) = o;
                            }
                        }
                    }
                }
                if (kEight) {
                    float top = 0.f;
                    uint64_t zero = 0;  // NaN where a value is not finite
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float u, v;
                        unpair2(y0[e], u, v);
                        top = max3(top, fabsf(u), fabsf(v));
                        unpair2(y1[e], u, v);
                        top = max3(top, fabsf(u), fabsf(v));
                        zero = fma2(y1[e], 0, fma2(y0[e], 0, zero));
                    }
                    float u, v;
                    unpair2(zero, u, v);
                    const unsigned bad = __ballot_sync(0xffffffffu, !(u + v == 0.f));
                    for (int d = lanes / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    if (kind != 0 && active && p.k >= 0) {
                        const unsigned group = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1) << (lane - sub);
                        const bool finite = (bad & group) == 0;
                        const int e8 = scale_exponent(__float_as_uint(top));
                        const uint64_t f2 = pair2(power_of_two(-e8), power_of_two(-e8));
                        uint8_t *to = static_cast<uint8_t *>(kind == 1 ? a.k_cache : a.v_cache) +
                                      (kind == 1 ? p.k + head * a.kc_st[2] : p.v + head * a.vc_st[2]);
#pragma unroll
                        for (int pack = 0; pack < 2; ++pack) {
                            uint32_t c[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                unpair2(mul2(pack ? y1[e] : y0[e], f2), u, v);
                                c[e] = finite ? codes_of(u, v) : 0u;
                            }
                            if (pack ? in1 : in0)
                                *reinterpret_cast<uint2 *>(to + (pack ? at1 : at0)) =
                                    make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                        }
                        if (sub == 0) {
                            uint8_t *byte = kind == 1 ? A.scales.k + p.ks + head * A.scales.k_st[2]
                                                      : A.scales.v + p.vs + head * A.scales.v_st[2];
                            *byte = (uint8_t)(finite ? e8 + 127 : kScaleNan);
                        }
                    }
                }
            }
            now = next;
        }
    }
}

// ---- the way back -----------------------------------------------------------------
//
// Bound by memory: a thread takes 16 codes to 32 bytes, four such loads in flight.
// 64 sequences of 156,896 rows in all, 8 heads of 128: 157 us, 6.2 TB/s.

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
    // Whole sequences into pages of 16 bits, slots in order, for the 16-bit attention:
    // page i of sequence b is page b * max_pages + i, and `table` that page table; or
    // (NULL) pages keep their numbers (one that sequences share is written by each, alike).
    // Slots before every row's window are left out.  A key or value that is NaN becomes a
    // NaN key, whose score is NaN for the rows that see it and masked for others.
    int32_t *table;
    int32_t window;
};

// x within fp16's largest; NaN stays NaN.
__device__ __forceinline__ float fp16_range(float x) {
    asm("{ .reg .f32 y; min.NaN.f32 y, %0, %1; max.NaN.f32 %0, y, %2; }"
        : "+f"(x)
        : "f"(65504.f), "f"(-65504.f));
    return x;
}

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
            a.x = fp16_range(a.x), a.y = fp16_range(a.y);
            b.x = fp16_range(b.x), b.y = fp16_range(b.y);
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
    int64_t row0 = r0;  // first row of the outputs
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
        if (A.table && threadIdx.x == 0 && slot0 - pg * A.batch.page_size == 0)
            A.table[(int64_t)b * A.batch.max_pages + pg] = b * A.batch.max_pages + pg;
        if ((pg + 1) * A.batch.page_size <= first) return;  // (the attention skips whole pages only)
        const int32_t id = __ldg(A.batch.pages + b * A.batch.pages_stride + pg);
        const bool ok = id >= 0 && id < A.batch.num_pages;
        if (!ok && threadIdx.x == 0) atomicOr(A.batch.status, SV_STATUS_BAD_PAGE);
        if (!A.table) {
            if (!ok) return;  // (zeros to the attention, too)
            row0 = (int64_t)id * A.batch.page_size + (slot0 - pg * A.batch.page_size);
        }
        if (warp == 0) {
            for (int w = lane; w < here; w += 32) {
                const int64_t in = slot0 + w - pg * A.batch.page_size;
                RowPlace p = {-1, -1, -1, -1, slot0 + w < s.len, 0};
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
        uint32_t scale[kAhead], value_scale[kAhead];  // (kPages: also a key's value's)
        uint16_t *to[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int i = i0 + e * kReadThreads;
            to[e] = nullptr;
            x[e] = x2[e] = make_uint4(0, 0, 0, 0);
            scale[e] = value_scale[e] = 127;
            if (i >= items) continue;
            const int head_of_all = A.by_chunks.div(i), ch = i - head_of_all * A.chunks;
            const int row_and_kind = A.by_heads.div(head_of_all), h = head_of_all - row_and_kind * A.kv_heads;
            const int w = row_and_kind >> 1, kind = row_and_kind & 1;
            const RowPlace &p = place[w];
            if (!p.known) continue;
            to[e] = static_cast<uint16_t *>(kind ? A.v : A.k) + (row0 + w) * (kind ? A.v_st[0] : A.k_st[0]) +
                    h * (kind ? A.v_st[1] : A.k_st[1]) + ch * 16;
            if (p.k < 0) continue;  // no such slot or page: zeros
            const int64_t from = (kind ? p.v + h * A.vc_st[2] : p.k + h * A.kc_st[2]) + ch * 16;
            if (kEight) {
                x[e] = __ldg(reinterpret_cast<const uint4 *>(
                    static_cast<const uint8_t *>(kind ? A.v_cache : A.k_cache) + from));
                scale[e] = __ldg(kind ? A.scales.v + p.vs + h * A.scales.v_st[2]
                                      : A.scales.k + p.ks + h * A.scales.k_st[2]);
                if (kPages) value_scale[e] = __ldg(A.scales.v + p.vs + h * A.scales.v_st[2]);
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
            if (kPages && value_scale[e] == kScaleNan) {
                // The 16-bit attention wants finite values in slots that rows do not see
                // (weights of zero times them must be zero), but masks scores: a vector
                // that is NaN is left to the key, and the value is zeros.
                const int i = i0 + e * kReadThreads;
                const bool key = (A.by_heads.div(A.by_chunks.div(i)) & 1) == 0;
                if (!key) x[e] = make_uint4(0, 0, 0, 0);
                scale[e] = key ? kScaleNan : 127;
            }
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
