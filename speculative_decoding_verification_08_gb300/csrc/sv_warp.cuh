// sv_warp.cuh -- the warp of logits into probability rows (temperature, top-k,
// top-p, min-p) and draws from them.
//
// A cluster of CTAs takes a row and keeps it in its shared memory (a slice per
// CTA), so the row is read from memory once whatever the filters need; rows of a
// call without filters go through plain_kernel at the end of this file.
//
// Every filter keeps a prefix of the row's order (logit descending, index
// ascending), so the kept set is one threshold on the 64-bit composite
// (ordered logit bits, ~index); min-p gives its logit directly.  Top-k and
// top-p find theirs in two sweeps: a histogram over the distance from the
// maximum (counts, or masses in fixed point, whose integer sums do not depend
// on the order of the atomics) narrows the border to a bin or two, then the
// elements of those bins are gathered, ranked, and the border is settled on
// exact values.  A border bin too full to gather (rows of equal logits) is
// settled by bisection of the composite instead, in up to 64 sweeps of the row: 256
// rows of 128256 fp32 rounded to whole numbers take 11.7 ms with top-p (274 us
// unrounded), 8.1 with a top-k of 20000 (315 us), one row of 32000 0.88 (24 us).
//
// Masses decide which tokens stay and which one is drawn, and must give the
// answers of a 64-bit evaluation.  fp64 runs at 1/64 of the fp32 rate here, so
// a weight exp((z - max) / T) is formed as a pair of floats (weight()): the
// exponent and the table-and-polynomial value keep their rounding errors in
// the low part.
//
// Bound by instructions and by the serial ends of a row's phases (search of the
// border, ranking, search of the drawn element), not by memory: 256 rows of
// 128256 fp32 with every filter, token and probabilities take 162 us (1.6 TB/s;
// 39 us at the memory's rate), 768 bf16 rows with top-p and min-p 368 us (87).
// Three CTAs to an SM hide part of one another's serial ends.
#pragma once

#include <cooperative_groups.h>
#include <string.h>

#include <type_traits>

#include "sv_barrier.cuh"
#include "sv_cache.cuh"

namespace sv {

constexpr int kMaxWarps = 32;
constexpr int kWarpMaxCluster = 8;
constexpr int kBins = 1024;            // of a histogram of counts and masses; of one alone twice as many
constexpr float kRangeOctaves = 40.f;  // the histogram's reach below the maximum
constexpr float kColdest = 1e-36f, kHottest = 1e36f;  // temperatures
constexpr float kTiny = 1e-35f;        // no histogram spans less
static_assert(kColdest * kRangeOctaves * 0.69f > kTiny, "the coldest row's reach");
constexpr float kMagic = 8388608.f;    // 2^23: adding it rounds to a whole number in the low bits
constexpr int kPlainThreads = 256;
constexpr int kLocalList = 160;        // border elements one CTA may gather
constexpr int kList = 1024;            // and the row
// Top-k up to here is settled on a list alone when top-p follows (a CTA's list
// holds it even when all of it lies in one slice).
constexpr int kFew = 128;
constexpr int kShared = 512;           // of them, ranked by the whole cluster

struct WarpParams {
    const void *z;
    int64_t zs, V;
    const float *temperature, *top_p, *min_p;
    const int32_t *top_k;
    const double *u;
    int32_t *token;
    float *probs;
    int64_t ps;
    uint32_t *status;
    int32_t R, slice;   // elements per CTA, a multiple of 16
    int32_t cached;     // 16-byte words of a slice that fit in shared memory
};

// Floats in order: a < b iff ordered(a) < ordered(b) (-0 and 0 alike).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ uint64_t composite(float z, int64_t v) {
    return ((uint64_t)ordered(z) << 32) | (uint32_t)~(uint32_t)v;
}

// 2^(j / 32), j = -16..15, as hi + lo (correctly rounded); every CTA copies it
// to shared memory, where its lanes read different entries at once.
__constant__ float2 kPow2[32] = {
    {0.707106769f, 1.21016175e-08f}, {0.722590387f, 1.66209997e-08f},
    {0.738413095f, -2.25044943e-08f}, {0.754582226f, -1.24796866e-08f},
    {0.771105409f, 4.03545242e-09f}, {0.787990451f, -2.83051271e-08f},
    {0.805245161f, 4.91810859e-09f}, {0.822877765f, -2.56248605e-08f},
    {0.840896428f, -1.23776633e-08f}, {0.859309673f, -2.4248088e-08f},
    {0.878126085f, -4.61788519e-09f}, {0.897354543f, -5.70752245e-09f},
    {0.917004049f, -5.61963898e-09f}, {0.93708384f, -2.33150281e-08f},
    {0.957603276f, 4.92266405e-09f}, {0.978572071f, -8.51090221e-09f},
    {1.f, 0.f}, {1.0218972f, -4.81155986e-08f},
    {1.04427373f, 4.83347016e-08f}, {1.06714046f, -5.93375198e-08f},
    {1.09050775f, -1.30775399e-08f}, {1.1143868f, -5.43554002e-08f},
    {1.13878858f, 5.38622231e-08f}, {1.1637249f, -4.05144149e-08f},
    {1.18920708f, 3.79763527e-08f}, {1.21524739f, -3.26739489e-08f},
    {1.24185777f, 4.4968381e-08f}, {1.26905096f, 1.41933332e-09f},
    {1.29683959f, -4.01899953e-08f}, {1.32523668f, -3.49637332e-08f},
    {1.35425556f, -1.01233493e-08f}, {1.38390994f, -5.87557736e-08f}};

struct ExpTable {
    float x[32], y[32];   // (columns: 32 lanes' lookups then meet no bank conflicts)
};

struct RowScale {
    float m;          // row maximum
    float ih, il;     // 1 / temperature as hi + lo
    float ch, cl;     // log2(e) / temperature
    float floor;      // -85 T: what lies further down weighs nothing
};

// exp(x), x = (z - max) / T, as hi + lo, to about 2^-35 relative; 0 below exp(-85).
//   z - max = d + dl and x = xh + xl to twice the fp32 digits; x = k ln2/32 + r
//   with |r| < 0.011; 2^(k/32) from the table, exp(r) - 1 = r + r^2/2 + r^3/6
//   + r^4/24.
__device__ __forceinline__ float2 weight(float z, const RowScale &S, const ExpTable &tab) {
    const float far = z - S.m, b = far - z;
    const bool in = far >= S.floor;
    const float d = in ? far : S.floor;
    const float dl = in ? (z - (far - b)) - (S.m + b) : 0.f;
    const float xh = d * S.ih;
    const float xl = fmaf(dl, S.ih, fmaf(d, S.il, fmaf(d, S.ih, -xh)));
    const float km = fmaf(xh, 46.1662413f, 12582912.f);  // 1.5 * 2^23: the low bits hold k
    const float k = km - 12582912.f;
    const float r = fmaf(k, -0.0216608495f, xh);   // exact: few bits are left
    const float rl = fmaf(k, 5.95204441e-11f, xl), q = r + rl;
    const float t = fmaf(q * q, fmaf(q, fmaf(q, 4.16666667e-2f, 0.166666667f), 0.5f), rl);
    const int ki = __float_as_int(km) + 16;
    const float2 T = make_float2(tab.x[ki & 31], tab.y[ki & 31]);
    const float scale = in ? __uint_as_float(((uint32_t)ki >> 5 << 23) + 0x3f800000u) : 0.f;
    const float v = T.x * r, vl = fmaf(T.x, r, -v), u = fmaf(T.x, t, fmaf(T.y, r, T.y));
    const float h = T.x + v;
    const float l = (v - (h - T.x)) + (vl + u);
    return make_float2(h * scale, l * scale);
}

__device__ __noinline__ float2 weight_of(float z, RowScale S, const ExpTable *tab) {
    return weight(z, S, *tab);
}

// Sums of weights as pairs of floats (fp64 runs at 1/64 of the fp32 rate here):
// relative errors near 2^-46.
struct dd2 {
    float h, l;
};

__device__ __forceinline__ dd2 norm2(float h, float l) {
    const float s = h + l;
    return {s, l - (s - h)};
}
__device__ __forceinline__ dd2 add_dd(dd2 a, dd2 b) {
    const float s = a.h + b.h, x = s - a.h;
    return norm2(s, ((a.h - (s - x)) + (b.h - x)) + (a.l + b.l));
}
__device__ __forceinline__ dd2 mul_dd(dd2 a, dd2 b) {
    const float p = a.h * b.h;
    return norm2(p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h));
}
__device__ __forceinline__ bool less_dd(dd2 a, dd2 b) {
    return a.h < b.h || (a.h == b.h && a.l < b.l);
}
__device__ __forceinline__ dd2 shfl_dd(dd2 a, int lane) {
    return {__shfl_sync(0xffffffffu, a.h, lane), __shfl_sync(0xffffffffu, a.l, lane)};
}
// The sum over the warp, the same in every lane (the steps are symmetric).
__device__ __forceinline__ dd2 warp_sum_dd(dd2 a) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        a = add_dd(a, {__shfl_xor_sync(0xffffffffu, a.h, d), __shfl_xor_sync(0xffffffffu, a.l, d)});
    return a;
}
__device__ __forceinline__ dd2 warp_scan_dd(dd2 a, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const dd2 o = {__shfl_up_sync(0xffffffffu, a.h, d), __shfl_up_sync(0xffffffffu, a.l, d)};
        const dd2 s = add_dd(o, a);
        a = lane >= d ? s : a;
    }
    return a;
}

// A running sum of weights (each at most 1): it starts at 4, so that every sum
// is larger than what is added and its rounding error is a two-term difference.
struct Mass {
    float h = 4.f, l = 0.f;
    __device__ __forceinline__ void add(float2 w) {
        const float s = h + w.x;
        l += (w.x - (s - h)) + w.y;
        h = s;
    }
    __device__ __forceinline__ dd2 value() const { return norm2(h - 4.f, l); }
};

// ---- exact weights two at a time, for maxima not far from zero -----------------
//
// Where no |z| is above some 64 T, exp(z / T) itself fits fp32's range: the
// difference from the maximum, and its rounding error, need not be formed, and
// a power of two 2^E takes the maximum's place.  Packed fp32 pairs halve the
// instructions.  768 rows of 128256 bf16 with top-p: 368 us, against 417 with
// weight() throughout; rows without filters 40 against 49 us.

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pair(float a, float b) {
    f32x2 y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ f32x2 pair(float a) { return pair(a, a); }
__device__ __forceinline__ float2 halves(f32x2 x) {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(x));
    return y;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return fma2(b, pair(-1.f), a); }

constexpr float kLn2 = 0.693147182f;
constexpr float kNear = 64.f;      // |max| / T up to here
constexpr int kNearDepth = 120;    // octaves below 2^E that are held

struct NearScale {
    float ih, il;   // 1 / temperature
    float lo;       // the smallest z
    uint32_t bias;  // of the exponent: one's less E
};

__device__ __forceinline__ NearScale near_scale(const RowScale &S, float temp, int E) {
    return {S.ih, S.il, (float)(E - kNearDepth) * (kLn2 * temp), 0x3f800000u - ((uint32_t)E << 23)};
}
// The octave above a maximum: exp(max / T) <= 2^E.
__device__ __forceinline__ int near_octave(float m, const RowScale &S) { return (int)ceilf(m * S.ch) + 1; }

struct Pair2 {
    f32x2 h, l;
};

// exp(z / T) / 2^E of two elements, each as hi + lo; steps as in weight().
__device__ __forceinline__ Pair2 near_weights(float z0, float z1, const NearScale &N, const ExpTable &tab) {
    const f32x2 z = pair(z0, z1);
    const f32x2 nx = mul2(z, pair(-N.ih));                                       // -xh
    const f32x2 xl = fma2(z, pair(N.il), fma2(z, pair(N.ih), nx));
    const f32x2 km = fma2(nx, pair(-46.1662413f), pair(12582912.f + 16.f));      // the low bits hold k + 16
    const f32x2 k = add2(km, pair(-12582912.f - 16.f));
    const f32x2 nr = fma2(k, pair(0.0216608495f), nx);                           // -r
    const f32x2 rl = fma2(k, pair(5.95204441e-11f), xl);
    const f32x2 r = mul2(nr, pair(-1.f)), q = add2(r, rl);
    const f32x2 t = fma2(mul2(q, q), fma2(q, fma2(q, pair(4.16666667e-2f), pair(0.166666667f)), pair(0.5f)), rl);
    const float2 ks = halves(km);
    const uint32_t k0 = __float_as_uint(ks.x), k1 = __float_as_uint(ks.y);
    const f32x2 Tx = pair(tab.x[k0 & 31], tab.x[k1 & 31]), Ty = pair(tab.y[k0 & 31], tab.y[k1 & 31]);
    const f32x2 scale = pair(__uint_as_float(((k0 & ~31u) << 18) + N.bias), __uint_as_float(((k1 & ~31u) << 18) + N.bias));
    const f32x2 v = mul2(Tx, r), nvl = fma2(Tx, nr, v);
    const f32x2 u = fma2(Tx, t, fma2(Ty, r, Ty));
    const f32x2 h = add2(Tx, v);
    const f32x2 l = add2(sub2(v, sub2(h, Tx)), sub2(u, nvl));
    return {mul2(h, scale), mul2(l, scale)};
}

// Two running sums, as Mass.
struct Mass2 {
    f32x2 h = pair(4.f), l = pair(0.f);
    __device__ __forceinline__ void add(Pair2 w) {
        const f32x2 s = add2(h, w.h);
        l = add2(l, add2(sub2(w.h, sub2(s, h)), w.l));
        h = s;
    }
    __device__ __forceinline__ dd2 value() const {
        const float2 a = halves(h), b = halves(l);
        return add_dd(norm2(a.x - 4.f, b.x), norm2(a.y - 4.f, b.y));
    }
    __device__ __forceinline__ void scale(float by) {
        const float2 a = halves(h), b = halves(l);
        const dd2 x = add_dd({4.f, 0.f}, {(a.x - 4.f) * by, b.x * by});
        const dd2 y = add_dd({4.f, 0.f}, {(a.y - 4.f) * by, b.y * by});
        h = pair(x.h, y.h);
        l = pair(x.l, y.l);
    }
};

// The mass itself, or the whole number that it misses by less than such a mass's
// error.  Where only the maxima of a row count, masses relative to the maximum are
// whole, and goals may fall exactly on a border; their factor 2^E exp(-m / T) does
// not cancel exactly.  (2^-34 of the mass: other masses lose nothing that counts.)
__device__ __forceinline__ dd2 whole_mass(dd2 a) {
    const float n = rintf(a.h), rest = (a.h - n) + a.l, k = rintf(rest);
    return fabsf(rest - k) <= 5.8207661e-11f * a.h ? norm2(n, k) : a;
}

// What turns such a mass into one relative to the maximum m: 2^E exp(-m / T).
__device__ __forceinline__ dd2 near_to_max(const RowScale &S, const ExpTable *tab, int E) {
    const float2 y = weight_of(0.f, S, tab);
    const float by = __uint_as_float((uint32_t)(127 + E) << 23);
    return {y.x * by, y.y * by};
}

namespace cg = cooperative_groups;

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp((z - max) / T) in fp32, good to about 2^-22: the exponent with its low
// part, its fraction through ex2.approx.
__device__ __forceinline__ float fast_weight(float z, const RowScale &S) {
    const float d = z - S.m;
    const float e = d * S.ch;
    if (!(e >= -125.f)) return 0.f;
    const float bb = d - z;
    const float dl = (z - (d - bb)) - (S.m + bb);
    float el = fmaf(d, S.ch, -e);
    el = fmaf(d, S.cl, el);
    el = fmaf(dl, S.ch, el);
    const float n = rintf(e);
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((e - n) + el));
    return __int_as_float(__float_as_int(y) + ((int)n << 23));
}

// A CTA's slice of the row, for the slow paths.
struct RowSlice {
    const void *z;
    const uint4 *words;
    int64_t base;
    int32_t n, shift, held;
    RowScale S;
};

// What the CTAs of a cluster read of one another.
struct alignas(16) WarpShared {
    unsigned long long bar;
    ExpTable tab;
    float top, low;                 // slice maximum and smallest finite logit
    int32_t bad;
    float ih, il, ch, cl;           // 1 / temperature, log2(e) / temperature
    dd2 min_off;                    // temperature * ln(min_p)
    uint32_t count, gathered;       // border elements
    int32_t list_end[kWarpMaxCluster], full, pick;
    float total;
    uint32_t coarse_count[32];      // of 32 groups of bins
    float coarse_mass[32];
    int32_t k_bin, lo_bin, hi_bin, k_before;
    uint64_t threshold;
    RowSlice slice;
    dd2 slice_mass[3];              // kept, above, all below t_goal
    dd2 rank_mass[kWarpMaxCluster]; // what stays of every rank's slice
    dd2 run_mass[kMaxWarps];       // kept mass of each warp's run
    dd2 part_mass[kMaxWarps];
    union {
        dd2 in_mass[kMaxWarps];
        uint64_t warp_key[kMaxWarps];
        float warp_f[2][kMaxWarps];
    };
    uint64_t list[kLocalList];
    union {
        alignas(16) uint32_t hist[2 * kBins];  // counts or masses; or counts, then masses
        uint64_t all[kList];        // the row's border elements, ranked
        struct {
            uint64_t raw[kShared], ranked[kShared];
        } share;
    };
};

static_assert(sizeof(WarpShared) <= 11264, "three CTAs of 64 KB slices to an SM");
static_assert(sizeof(WarpShared) % 16 == 0 && offsetof(WarpShared, hist) % 16 == 0,
              "16-byte accesses to the histogram and to the words behind this");

// A value that all lanes hold, marked as such: in branches that the compiler
// takes for divergent, every shuffle costs hundreds of cycles.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ float uniform(float x) { return __shfl_sync(0xffffffffu, x, 0); }

// The cluster's barrier in two parts, for a CTA's end.  The arrival releases: what
// the CTA has read of another's shared memory has been read by then.
__device__ __forceinline__ void cluster_arrive_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_all() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <class T>
struct WordOf {
    static constexpr int kElems = 16 / (int)sizeof(T);
};

template <class T>
__device__ __forceinline__ void unpack(uint4 w, float (&x)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 4) {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    } else {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            T a, b;
            *reinterpret_cast<uint16_t *>(&a) = (uint16_t)(u[i] & 0xffffu);
            *reinterpret_cast<uint16_t *>(&b) = (uint16_t)(u[i] >> 16);
            x[2 * i] = to_f32<T>(a);
            x[2 * i + 1] = to_f32<T>(b);
        }
    }
}

template <class T>
__device__ __forceinline__ T minus_inf();
template <>
__device__ __forceinline__ float minus_inf() {
    return -INFINITY;
}
template <>
__device__ __forceinline__ __nv_bfloat16 minus_inf() {
    return __ushort_as_bfloat16(0xff80u);
}
template <>
__device__ __forceinline__ __half minus_inf() {
    return __ushort_as_half(0xfc00u);
}

// A histogram's increment, left out for -inf (padding among it), without a branch.
__device__ __forceinline__ void add_if_finite(uint32_t *bin, uint32_t by, float x) {
    asm volatile("{ .reg .pred p; setp.gt.f32 p, %2, 0fFF800000; @p red.shared.add.u32 [%0], %1; }" ::"r"(
                     smem_u32(bin)),
                 "r"(by), "f"(x)
                 : "memory");
}

__device__ __forceinline__ float scan_f32(float x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const float o = __shfl_up_sync(0xffffffffu, x, d);
        x += lane >= d ? o : 0.f;
    }
    return x;
}
__device__ __forceinline__ uint32_t scan_u32(uint32_t x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, x, d);
        x += lane >= d ? o : 0u;
    }
    return x;
}

// One or two neighbouring bins of the row, added over the ranks.  (A few words
// of each CTA: reading whole histograms took most of a row's time.)
__device__ __forceinline__ uint2 row_bins(WarpShared &sh, int C, int slot, int per_lane) {
    cg::cluster_group cluster = cg::this_cluster();
    uint2 s = make_uint2(0, 0);
    uint32_t x[kWarpMaxCluster], y[kWarpMaxCluster];
#pragma unroll
    for (int c = 0; c < kWarpMaxCluster; ++c) {
        x[c] = y[c] = 0;
        if (c < C) {
            const uint32_t *h = cluster.map_shared_rank(sh.hist, c) + slot;
            x[c] = h[0];
            if (per_lane == 2) y[c] = h[1];
        }
    }
#pragma unroll
    for (int c = 0; c < kWarpMaxCluster; ++c) {
        s.x += x[c];
        s.y += y[c];
    }
    return s;
}

// ---- slow paths, rarely taken: out of line, an element at a time --------------

template <class T>
__device__ __forceinline__ float slice_elem(const RowSlice &c, int e) {
    const int at = e + c.shift;
    const T *src = at / (16 / (int)sizeof(T)) < c.held ? reinterpret_cast<const T *>(c.words) + at
                                                       : static_cast<const T *>(c.z) + e;
    return to_f32<T>(*src);
}

// The row's first element (largest logit, lowest index); by the whole cluster.
template <class T>
__device__ __noinline__ uint64_t first_of_row(WarpShared &sh) {
    cg::cluster_group cluster = cg::this_cluster();
    const RowSlice &c = sh.slice;
    uint64_t first = 0;
#pragma unroll 1
    for (int e = threadIdx.x; e < c.n; e += blockDim.x) {
        const float x = slice_elem<T>(c, e);
        if (x == c.S.m) {
            const uint64_t key = composite(x, c.base + e);
            first = key > first ? key : first;
        }
    }
#pragma unroll 1
    for (int d = 16; d > 0; d >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, first, d);
        first = o > first ? o : first;
    }
    cluster.sync();
    if (threadIdx.x % 32 == 0) sh.warp_key[threadIdx.x / 32] = first;
    cluster.sync();
#pragma unroll 1
    for (int r = 0; r < (int)cluster.num_blocks(); ++r)
#pragma unroll 1
        for (int w = 0; w < (int)blockDim.x / 32; ++w) {
            const uint64_t o = cluster.map_shared_rank(&sh, r)->warp_key[w];
            first = o > first ? o : first;
        }
    return first;
}

// Mass (or number) of the row's elements at or above a composite; by the whole
// cluster.  run_mass keeps the parts of this CTA's warps (masses, by runs).
template <class T>
__device__ __noinline__ dd2 sum_from(WarpShared &sh, uint64_t from, bool masses) {
    cg::cluster_group cluster = cg::this_cluster();
    const RowSlice &c = sh.slice;
    Mass a;
#pragma unroll 1
    for (int e = threadIdx.x; e < c.n; e += blockDim.x) {
        const float x = slice_elem<T>(c, e);
        if (x > -INFINITY && composite(x, c.base + e) >= from)
            a.add(masses ? weight_of(x, c.S, &sh.tab) : make_float2(1.f, 0.f));
    }
    __syncwarp();
    const dd2 own = warp_sum_dd(a.value());
    cluster.sync();  // the last sum has been read everywhere
    if (threadIdx.x % 32 == 0) sh.part_mass[threadIdx.x / 32] = own;
    cluster.sync();
    dd2 s = {0.f, 0.f};
#pragma unroll 1
    for (int r = 0; r < (int)cluster.num_blocks(); ++r)
#pragma unroll 1
        for (int w = 0; w < (int)blockDim.x / 32; ++w)
            s = add_dd(s, cluster.map_shared_rank(&sh, r)->part_mass[w]);
    return s;
}

// The threshold that top-k (k > 0) and then top-p (p < 1) leave, by bisection of
// the composite over the whole row: for borders with too many elements to
// gather.
template <class T>
__device__ __noinline__ uint64_t bisect_row(WarpShared &sh, int64_t k, float p) {
    uint64_t thr = 0;
    const uint64_t top = first_of_row<T>(sh);
#pragma unroll 1
    for (int by = 0; by < 2; ++by) {   // top-k, top-p
        if (by == 0 ? k <= 0 : !(p < 1.f)) continue;
        dd2 goal = {0.f, 0.f};
        if (by == 1) goal = mul_dd(sum_from<T>(sh, thr, true), {p > 0.f ? p : 0.f, 0.f});
        uint64_t l = thr, h = top;
#pragma unroll 1
        while (l < h) {
            const uint64_t mid = l + (h - l) / 2;
            // (counts as pairs of floats are whole up to 2^47)
            const dd2 s = sum_from<T>(sh, mid + 1, by == 1);
            if (by == 0 ? (double)s.h + (double)s.l >= (double)k : !less_dd(s, goal)) l = mid + 1;
            else h = mid;
        }
        thr = l;
    }
    return thr;
}

// Ranks the row's border in place, every CTA for itself: for lists too long for
// the shared ranking.
__device__ __noinline__ void rank_alone(WarpShared &sh, int got) {
    constexpr int kMost = 4;   // elements per thread
    const int n = (int)blockDim.x;
    uint64_t key[kMost];
    int at_of[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        const int i = (int)threadIdx.x + j * n;
        key[j] = i < got ? sh.all[i] : 0;
        at_of[j] = 0;
    }
    if (got <= n) {
        if ((int)threadIdx.x / 32 * 32 < got)
#pragma unroll 8
            for (int x = 0; x < got; ++x) at_of[0] += sh.all[x] > key[0];
    } else {
#pragma unroll 1
        for (int x = 0; x < got; ++x) {
            const uint64_t o = sh.all[x];
#pragma unroll
            for (int j = 0; j < kMost; ++j) at_of[j] += o > key[j];
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMost; ++j)
        if ((int)threadIdx.x + j * n < got) sh.all[at_of[j]] = key[j];
    __syncthreads();
}

// The element of r0 .. r1 - 1 whose running mass, from `at` on, passes the goal;
// or, where rounding lets none, the last with mass.  By the whole CTA; goal and
// at are warp 0's.  U loads at a time: one from shared memory, where short code
// counts (a single row's time is mostly its first passes through the code).
template <class T, int kThreads, int U>
__device__ __forceinline__ void draw_element(const RowSlice &c, const ExpTable &tab, dd2 *part_mass, uint64_t thr,
                                             int r0, int r1, dd2 goal, dd2 at, int32_t *token) {
    constexpr int kWarps = kThreads / 32;
    const int warp = uniform((int)threadIdx.x / 32), lane = threadIdx.x % 32;
    // every warp a part, its lanes in turn
    const int part = (r1 - r0 + kThreads - 1) / kThreads * 32;
    auto mass_of = [&](float x, int e) -> float2 {   // of element e, if it stays
        return x > -INFINITY && composite(x, c.base + e) >= thr ? weight_of(x, c.S, &tab) : make_float2(0.f, 0.f);
    };
    {
        const int p0 = min(r1, r0 + part * warp), p1 = min(r1, p0 + part);
        Mass a;
#pragma unroll 1
        for (int e = p0 + lane; e - lane < p1; e += 32 * U) {
            float x[U];
#pragma unroll
            for (int i = 0; i < U; ++i) x[i] = e + 32 * i < p1 ? slice_elem<T>(c, e + 32 * i) : -INFINITY;
#pragma unroll
            for (int i = 0; i < U; ++i) a.add(mass_of(x[i], e + 32 * i));
        }
        __syncwarp();
        const dd2 own = warp_sum_dd(a.value());
        if (lane == 0) part_mass[warp] = own;
    }
    __syncthreads();
    if (warp != 0) return;
    // the first of 32 masses that passes the goal, and the mass before it
    auto choose = [&](dd2 mass) -> int {
        const dd2 reach = add_dd(at, warp_scan_dd(mass, lane));
        const unsigned some = __ballot_sync(0xffffffffu, mass.h > 0.f);
        const unsigned over = __ballot_sync(0xffffffffu, mass.h > 0.f && less_dd(goal, reach));
        const int q = over ? __ffs(over) - 1 : 31 - __clz(some);
        if (q > 0) at = shfl_dd(reach, q - 1);
        return q;
    };
    const int q = choose(lane < kWarps ? part_mass[lane] : dd2{0.f, 0.f});
    const int q0 = min(r1, r0 + part * q), q1 = min(r1, q0 + part), per = part / 32;
    int l0 = q0, l1 = q1;
    if (per > 2) {
        // of a long part first the lane's stretch
        l0 = min(q1, q0 + per * lane);
        l1 = min(q1, l0 + per);
        Mass a;
#pragma unroll 1
        for (int i = 0; i < per; i += (U + 1) / 2) {
            float x[(U + 1) / 2];
#pragma unroll
            for (int j = 0; j < (U + 1) / 2; ++j) x[j] = l0 + i + j < l1 ? slice_elem<T>(c, l0 + i + j) : -INFINITY;
#pragma unroll
            for (int j = 0; j < (U + 1) / 2; ++j) a.add(mass_of(x[j], l0 + i + j));
        }
        __syncwarp();
        const int l = choose(a.value());
        l0 = __shfl_sync(0xffffffffu, l0, l);
        l1 = __shfl_sync(0xffffffffu, l1, l);
    }
    int hit = -1, end = -1;
#pragma unroll 1
    for (int e = l0; e < l1 && hit < 0; e += 32) {
        const float2 y = e + lane < l1 ? mass_of(slice_elem<T>(c, e + lane), e + lane) : make_float2(0.f, 0.f);
        __syncwarp();
        const dd2 upto = add_dd(at, warp_scan_dd({y.x, y.y}, lane));
        const unsigned has = __ballot_sync(0xffffffffu, y.x > 0.f);
        const unsigned past = __ballot_sync(0xffffffffu, y.x > 0.f && less_dd(goal, upto));
        if (has) end = e + 31 - __clz(has);
        if (past) hit = e + __ffs(past) - 1;
        at = shfl_dd(upto, 31);
    }
    if (lane == 0) *token = (int32_t)(c.base + (hit >= 0 ? hit : end));
}

// Elements e0 .. of a row of probabilities, E of them, 16 bytes at a time where
// that is aligned.
template <int E>
__device__ __forceinline__ void store_probs(float *out, int e0, int n, bool vec, const float (&y)[E]) {
    if (vec && e0 >= 0 && e0 + E <= n) {
#pragma unroll
        for (int i = 0; i < E; i += 4)
            *reinterpret_cast<float4 *>(out + e0 + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (e0 + i >= 0 && e0 + i < n) out[e0 + i] = y[i];
    }
}

// kHeld: every slice fits in shared memory, in words padded with -inf to whole
// rounds of the block, so that the sweeps need no bounds.
// kThreads: 256, three CTAs to an SM, or 1024 for slices that fill one.
template <class T, bool kHeld, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 1024 ? 1 : 3) warp_kernel(const __grid_constant__ WarpParams A) {
    constexpr int E = WordOf<T>::kElems, kWarps = kThreads / 32;
    extern __shared__ __align__(16) char raw[];
    WarpShared &sh = *reinterpret_cast<WarpShared *>(raw);
    uint4 *words = reinterpret_cast<uint4 *>(raw + sizeof(WarpShared));
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = uniform(tid / 32), lane = tid % 32;
    const int64_t r = blockIdx.x / C;
    const int64_t base = min(A.V, (int64_t)rank * A.slice);  // this CTA's elements
    const int n = (int)(min(A.V, base + A.slice) - base);
    const T *z = static_cast<const T *>(A.z) + r * A.zs + base;
    // word w holds elements w * E - shift ..; what lies outside is -inf
    const int shift = (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
    const int W = n > 0 ? (n + shift + E - 1) / E : 0;
    const int held = kHeld ? W : min(W, A.cached);

    // ---- the slice into shared memory ------------------------------------
    if (tid == 0) {
        mbar_init(&sh.bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.bad = 0;
        sh.count = 0;
    }
    if (tid >= 32 && tid < 64) {
        sh.tab.x[lane] = kPow2[lane].x;
        sh.tab.y[lane] = kPow2[lane].y;
    }
    __syncthreads();
    wait_for_primary_grid();
    const int w0 = shift ? 1 : 0;                          // first whole word
    const int w1 = min(held, (n + shift) / E);             // one past the last
    const int whole = max(0, w1 - w0);
    if (tid == 0) {
        mbar_arrive_expect_tx(&sh.bar, (uint32_t)whole * 16u);
        const char *src = reinterpret_cast<const char *>(z - shift) + w0 * 16;
#pragma unroll 1
        for (int at = 0; at < whole; at += 1024) {
            const int part = min(1024, whole - at);
            bulk_copy_g2s(words + w0 + at, src + (int64_t)at * 16, (uint32_t)part * 16u, &sh.bar);
        }
    }
    if (tid < 2 * E) {  // the ragged words at both ends
        const int w = tid < E ? 0 : W - 1;
        if (w >= 0 && w < held && (w < w0 || w >= w1)) {
            const int e = w * E - shift + tid % E;
            reinterpret_cast<T *>(words)[w * E + tid % E] = e >= 0 && e < n ? z[e] : minus_inf<T>();
        }
    }
    // every warp takes a run of words, its lanes in turn
    const int run = (W + kThreads - 1) / kThreads * 32;
    if (kHeld)
#pragma unroll 1
        for (int w = W + tid; w < run * kWarps; w += kThreads)
#pragma unroll
            for (int i = 0; i < E; ++i) reinterpret_cast<T *>(words)[w * E + i] = minus_inf<T>();
    // the row's settings; what of them needs fp64 is one thread's work while
    // the copy runs
    const float temp = uniform(A.temperature ? A.temperature[r] : 1.f);
    const int64_t k = uniform(A.top_k ? A.top_k[r] : 0);
    const float p = uniform(A.top_p ? A.top_p[r] : 1.f);
    const float mp = uniform(A.min_p ? A.min_p[r] : 0.f);
    if (tid == 64) {
        const double i = 1.0 / (double)temp, c = i * 1.4426950408889634;
        sh.ih = (float)i;
        sh.il = (float)(i - (double)sh.ih);
        sh.ch = (float)c;
        sh.cl = (float)(c - (double)sh.ch);
    }
    if (tid == 96 && mp > 0.f) {
        const double off = (double)temp * log((double)mp);
        sh.min_off = {(float)off, (float)(off - (double)(float)off)};
    }
    const bool came = mbar_wait(&sh.bar, 0);
    // (one that gave up waits once more: the copies should land before the CTA ends)
    if (!came) mbar_wait(&sh.bar, 0);
    if (!__syncthreads_and(came) && tid == 0) {
        atomicOr(A.status, SV_STATUS_TIMEOUT);
        sh.bad = 1;
    }

    const int s0 = kHeld ? run * warp : min(W, run * warp), s1 = kHeld ? s0 + run : min(W, s0 + run);
    auto load = [&](int w, float (&x)[E]) {
        if (kHeld || w < held) {
            unpack<T>(words[w], x);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int e = w * E - shift + i;
                x[i] = e >= 0 && e < n ? to_f32<T>(z[e]) : -INFINITY;
            }
        }
    };
    auto index_of = [&](int w, int i) -> int64_t { return base + w * E - shift + i; };
    auto largest = [&](const float (&x)[E]) -> float {
        float y = x[0];
#pragma unroll
        for (int i = 1; i < E; ++i) y = fmaxf(y, x[i]);
        return y;
    };

    // ---- the maximum (NaN where there is one) ------------------------------
    {
        float top = -INFINITY, low = INFINITY;
        // (the smallest of a sample: it only sets the histogram's scale)
#pragma unroll 4
        for (int w = s0 + lane; w < s1; w += 32) {
            float x[E];
            load(w, x);
#pragma unroll
            for (int i = 0; i < E; ++i) top = max_nan(top, x[i]);
            low = fminf(low, x[0] == -INFINITY ? INFINITY : x[0]);
        }
#pragma unroll 1
        for (int d = 16; d > 0; d >>= 1) {
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, d));
        }
        if (lane == 0) {
            sh.warp_f[0][warp] = top;
            sh.warp_f[1][warp] = low;
        }
#pragma unroll 1
        for (int i = tid; i < 2 * kBins; i += kThreads) sh.hist[i] = 0;
        __syncthreads();
        if (warp == 0) {
            top = lane < kWarps ? sh.warp_f[0][lane] : -INFINITY;
            low = lane < kWarps ? sh.warp_f[1][lane] : INFINITY;
#pragma unroll 1
            for (int d = 16; d > 0; d >>= 1) {
                top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
                low = fminf(low, __shfl_xor_sync(0xffffffffu, low, d));
            }
            if (lane == 0) {
                sh.top = top;
                sh.low = low;
            }
        }
    }
    cluster.sync();
    float m = -INFINITY, low = INFINITY;
    int bad = 0;
    if (lane < C) {
        const WarpShared *o = cluster.map_shared_rank(&sh, lane);
        m = o->top;
        low = o->low;
        bad = o->bad;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, d));
    }
    m = uniform(m);
    low = uniform(low);
    bad = uniform(__any_sync(0xffffffffu, bad)) || !(m < INFINITY) || !(temp >= kColdest && temp <= kHottest);
    float *out = A.probs ? A.probs + r * A.ps + base : nullptr;
    if (bad || m == -INFINITY) {
        if (rank == 0 && tid == 0) {
            atomicOr(A.status, bad ? SV_STATUS_BAD_VALUE : SV_STATUS_ZERO_MASS);
            if (A.token) A.token[r] = -1;
        }
        if (out)
#pragma unroll 1
            for (int e = tid; e < n; e += kThreads) out[e] = 0.f;
        cluster.sync();
        return;
    }
    const RowScale S = {m, sh.ih, sh.il, sh.ch, sh.cl, -85.f * temp};
    const bool by_k = k > 0 && k < A.V, by_p = p < 1.f;
    float zmin = -INFINITY;  // min-p's lowest logit
    if (mp > 0.f) {
        zmin = m;
        if (mp <= 1.f) {
            // the smallest float at or above max + temperature * ln(min_p)
            const dd2 edge = add_dd({m, 0.f}, sh.min_off);
            zmin = fminf(edge.l > 0.f ? nextafterf(edge.h, INFINITY) : edge.h, m);
        }
    }

    if (tid == 0) sh.slice = {z, words, base, n, shift, held, S};
    // ---- top-k and top-p: the border bins -------------------------------------
    // Top-p after a small top-k: the list gathers all that top-k leaves, and the
    // histogram counts only.  (k below 200, top-p: 256 rows of 128256 bf16 97
    // against 105 us, 64 of 262144 fp32 with min-p too 107 against 120.)
    const bool few = by_k && by_p && k <= kFew, by_h = by_p && !few;
    // t(x) = 2^23 + the element's bin: a monotone function of x, so that bins
    // are runs of the row's order
    const bool both = by_k && by_h;
    const int bins = both ? kBins : 2 * kBins;
    // the last bin is for what lies further down
    // (kTiny: bins per unit stay finite; the coldest temperature's reach is above it,
    // so that a bin never spans more than kRangeOctaves / (bins - 2))
    const float reach = kRangeOctaves / S.ch, span = low < m ? fmaxf(fminf(m - low, reach), kTiny) : reach;
    const float per = (float)(bins - 2) / span;                          // bins per unit of z
    auto t_of = [&](float x) -> float {
        return fminf(fmaf(m - x, per, kMagic), kMagic + (float)(bins - 1));
    };
    const float never = kMagic + (float)bins;
    // kept by top-k and top-p for sure: t < t_keep; to be settled: t_keep <= t
    // <= t_last, and t == t_k, of which top-k keeps the k_left largest
    float t_keep = never, t_last = 0.f, t_k = never;
    int64_t k_left = 0;
    uint64_t thr = 0;       // kept: composite >= thr
    bool far = false;
    if (by_k || by_h) {
        // masses relative to the bin's middle, in fixed point: that short arc of
        // the exponential (at most +-0.02 octaves) to its square term; eight
        // ranks' elements in one bin stay below 2^32
        const float drop = S.ch / per;                                   // octaves per bin
        const float unit = exp2f((float)min(22, 27 - (31 - __clz(A.slice + 16))));
        const float c1 = -unit * 0.693147182f * drop, c2 = unit * 0.240226507f * drop * drop;
        uint32_t *masses = sh.hist + (both ? kBins : 0);
        auto count_up = [&](auto want_k, auto want_p) {
#pragma unroll 1
            for (int w = s0 + lane; w < s1; w += 32) {
                float x[E];
                load(w, x);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float d = m - x[i], t = fminf(fmaf(d, per, kMagic), never - 1.f);
                    const int b = __float_as_int(t) & (2 * kBins - 1);
                    if (decltype(want_k)::value) add_if_finite(&sh.hist[b], 1u, x[i]);
                    if (decltype(want_p)::value) {
                        const float f = fminf(fmaf(d, per, kMagic - t), 0.5f);
                        const float y = fmaf(f, fmaf(f, c2, c1), unit + kMagic);
                        add_if_finite(&masses[b], __float_as_uint(y) & 0x7fffffu, x[i]);
                    }
                }
            }
        };
        const std::true_type yes{};
        const std::false_type no{};
        if (both) count_up(yes, yes);
        else if (by_k) count_up(yes, no);
        else count_up(no, yes);
        __syncthreads();
        // sums of 32 groups of bins, a warp to a group
        const int group = bins / 32, per_lane = group / 32;
        const float inv_unit = 1.f / unit;
        for (int g = warp; g < 32; g += kWarps) {
            uint32_t c = 0;
            float y = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (h < per_lane) {
                    const int b = g * group + h * 32 + lane;
                    if (by_k) c += sh.hist[b];
                    if (by_h) y += (float)masses[b] * (pow2(-drop * (float)b) * inv_unit);
                }
            if (by_k) c = __reduce_add_sync(0xffffffffu, c);
            if (by_h)
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
            if (lane == 0) {
                sh.coarse_count[g] = c;
                sh.coarse_mass[g] = y;
            }
        }
        cluster.sync();
        // every rank's first warp: the row's groups, then the bins of the ones
        // that hold the borders
        if (warp == 0) {
            uint32_t count = 0;
            float mass = 0.f;
            {
                uint32_t x[kWarpMaxCluster];
                float y[kWarpMaxCluster];
#pragma unroll
                for (int c = 0; c < kWarpMaxCluster; ++c) {
                    x[c] = 0;
                    y[c] = 0.f;
                    if (c < C) {
                        const WarpShared *o = cluster.map_shared_rank(&sh, c);
                        x[c] = o->coarse_count[lane];
                        y[c] = o->coarse_mass[lane];
                    }
                }
#pragma unroll
                for (int c = 0; c < kWarpMaxCluster; ++c) {
                    count += x[c];
                    mass += y[c];
                }
            }
            int k_bin = bins, k_before = 0, lo = bins, hi = bins;
            const float m_upto = scan_f32(mass, lane);
            const uint32_t c_upto = scan_u32(count, lane);
            float m_all = __shfl_sync(0xffffffffu, m_upto, 31), slack = 0.f;
            // (a row with no more than k logits has no border of top-k)
            if (by_k && (int64_t)__shfl_sync(0xffffffffu, c_upto, 31) > k) {
                const int g = __ffs(__ballot_sync(0xffffffffu, (int64_t)c_upto >= k)) - 1;
                const uint32_t before = __shfl_sync(0xffffffffu, c_upto - count, g);
                const uint2 own = row_bins(sh, C, g * group + lane * per_lane, per_lane);
                const uint32_t upto = before + scan_u32(own.x + own.y, lane);
                const int l = __ffs(__ballot_sync(0xffffffffu, (int64_t)upto >= k)) - 1;
                const bool first = per_lane == 1 || (int64_t)(upto - own.y) >= k;
                const int second = __shfl_sync(0xffffffffu, (int)!first, l);
                k_bin = g * group + l * per_lane + second;
                k_before = (int)__shfl_sync(0xffffffffu, upto - own.y - (first ? own.x : 0u), l);
                const uint32_t inside = __shfl_sync(0xffffffffu, first ? own.x : own.y, l);
                if (by_h) {   // (then a bin to a lane)
                    const uint2 w = row_bins(sh, C, kBins + g * group + lane, 1);
                    const float y = (float)w.x * (pow2(-drop * (float)(g * group + lane)) * inv_unit);
                    const float start = __shfl_sync(0xffffffffu, m_upto - mass, g) +
                                        __shfl_sync(0xffffffffu, scan_f32(y, lane) - y, l);
                    const float part = __shfl_sync(0xffffffffu, y, l) * ((float)(k - k_before) / (float)inside);
                    m_all = start + part;
                    slack = 0.03f * part;   // the bin's elements differ by less
                }
            }
            if (by_h) {
                // bins lo..hi hold the first element before which at least the goal
                // lies, whatever the approximate masses are off by
                // (the last bin's mass is too large, by less than what it is)
                const float last = (float)row_bins(sh, C, (both ? kBins : 0) + bins - 1, 1).x *
                                   (pow2(-drop * (float)(bins - 1)) * inv_unit);
                const float err = 2e-5f + 0.5f * inv_unit, goal = p * m_all, rest = m_all - goal,
                            loose = slack + 4e-6f * m_all + last;
                auto low_ok = [&](float through) -> bool {
                    return through * (1.f + err) >= goal * (1.f - err) - loose &&
                           (m_all - through) * (1.f - err) <= rest * (1.f + err) + loose;
                };
                auto high_ok = [&](float through) -> bool {
                    return through * (1.f - err) >= goal * (1.f + err) + loose ||
                           (m_all - through) * (1.f + err) <= rest * (1.f - err) - loose;
                };
                const unsigned gl = __ballot_sync(0xffffffffu, low_ok(m_upto));
                const unsigned gh = __ballot_sync(0xffffffffu, high_ok(m_upto));
#pragma unroll 1
                for (int side = 0; side < 2; ++side) {
                    const unsigned at = side == 0 ? gl : gh;
                    if (at == 0) continue;
                    const int g = __ffs(at) - 1;
                    const uint2 w = row_bins(sh, C, (both ? kBins : 0) + g * group + lane * per_lane, per_lane);
                    const float b0 = (float)(g * group + lane * per_lane);
                    const float y0 = (float)w.x * (pow2(-drop * b0) * inv_unit);
                    const float y1 = (float)w.y * (pow2(-drop * (b0 + 1.f)) * inv_unit);
                    const float upto = __shfl_sync(0xffffffffu, m_upto - mass, g) + scan_f32(y0 + y1, lane);
                    const bool in1 = side == 0 ? low_ok(upto) : high_ok(upto);
                    const bool in0 = side == 0 ? low_ok(upto - y1) : high_ok(upto - y1);
                    // (where rounding lets none pass: the group's last bin)
                    const unsigned bin = __ballot_sync(0xffffffffu, in1);
                    const int l = bin ? __ffs(bin) - 1 : 31;
                    const int second = __shfl_sync(0xffffffffu, (int)(per_lane == 2 && !in0), l);
                    (side == 0 ? lo : hi) = g * group + l * per_lane + second;
                }
            }
            if (lane == 0) {
                sh.k_bin = k_bin;
                sh.k_before = k_before;
                sh.lo_bin = lo;
                sh.hi_bin = hi;
            }
        }
        __syncthreads();
        const int k_bin = uniform(sh.k_bin);
        far = k_bin == bins - 1;    // what lies there is in no order: by bisection
        if (k_bin < bins) {
            t_k = kMagic + (float)k_bin;
            k_left = k - sh.k_before;
            t_keep = t_k;
        }
        if (few) {
            t_keep = kMagic;
            t_last = kMagic + (float)min(k_bin, bins - 1);
        }
        if (by_h) {
            const int edge = min(k_bin, bins - 1);    // nothing below it is left
            t_keep = kMagic + (float)min(uniform(sh.lo_bin), edge);
            t_last = kMagic + (float)min(uniform(sh.hi_bin), edge);
        }
    }

    // ---- masses of what stays, and the border's elements ----------------------
    // above: before the border (for top-p's goal); in: all that top-k leaves, its
    // own border bin aside; kept: what stays for sure
    Mass above, in, kept;
    const float t_goal = by_h ? t_k : 0.f;           // `in` wanted below it
    const bool dense = by_h ? t_k >= never : t_keep >= never && zmin == -INFINITY;
    const float t_far = fmaxf(fmaxf(t_goal, t_last), t_k < never ? t_k : 0.f);
    // (all but the first of a dense row in pairs, where its maximum allows that)
    const bool near = kHeld && dense && fabsf(m) <= kNear * temp;
    const int octave = near ? near_octave(m, S) : 0;
    const NearScale N = near_scale(S, temp, octave);
    // (below this no element can have t <= t_last: t_of's rounding is half a bin,
    // and only the last bin has no lower end)
    const float z_last = t_last >= never - 1.f ? -INFINITY : m - (t_last - kMagic + 1.f) / per;
    Mass2 near_all;
    Mass near_above, near_kept;
#pragma unroll 1
    for (int w = s0 + lane; w < s1; w += 32) {
        float x[E];
        load(w, x);
        if (kHeld && near) {
            float least = x[0];
#pragma unroll
            for (int i = 1; i < E; ++i) least = fminf(least, x[i]);
            if (__all_sync(0xffffffffu, least >= N.lo)) {
#pragma unroll
                for (int i = 0; i < E; i += 2) {
                    const Pair2 y = near_weights(x[i], x[i + 1], N, sh.tab);
                    near_all.add(y);
                    if (!by_p) continue;
                    const float2 h = halves(y.h), l = halves(y.l);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (x[i + j] < z_last) continue;
                        const float t = t_of(x[i + j]);
                        if (t > t_last) continue;
                        const float2 one = j == 0 ? make_float2(h.x, l.x) : make_float2(h.y, l.y);
                        if (t < t_keep) {
                            near_above.add(one);
                            if (mp > 0.f && x[i + j] >= zmin) near_kept.add(one);
                        } else {
                            const uint32_t at = atomicAdd(&sh.count, 1u);
                            if (at < kLocalList) sh.list[at] = composite(x[i + j], index_of(w, i + j));
                        }
                    }
                }
                continue;
            }
        }
        if (dense) {
            // every element's weight, four chains at a time
#pragma unroll
            for (int h = 0; h < E; h += 4) {
                float2 y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = weight(x[h + i], S, sh.tab);
                if (by_p) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        in.add(y[i]);
                        const float t = t_of(x[h + i]);
                        if (t < t_keep) {
                            above.add(y[i]);
                            if (mp > 0.f && x[h + i] >= zmin) kept.add(y[i]);
                        } else if (t <= t_last && x[h + i] > -INFINITY) {
                            const uint32_t at = atomicAdd(&sh.count, 1u);
                            if (at < kLocalList) sh.list[at] = composite(x[h + i], index_of(w, h + i));
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) kept.add(y[i]);
                }
            }
            continue;
        }
        const float x_top = largest(x), t_top = t_of(x_top);
        if (x_top == -INFINITY || (t_top > t_far && (t_top >= t_keep || x_top < zmin))) continue;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float t = t_of(x[i]);
            if (!(x[i] > -INFINITY) || (t > t_far && (t >= t_keep || x[i] < zmin))) continue;
            const bool stays = t < t_keep;
            if ((stays && x[i] >= zmin) || t < t_goal) {
                const float2 y = weight_of(x[i], S, &sh.tab);
                if (t < t_goal) in.add(y);
                if (stays && by_p) above.add(y);
                if (stays && x[i] >= zmin) kept.add(y);
            }
            if ((t >= t_keep && t <= t_last) || t == t_k) {
                const uint32_t at = atomicAdd(&sh.count, 1u);
                if (at < kLocalList) sh.list[at] = composite(x[i], index_of(w, i));
            }
        }
    }
    __syncwarp();
    {
        dd2 own_kept = kept.value(), own_above = above.value(), own_in = in.value();
        if (near) {
            const dd2 by = near_to_max(S, &sh.tab, octave), all = whole_mass(mul_dd(near_all.value(), by));
            own_above = add_dd(own_above, whole_mass(mul_dd(near_above.value(), by)));
            own_kept = add_dd(own_kept, by_p ? whole_mass(mul_dd(near_kept.value(), by)) : all);
            own_in = add_dd(own_in, all);
        }
        if (dense && by_p && !(mp > 0.f)) own_kept = own_above;
        const dd2 a = warp_sum_dd(own_kept);
        if (lane == 0) sh.run_mass[warp] = a;
        if (by_h) {
            const dd2 b = warp_sum_dd(own_above), c = warp_sum_dd(own_in);
            if (lane == 0) {
                sh.part_mass[warp] = b;
                sh.in_mass[warp] = c;
            }
        }
    }
    __syncthreads();
    if (warp < (by_h ? 3 : 1)) {
        const dd2 *from = warp == 0 ? sh.run_mass : warp == 1 ? sh.part_mass : sh.in_mass;
        const dd2 s = warp_sum_dd(lane < kWarps ? from[lane] : dd2{0.f, 0.f});
        if (lane == 0) {
            sh.slice_mass[warp] = s;
            if (warp == 0) sh.gathered = sh.count;
        }
    }
    cluster.sync();
    // every rank: the row's masses (in rank order) and border
    dd2 row_above = {0.f, 0.f}, row_in = {0.f, 0.f};   // (warp 0)
    if (warp == 0) {
        dd2 a = {0.f, 0.f}, b = a, c = a;
        int have = 0;
        if (lane < C) {
            const WarpShared *o = cluster.map_shared_rank(&sh, lane);
            a = o->slice_mass[0];
            b = o->slice_mass[1];
            c = o->slice_mass[2];
            have = (int)o->gathered;
        }
        const bool over = __any_sync(0xffffffffu, have > kLocalList);
        int at = have;
#pragma unroll
        for (int d = 1; d < kWarpMaxCluster; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, at, d);
            if (lane >= d) at += o;
        }
        if (by_h) {
            row_above = warp_sum_dd(b);
            row_in = warp_sum_dd(c);
        }
        if (lane < kWarpMaxCluster) {
            sh.rank_mass[lane] = a;
            sh.list_end[lane] = at;
        }
        if (lane == C - 1) sh.full = over || at > kList;
    }
    __syncthreads();
    int got = uniform(sh.list_end[C - 1]);
    const bool full = uniform(sh.full) != 0 || far;
    // (the histogram that the lists lie over has been read everywhere)
    if (!full)
#pragma unroll 1
        for (int s = warp; s < C; s += kWarps) {
            const int to = s > 0 ? sh.list_end[s - 1] : 0, cnt = sh.list_end[s] - to;
            const uint64_t *from = cluster.map_shared_rank(sh.list, s);
#pragma unroll 1
            for (int i = lane; i < cnt; i += 32) sh.all[to + i] = from[i];
        }
    const uint64_t *border = sh.all;   // in the row's order
    if (got > 0 || full) {
        if (full) {
            thr = bisect_row<T>(sh, t_k < never ? k : 0, by_p ? p : 1.f);
        } else {
            __syncthreads();
            // rank them: an element goes to the number of larger ones.  By one
            // warp (against one CTA: 768 rows of 128256 bf16 with top-p take as
            // long, one row of 32000 15.4 instead of 15.6 us), by the cluster
            // (those rows 367 instead of 379 us, 256 rows of 128256 fp32 186
            // instead of 199), or by every CTA where the list leaves no room
            // for a second one.
            if (got <= 32) {
                if (warp == 0) {
                    const uint64_t key = lane < got ? sh.share.raw[lane] : 0;
                    int at = 0;
#pragma unroll 1
                    for (int x = 0; x < got; ++x) at += __shfl_sync(0xffffffffu, key, x) > key;
                    if (lane < got) sh.share.ranked[at] = key;
                }
                __syncthreads();
            } else if (got <= kShared) {
                // every rank places a share of them, eight threads to an element,
                // in every rank's list
                const int part = lane % 8, total_groups = kThreads / 8 * C;
#pragma unroll 1
                for (int i0 = 0; i0 < got; i0 += total_groups) {
                    const int i = i0 + (tid / 8) * C + rank;
                    const uint64_t key = i < got ? sh.share.raw[i] : 0;
                    int at = 0;
                    if (i < got)
#pragma unroll 1
                        for (int x = part; x < got; x += 8) at += sh.share.raw[x] > key;
                    at += __shfl_xor_sync(0xffffffffu, at, 1);
                    at += __shfl_xor_sync(0xffffffffu, at, 2);
                    at += __shfl_xor_sync(0xffffffffu, at, 4);
                    if (i < got && part < C)
                        cluster.map_shared_rank(&sh, part)->share.ranked[at] = key;
                }
                cluster.sync();
            } else {
                rank_alone(sh, got);
            }
            border = got <= kShared ? sh.share.ranked : sh.all;
            if (warp == 0) {
                // the elements that top-k leaves: those above its border bin
                // (first in the order) and k_left of it
                int stay = got, above_k = 0;
                if (t_k < never) {
#pragma unroll 1
                    for (int i = lane; i < got; i += 32)
                        above_k += t_of(unordered((uint32_t)(border[i] >> 32))) < t_k;
#pragma unroll 1
                    for (int d = 16; d > 0; d >>= 1) above_k += __shfl_xor_sync(0xffffffffu, above_k, d);
                    stay = above_k + (int)k_left;
                }
                if (few || (by_p && t_k < never)) {
                    // the mass that is not in row_in yet
                    Mass a;
#pragma unroll 1
                    for (int i = (few ? 0 : above_k) + lane; i < stay; i += 32)
                        a.add(weight_of(unordered((uint32_t)(border[i] >> 32)), S, &sh.tab));
                    __syncwarp();
                    row_in = add_dd(row_in, warp_sum_dd(a.value()));
                }
                if (t_k < never && t_last < t_k && by_p) stay = above_k;
                int last = stay - 1;
                if (by_p) {
                    // the last element before which less than the goal lies
                    const dd2 goal = mul_dd(row_in, {p > 0.f ? p : 0.f, 0.f});
                    dd2 at = row_above;
                    last = -1;
#pragma unroll 1
                    for (int i = 0; i < stay; i += 32) {
                        dd2 y = {0.f, 0.f};
                        if (i + lane < stay) {
                            const float2 q = weight_of(unordered((uint32_t)(border[i + lane] >> 32)), S, &sh.tab);
                            y = {q.x, q.y};
                        }
                        const dd2 inc = warp_scan_dd(y, lane);
                        dd2 ex = {__shfl_up_sync(0xffffffffu, inc.h, 1), __shfl_up_sync(0xffffffffu, inc.l, 1)};
                        if (lane == 0) ex = {0.f, 0.f};
                        const bool stays = i + lane < stay && less_dd(add_dd(at, ex), goal);
                        const unsigned any = __ballot_sync(0xffffffffu, stays);
                        if (any) last = i + 31 - __clz(any);
                        at = add_dd(at, shfl_dd(inc, 31));
                    }
                }
                if (lane == 0) {
                    // none of the border's: everything above it, at least the row's first
                    const bool first_too = last < 0 && t_keep <= kMagic;
                    sh.threshold = last >= 0 ? border[last] : first_too ? border[0] : border[0] + 1;
                }
            }
            __syncthreads();
            thr = sh.threshold;
        }
    }
    // min-p's threshold: whole values, or the row's first element alone
    if (mp > 0.f) {
        const uint64_t t = mp > 1.f ? first_of_row<T>(sh) : (uint64_t)ordered(zmin) << 32;
        thr = t > thr ? t : thr;
    }
    if (full || mp > 1.f) {
        // the sums above do not hold: once more, with the threshold at hand
        Mass a;
#pragma unroll 1
        for (int e = s0 * E - shift + lane; e < s1 * E - shift; e += 32) {
            if (e < 0 || e >= n) continue;
            const float x = slice_elem<T>(sh.slice, e);
            if (x > -INFINITY && composite(x, base + e) >= thr) a.add(weight_of(x, S, &sh.tab));
        }
        __syncwarp();
        const dd2 own = warp_sum_dd(a.value());
        cluster.sync();
        if (lane == 0) sh.run_mass[warp] = own;
        cluster.sync();
        if (warp == 0 && lane < C) {
            dd2 s = {0.f, 0.f};
#pragma unroll 1
            for (int w = 0; w < kWarps; ++w)
                s = add_dd(s, cluster.map_shared_rank(&sh, lane)->run_mass[w]);
            sh.rank_mass[lane] = s;
        }
        got = 0;
    }
    cluster_arrive_all();  // the last access to another CTA's shared memory is made
    // the border elements that stay, into the runs and ranks they belong to;
    // every rank adds them up alike, so that all agree on where the goal lies
    if (got > 0) {
        // their weights, in the half of the lists that is free
        const bool stored = got <= kShared;
        float2 *weights = reinterpret_cast<float2 *>(border == sh.all ? sh.share.ranked : sh.share.raw);
        if (stored) {
#pragma unroll 1
            for (int i = tid; i < got; i += kThreads)
                weights[i] = border[i] >= thr ? weight_of(unordered((uint32_t)(border[i] >> 32)), S, &sh.tab)
                                              : make_float2(0.f, 0.f);
            __syncthreads();
        }
        // warp w adds up rank w's, and those of its own run
        Mass mine, of_rank;
        const uint32_t rank_base = (uint32_t)warp * (uint32_t)A.slice;
#pragma unroll 1
        for (int i = lane; i < got; i += 32) {
            const uint64_t key = border[i];
            if (key < thr) break;       // (in the row's order)
            const float2 y = stored ? weights[i]
                                            : weight_of(unordered((uint32_t)(key >> 32)), S, &sh.tab);
            const uint32_t v = ~(uint32_t)key;
            if (warp < C && v - rank_base < (uint32_t)A.slice) of_rank.add(y);
            const uint32_t e = v - (uint32_t)base;
            const int w = (int)((e + (uint32_t)shift) / (uint32_t)E);
            if (e < (uint32_t)n && w >= s0 && w < s1) mine.add(y);
        }
        __syncwarp();
        const dd2 a = warp_sum_dd(mine.value()), b = warp_sum_dd(of_rank.value());
        if (lane == 0) {
            sh.run_mass[warp] = add_dd(sh.run_mass[warp], a);
            if (warp < C) sh.rank_mass[warp] = add_dd(sh.rank_mass[warp], b);
        }
    }
    __syncthreads();

    // ---- the total and the draw -------------------------------------------------
    // The first rank, run, part and element whose running mass passes the goal,
    // or, where rounding lets none, the last with mass.
    dd2 goal = {0.f, 0.f}, at = {0.f, 0.f};   // (warp 0)
    if (warp == 0) {
        const dd2 own = lane < C ? sh.rank_mass[lane] : dd2{0.f, 0.f};
        const dd2 upto = warp_scan_dd(own, lane);
        const dd2 total = shfl_dd(upto, 31);
        if (lane == 0) {
            sh.total = total.h;
            sh.pick = -1;
        }
        if (A.token) {
            // the goal rounded as in 64 bits
            const double g = A.u[r] * ((double)total.h + (double)total.l);
            const float gh = (float)g;
            goal = {gh, (float)(g - (double)gh)};
            const unsigned some = __ballot_sync(0xffffffffu, own.h > 0.f);
            const unsigned over = __ballot_sync(0xffffffffu, own.h > 0.f && less_dd(goal, upto));
            const int holder = over ? __ffs(over) - 1 : 31 - __clz(some);
            if (holder == rank) {
                if (rank > 0) at = shfl_dd(upto, rank - 1);
                const dd2 mass = lane < kWarps ? sh.run_mass[lane] : dd2{0.f, 0.f};
                const dd2 reach = add_dd(at, warp_scan_dd(mass, lane));
                const unsigned runs = __ballot_sync(0xffffffffu, mass.h > 0.f);
                const unsigned past = __ballot_sync(0xffffffffu, mass.h > 0.f && less_dd(goal, reach));
                const int pick = past ? __ffs(past) - 1 : 31 - __clz(runs);
                if (pick > 0) at = shfl_dd(reach, pick - 1);
                if (lane == 0) sh.pick = pick;
            }
        }
    }
    __syncthreads();
    // ---- the row ------------------------------------------------------------------
    if (out) {
        const float inv = 1.f / sh.total;
        const float kz = fmaxf(zmin, unordered((uint32_t)(thr >> 32)));
        const bool all_stay = thr == 0;
        const bool vec = ((reinterpret_cast<uintptr_t>(out) - (uintptr_t)shift * 4u) & 15u) == 0;
#pragma unroll 1
        for (int w = s0 + lane; w < s1; w += 32) {
            float x[E], y[E];
            load(w, x);
#pragma unroll
            for (int i = 0; i < E; ++i) y[i] = 0.f;
            if (all_stay || largest(x) >= kz) {
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (all_stay || (x[i] >= kz && composite(x[i], index_of(w, i)) >= thr))
                        y[i] = fast_weight(x[i], S) * inv;
            }
            const int e0 = w * E - shift;
            store_probs<E>(out, e0, n, vec, y);
        }
    }
    // ---- the drawn element, on the rank that holds it ---------------------------
    const int pick = uniform(sh.pick);
    if (pick >= 0) {
        const int r0 = max(0, run * pick * E - shift), r1 = min(n, run * (pick + 1) * E - shift);
        draw_element<T, kThreads, 1>(sh.slice, sh.tab, sh.part_mass, thr, r0, r1, goal, at, A.token + r);
    }

    cluster_wait_all();  // no CTA leaves while another may read its shared memory
}

// ---- no filter at all ---------------------------------------------------------

struct PlainShared {
    ExpTable tab;
    float ih, il, ch, cl;
    float run_top[kPlainThreads / 32];   // each warp's run: its maximum, and its mass relative to that
    dd2 run_mass[kPlainThreads / 32];
    float top;                           // and the slice's
    dd2 slice_mass;
    dd2 part_mass[kPlainThreads / 32];
    RowSlice slice;
    float total;
    int32_t pick;
};

// A row that no filter applies to needs its maximum and its mass only, and both
// come in one pass over memory: every warp's sum is relative to the maximum so
// far of its run, and is rescaled when that grows (a handful of times).  Nothing
// is kept in shared memory; what is read again, the drawn run and, for
// probabilities, the row, mostly comes from L2.
//
// 64 rows of 262144 fp32 logits take 40 us (1.7 TB/s; 84 through warp_kernel),
// 256 of 128256 with probabilities 96 (150), one of 32000 11 (12).  Bound by
// arithmetic: some 38 instructions an element, the fp32 pipe busy for half the
// time, the rest going to the barriers at a row's end.  Loads one step ahead
// gain 2 %, more registers for three CTAs an SM instead of four lose 9 %.
template <class T>
__global__ void __launch_bounds__(kPlainThreads, 4) plain_kernel(const __grid_constant__ WarpParams A) {
    constexpr int E = WordOf<T>::kElems, kWarps = kPlainThreads / 32, U = 16 / E;
    __shared__ PlainShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = uniform(tid / 32), lane = tid % 32;
    const int64_t r = blockIdx.x / C;
    const int64_t base = min(A.V, (int64_t)rank * A.slice);
    const int n = (int)(min(A.V, base + A.slice) - base);
    const T *z = static_cast<const T *>(A.z) + r * A.zs + base;
    const int shift = (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
    const uint4 *words = reinterpret_cast<const uint4 *>(z - shift);
    const int W = n > 0 ? (n + shift + E - 1) / E : 0;
    const int w0 = shift ? 1 : 0, w1 = (n + shift) / E;   // whole words
    if (tid < 32) {
        sh.tab.x[lane] = kPow2[lane].x;
        sh.tab.y[lane] = kPow2[lane].y;
    }
    wait_for_primary_grid();
    const float temp = uniform(A.temperature ? A.temperature[r] : 1.f);
    if (tid == 64) {
        const double i = 1.0 / (double)temp, c = i * 1.4426950408889634;
        sh.ih = (float)i;
        sh.il = (float)(i - (double)sh.ih);
        sh.ch = (float)c;
        sh.cl = (float)(c - (double)sh.ch);
    }
    __syncthreads();
    RowScale S = {-INFINITY, sh.ih, sh.il, sh.ch, sh.cl, -85.f * temp};

    // U words of a lane, 32 apart; what lies outside the slice is -inf
    auto fetch = [&](int w, uint4 (&v)[U]) {
        if (w - lane >= w0 && w - lane + 32 * U <= w1) {
#pragma unroll
            for (int j = 0; j < U; ++j) v[j] = __ldg(words + w + 32 * j);
        } else {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int at = w + 32 * j;
                if (at >= w0 && at < w1) {
                    v[j] = __ldg(words + at);
                } else {
                    T q[E];
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const int e = at * E - shift + i;
                        q[i] = e >= 0 && e < n ? z[e] : minus_inf<T>();
                    }
                    memcpy(&v[j], q, 16);
                }
            }
        }
    };
    auto spread = [&](const uint4 (&v)[U], float (&x)[16]) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            float y[E];
            unpack<T>(v[j], y);
#pragma unroll
            for (int i = 0; i < E; ++i) x[j * E + i] = y[i];
        }
    };

    // every warp takes a run of words
    const int run = (W + kPlainThreads - 1) / kPlainThreads * 32;
    const int s0 = min(W, run * warp), s1 = min(W, s0 + run);
    // (a run ends inside a lane's words: what follows is the next run's)
    auto outside = [&](int w, float (&x)[16], float instead) {
        if (w - lane + 32 * U > s1)
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (w + 32 * j >= s1)
#pragma unroll
                    for (int i = 0; i < E; ++i) x[j * E + i] = instead;
    };
    auto largest_of = [&](float x) -> float {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, d));
        return uniform(x);
    };
    // near zero, in pairs, as far as that goes
    Mass a;
    int w = s0 + lane;
    uint4 v[U];
    fetch(w, v);
    {
        Mass2 near;
        NearScale N = near_scale(S, temp, 0);
        int octave = 0;
        float hi = -INFINITY, top = -INFINITY;
        N.lo = INFINITY;
#pragma unroll 1
        for (; w - lane < s1; w += 32 * U) {
            float x[16];
            spread(v, x);
            if (w - lane + 32 * U < s1) fetch(w + 32 * U, v);
            outside(w, x, N.lo < INFINITY ? N.lo : -INFINITY);   // (2^-120: nothing)
            float most = x[0], least = x[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) {
                most = fmaxf(most, x[i]);
                least = fminf(least, x[i]);
            }
            if (!__all_sync(0xffffffffu, most <= hi && least >= N.lo)) {
                float high = most, low = least;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, d));
                    low = fminf(low, __shfl_xor_sync(0xffffffffu, low, d));
                }
                high = uniform(high);
                low = uniform(low);
                int up = octave;
                if (high > hi) {
                    if (!(fabsf(high) <= kNear * temp)) break;
                    up = near_octave(high, S);
                }
                if (!(low >= (float)(up - kNearDepth) * (kLn2 * temp))) break;
                if (hi > -INFINITY) near.scale(exp2f((float)max(octave - up, -126)));
                octave = up;
                hi = (float)octave * (kLn2 * temp);
                N = near_scale(S, temp, octave);
            }
            top = fmaxf(top, most);
#pragma unroll
            for (int i = 0; i < 16; i += 2) near.add(near_weights(x[i], x[i + 1], N, sh.tab));
        }
        top = largest_of(top);
        if (top > -INFINITY) {
            S.m = top;
            const dd2 v = whole_mass(mul_dd(near.value(), near_to_max(S, &sh.tab, octave)));
            const dd2 start = add_dd({4.f, 0.f}, v);
            a.h = start.h;
            a.l = start.l;
            // (a NaN shows in the sum alone)
            if (__any_sync(0xffffffffu, !(a.h < INFINITY))) S.m = __int_as_float(0x7fffffff);
        }
    }
    // the rest relative to the maximum so far
#pragma unroll 1
    for (; w - lane < s1; w += 32 * U) {
        float x[16];
        fetch(w, v);
        spread(v, x);
        outside(w, x, -INFINITY);
        float most = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) most = max_nan(most, x[i]);
        if (__any_sync(0xffffffffu, !(most <= S.m))) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, d));
            const float old = S.m;
            S.m = max_nan(old, uniform(most));
            const float2 by = weight_of(old, S, &sh.tab);   // (of -inf: 0)
            const dd2 v = mul_dd(a.value(), {by.x, by.y}), start = add_dd({4.f, 0.f}, v);
            a.h = start.h;
            a.l = start.l;
        }
        if (!(fabsf(S.m) < INFINITY)) continue;
#pragma unroll
        for (int h = 0; h < 16; h += 4) {
            float2 y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = weight(x[h + i], S, sh.tab);
#pragma unroll
            for (int i = 0; i < 4; ++i) a.add(y[i]);
        }
    }
    __syncwarp();
    {
        const dd2 own = warp_sum_dd(a.value());
        if (lane == 0) {
            sh.run_top[warp] = S.m;
            sh.run_mass[warp] = own;
        }
    }
    __syncthreads();
    // a warp's 32 masses relative to their tops, as relative to m
    auto rebase = [&](float top, dd2 mass, float m) -> dd2 {
        RowScale to = S;
        to.m = m;
        const float2 by = weight_of(fabsf(m) < INFINITY ? top : -INFINITY, to, &sh.tab);
        // (a mass counts if its largest element has weight)
        return by.x > 0.f ? mul_dd(mass, {by.x, by.y}) : dd2{0.f, 0.f};
    };
    if (warp == 0) {
        const float own = lane < kWarps ? sh.run_top[lane] : -INFINITY;
        const float top = largest_of(own);
        const dd2 mass = warp_sum_dd(rebase(own, lane < kWarps ? sh.run_mass[lane] : dd2{0.f, 0.f}, top));
        if (lane == 0) {
            sh.top = top;
            sh.slice_mass = mass;
            sh.pick = -1;
        }
    }
    cluster.sync();
    float top = -INFINITY;
    dd2 mass = {0.f, 0.f};
    if (lane < C) {
        const PlainShared *o = cluster.map_shared_rank(&sh, lane);
        top = o->top;
        mass = o->slice_mass;
    }
    const float m = largest_of(top);
    const dd2 own = rebase(top, mass, m);
    cluster_arrive_all();  // the last access to another CTA's shared memory is made
    float *out = A.probs ? A.probs + r * A.ps + base : nullptr;
    const bool bad = !(m < INFINITY) || !(temp >= kColdest && temp <= kHottest);
    if (bad || m == -INFINITY) {
        if (rank == 0 && tid == 0) {
            atomicOr(A.status, bad ? SV_STATUS_BAD_VALUE : SV_STATUS_ZERO_MASS);
            if (A.token) A.token[r] = -1;
        }
        if (out)
#pragma unroll 1
            for (int e = tid; e < n; e += kPlainThreads) out[e] = 0.f;
        cluster_wait_all();
        return;
    }
    S.m = m;
    // the first rank, then run, whose running mass passes the goal
    dd2 goal = {0.f, 0.f}, at = {0.f, 0.f};   // (warp 0)
    if (warp == 0) {
        const dd2 upto = warp_scan_dd(own, lane);
        const dd2 total = shfl_dd(upto, 31);
        if (lane == 0) {
            sh.total = total.h;
            sh.slice = {z, words, base, n, shift, 0, S};
        }
        if (A.token) {
            const double g = A.u[r] * ((double)total.h + (double)total.l);   // rounded as in 64 bits
            const float gh = (float)g;
            goal = {gh, (float)(g - (double)gh)};
            const unsigned some = __ballot_sync(0xffffffffu, own.h > 0.f);
            const unsigned over = __ballot_sync(0xffffffffu, own.h > 0.f && less_dd(goal, upto));
            const int holder = over ? __ffs(over) - 1 : 31 - __clz(some);
            if (holder == rank) {
                if (rank > 0) at = shfl_dd(upto, rank - 1);
                const dd2 part = rebase(lane < kWarps ? sh.run_top[lane] : -INFINITY,
                                        lane < kWarps ? sh.run_mass[lane] : dd2{0.f, 0.f}, m);
                const dd2 reach = add_dd(at, warp_scan_dd(part, lane));
                const unsigned runs = __ballot_sync(0xffffffffu, part.h > 0.f);
                const unsigned past = __ballot_sync(0xffffffffu, part.h > 0.f && less_dd(goal, reach));
                const int pick = past ? __ffs(past) - 1 : 31 - __clz(runs);
                if (pick > 0) at = shfl_dd(reach, pick - 1);
                if (lane == 0) sh.pick = pick;
            }
        }
    }
    __syncthreads();
    if (out) {
        const float inv = 1.f / sh.total;
        const bool vec = ((reinterpret_cast<uintptr_t>(out) - (uintptr_t)shift * 4u) & 15u) == 0;
#pragma unroll 1
        for (int w = s0 + lane; w - lane < s1; w += 32 * U) {
            float x[16];
            fetch(w, v);
            spread(v, x);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                float y[E];
#pragma unroll
                for (int i = 0; i < E; ++i) y[i] = fast_weight(x[j * E + i], S) * inv;
                if (w + 32 * j < s1) store_probs<E>(out, (w + 32 * j) * E - shift, n, vec, y);
            }
        }
    }
    const int pick = uniform(sh.pick);
    if (pick >= 0) {
        const int r0 = max(0, run * pick * E - shift), r1 = min(n, run * (pick + 1) * E - shift);
        draw_element<T, kPlainThreads, 8>(sh.slice, sh.tab, sh.part_mass, 0, r0, r1, goal, at, A.token + r);
    }
    cluster_wait_all();
}

}  // namespace sv
