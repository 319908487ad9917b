// sv_warp.cuh -- the warp of logits into probability rows (temperature, top-k,
// top-p, min-p) and draws from them.
//
// Every filter keeps a prefix of the row's order (logit descending, index
// ascending), so the kept set is one threshold on the 64-bit composite
// (ordered logit bits, ~index).  A row's thresholds are found by bisection:
// counts for top-k, masses for top-p; min-p gives its logit directly.
//
// Masses decide which tokens stay and which one is drawn, and must give the
// answers of a 64-bit evaluation.  fp64 runs at 1/64 of the fp32 rate here, so
// a weight exp((z - max) / T) is formed as a pair of floats (weight()): the
// exponent and the table-and-polynomial value keep their rounding errors in
// the low part, good to about 5e-12 relative.
#pragma once

#include "sv_cache.cuh"

namespace sv {

constexpr int kWarpThreads = 1024;
constexpr int kWarpWarps = kWarpThreads / 32;

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
    int32_t R;
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

// 2^(j / 32), j = -16..16, as hi + lo, in shared memory.
struct ExpTable {
    float2 t[33];
};

__device__ __forceinline__ void fill_table(ExpTable &tab) {
    for (int i = threadIdx.x; i < 33; i += blockDim.x) {
        const double x = exp2((i - 16) / 32.0);
        const float h = (float)x;
        tab.t[i] = make_float2(h, (float)(x - (double)h));
    }
}

struct RowScale {
    float m, ch, cl;  // row maximum; log2(e) / temperature as hi + lo
};

__device__ __forceinline__ RowScale row_scale(float m, float temperature) {
    const double c = 1.4426950408889634 / (double)temperature;
    RowScale s;
    s.m = m;
    s.ch = (float)c;
    s.cl = (float)(c - (double)s.ch);
    return s;
}

// exp((z - max) / T) as x + y (hi, lo); 0 below 2^-100.
//   z - max = d + dl exactly; (d + dl) * c = e + el; e = n + j/32 + r with
//   |r| <= 1/64; 2^e = 2^n T_j (1 + s), s = 2^r - 1 by its series to r^5.
__device__ __forceinline__ float2 weight(float z, const RowScale &S, const ExpTable &tab) {
    const float d = z - S.m;
    const float e = d * S.ch;
    if (!(e >= -100.f)) return make_float2(0.f, 0.f);
    const float bb = d - z;
    const float dl = (z - (d - bb)) - (S.m + bb);
    float el = fmaf(d, S.ch, -e);
    el = fmaf(d, S.cl, el);
    el = fmaf(dl, S.ch, el);
    const float k = rintf(e * 32.f);
    const float r = fmaf(k, -0.03125f, e);  // exact
    const int ki = (int)k;
    const int n = (ki + 16) >> 5, j = ki - n * 32;  // j in [-16, 15]
    const float2 T = tab.t[j + 16];
    const float ph = r * 0.693147182f;
    float pl = fmaf(r, 0.693147182f, -ph);
    pl = fmaf(r, -1.90465421e-9f, pl);
    pl = fmaf(el, 0.693147182f, pl);
    float q = fmaf(r, 1.33335581e-3f, 9.61812911e-3f);
    q = fmaf(r, q, 5.55041087e-2f);
    q = fmaf(r, q, 2.40226507e-1f);
    const float t = fmaf(r * r, q, pl);
    const float sh = ph + t, sl = t - (sh - ph);
    const float u = T.x * sh;
    const float ul = fmaf(T.x, sl, fmaf(T.x, sh, -u)) + fmaf(T.y, sh, T.y);
    const float wh = T.x + u, wl = (u - (wh - T.x)) + ul;
    const float scale = __int_as_float((n + 127) << 23);
    return make_float2(wh * scale, wl * scale);
}

// A running sum of weights.
struct Mass {
    float h = 0.f, l = 0.f;
    __device__ __forceinline__ void add(float2 w) {
        const float s = h + w.x, b = s - h;
        l += ((h - (s - b)) + (w.x - b)) + w.y;
        h = s;
    }
    __device__ __forceinline__ double value() const { return (double)h + (double)l; }
};

template <class T>
__device__ __forceinline__ T block_sum(T x, T *sm) {
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = x;
    __syncthreads();
    T s = 0;
    for (int w = 0; w < kWarpWarps; ++w) s += sm[w];  // one order on every thread
    return s;
}

template <class T>
__global__ void __launch_bounds__(kWarpThreads) warp_kernel(const __grid_constant__ WarpParams A) {
    __shared__ ExpTable tab;
    __shared__ double sm[kWarpWarps];
    __shared__ uint64_t smk[kWarpWarps];
    __shared__ int64_t found;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t r = blockIdx.x;
    const T *z = static_cast<const T *>(A.z) + r * A.zs;
    const int64_t V = A.V;
    auto at = [&](int64_t v) -> float { return to_f32<T>(z[v]); };
    fill_table(tab);
    if (tid == 0) found = -1;

    // the row's first element in the order; NaN and +inf counted as bad
    uint64_t top = 0;
    int bad = 0;
    for (int64_t v = tid; v < V; v += kWarpThreads) {
        const float x = at(v);
        bad |= !(x < INFINITY);
        const uint64_t c = composite(x, v);
        top = c > top ? c : top;
    }
    for (int d = 16; d > 0; d >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, top, d);
        top = o > top ? o : top;
    }
    if (lane == 0) smk[warp] = top;
    bad = __syncthreads_or(bad);
    for (int w = 0; w < kWarpWarps; ++w) top = smk[w] > top ? smk[w] : top;
    const float m = unordered((uint32_t)(top >> 32));
    const float temp = A.temperature ? A.temperature[r] : 1.f;
    bad |= !(temp > 0.f && temp < INFINITY);
    if (bad || m == -INFINITY) {
        if (tid == 0) {
            atomicOr(A.status, bad ? SV_STATUS_BAD_VALUE : SV_STATUS_ZERO_MASS);
            if (A.token) A.token[r] = -1;
        }
        if (A.probs)
            for (int64_t v = tid; v < V; v += kWarpThreads) A.probs[r * A.ps + v] = 0.f;
        return;
    }
    const RowScale S = row_scale(m, temp);

    auto count_from = [&](uint64_t thr) -> int64_t {  // elements at or above thr
        int64_t c = 0;
        for (int64_t v = tid; v < V; v += kWarpThreads) c += composite(at(v), v) >= thr;
        return block_sum<int64_t>(c, reinterpret_cast<int64_t *>(smk));
    };
    auto mass_from = [&](uint64_t thr) -> double {  // their mass
        Mass a;
        for (int64_t v = tid; v < V; v += kWarpThreads) {
            const float x = at(v);
            if (composite(x, v) >= thr) a.add(weight(x, S, tab));
        }
        return block_sum<double>(a.value(), sm);
    };

    uint64_t thr = 0;  // kept: composite >= thr
    const int64_t k = A.top_k ? A.top_k[r] : 0;
    if (k > 0 && k < V) {
        uint64_t lo = 0, hi = top;  // count(lo) >= k; the largest such threshold
        while (lo < hi) {
            const uint64_t mid = lo + (hi - lo) / 2 + 1;
            if (count_from(mid) >= k) lo = mid;
            else hi = mid - 1;
        }
        thr = lo;
    }
    const float p = A.top_p ? A.top_p[r] : 1.f;
    if (p < 1.f) {
        const double goal = (double)p * mass_from(thr);
        // the smallest threshold whose successors (strictly before it) weigh less than the goal
        uint64_t lo = thr, hi = top;
        while (lo < hi) {
            const uint64_t mid = lo + (hi - lo) / 2;
            if (mass_from(mid + 1) < goal) hi = mid;
            else lo = mid + 1;
        }
        thr = lo;
    }
    const float mp = A.min_p ? A.min_p[r] : 0.f;
    if (mp > 0.f) {
        uint64_t t = top;
        if (mp <= 1.f) {
            const double edge = (double)m + (double)temp * log((double)mp);
            float f = (float)edge;
            if ((double)f < edge) f = nextafterf(f, INFINITY);
            t = (uint64_t)ordered(f) << 32;
        }
        t = t < top ? t : top;
        thr = t > thr ? t : thr;
    }

    const double total = mass_from(thr);
    if (A.token && A.u) {
        const double goal = A.u[r] * total;
        // each warp takes a run of the row: its mass, the run that crosses the
        // goal, then that run again in steps of 32
        const int64_t run = (V + kWarpWarps - 1) / kWarpWarps;
        const int64_t v0 = min(V, run * warp), v1 = min(V, v0 + run);
        Mass a;
        for (int64_t v = v0 + lane; v < v1; v += 32) {
            const float x = at(v);
            if (composite(x, v) >= thr) a.add(weight(x, S, tab));
        }
        double w = a.value();
        for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
        __syncthreads();
        if (lane == 0) sm[warp] = w;
        __syncthreads();
        double before = 0;
        int mine = -1;
        for (int i = 0; i < kWarpWarps; ++i) {
            if (sm[i] > 0) mine = i;
            if (before + sm[i] > goal) break;
            if (sm[i] > 0 && i + 1 < kWarpWarps) {
                bool more = false;
                for (int x = i + 1; x < kWarpWarps; ++x) more |= sm[x] > 0;
                if (!more) break;
            }
            before += sm[i];
        }
        if (warp == mine) {
            int64_t last = -1, hit = -1;
            for (int64_t v = v0; v < v1 && hit < 0; v += 32) {
                float2 x = make_float2(0.f, 0.f);
                if (v + lane < v1) {
                    const float y = at(v + lane);
                    if (composite(y, v + lane) >= thr) x = weight(y, S, tab);
                }
                double inc = (double)x.x + (double)x.y;
                const bool has = inc > 0;
                for (int d = 1; d < 32; d <<= 1) {
                    const double o = __shfl_up_sync(0xffffffffu, inc, d);
                    if (lane >= d) inc += o;
                }
                const unsigned any = __ballot_sync(0xffffffffu, has);
                const unsigned over = __ballot_sync(0xffffffffu, has && before + inc > goal);
                if (any) last = v + 31 - __clz(any);
                if (over) hit = v + __ffs(over) - 1;
                before += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) found = hit >= 0 ? hit : last;
        }
        __syncthreads();
        if (tid == 0) A.token[r] = (int32_t)found;
    }
    if (A.probs) {
        const double inv = 1.0 / total;
        const float ih = (float)inv;
        for (int64_t v = tid; v < V; v += kWarpThreads) {
            const float x = at(v);
            float o = 0.f;
            if (composite(x, v) >= thr) o = weight(x, S, tab).x * ih;
            A.probs[r * A.ps + v] = o;
        }
    }
}

}  // namespace sv
