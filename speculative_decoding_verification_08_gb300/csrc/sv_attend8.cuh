// sv_attend8.cuh -- attention of few new rows over a paged cache of 8-bit values,
// on the fifth-generation tensor cores.
//
// Rows are packed as in sv_attend.cuh (the G query heads of a kv head side by side),
// but the products are the transposed ones: a key block's 128 slots are the 128
// lanes of tensor memory and the tile's up to kRows8 rows its columns,
//   S^T = K Q^T,   O^T += V^T P^T.
// So a thread has one slot and all rows: the exponentials of a block are spread
// over four warps however few rows there are, a slot's scales are two numbers of
// its thread, and the tensor cores are not fed empty rows.
//
// Keys go to the tensor cores as the e4m3 codes they are.  The queries become 8-bit
// floats beside them: relative to one power of two for the tile, each value is the
// sum of 3 (bf16) or 4 (fp16) e5m2 numbers, the nearest to what the ones before it
// left (3 significant bits each, 2 and the sign of the rest), exact down to 2^-24 of
// the tile's largest and good to 2^-33 of it below.  The parts are columns of their own
// (their products are added in fp32 by the softmax threads), so a block of keys is
// read from shared memory once.
// Values need their slots' axis contiguous for the second product, which 16-bit types
// have: four warps turn codes into fp16 (exact).  Their scales go into the weights,
// relative to a power of two that follows the largest scale: weight times scale, in
// fp16 and taken 2^7 times as large, is the one rounding between fp32 scores and the
// result (11 bits; what is below 2^-21 of the row's and the scales' largest is rounded
// to steps of 2^-31 of them).
//
// Softmax: weights are relative to a reference per row, which follows the row's
// maximum only when a score is more than 2^8 above it; whether any is, is one vote
// of the 128 threads per block, and finding the new maxima the rare way.  Two groups of
// four warps take the even and the odd blocks of a tile, each with scores, weights,
// outputs and references of its own, and join them at the tile's end.
//
// Work split, partial states and their join: as in sv_attend.cuh.
//
// Warps 0-7 softmax, 8-11 values to fp16, 12 copies (TMA boxes of page pieces), 13
// issues S, 14 issues O, 15 walks the CTA's run, publishes its pieces and prepares
// the queries.  Every wait is bounded, as there.
#pragma once

#include "sv_append8.cuh"
#include "sv_attend.cuh"

namespace sv {

constexpr int kMaxRows8 = 32;   // packed rows of a tile at most
constexpr int kTileCost8 = 3;   // a tile's fixed cost in key blocks
constexpr int kThreads8 = 512;
constexpr int kSoftmaxRegs8 = 168, kOtherRegs8 = 88;
static_assert(256 * kSoftmaxRegs8 + 256 * kOtherRegs8 <= kThreads8 * 128, "register split");
constexpr int kRaw = kKeys * 128;     // a block of codes
constexpr int kRing8 = 3;             // blocks of keys, and of values, in flight
constexpr float kUnset = 3e38f;       // minus the reference of a row that has seen nothing
constexpr int kNoScale = -200;        // below every e8m0 exponent

struct Attend8Params {
    AttendParams a;
    Scales scales;
};

template <class T, int kRows8>
struct Attend8Smem {
    static constexpr int kParts = __is_same(T, __nv_bfloat16) ? 3 : 4;
    // columns of scores: a whole product has a multiple of 16
    static constexpr int kScoreCols = (kParts * kRows8 + 15) / 16 * 16;
    static constexpr int kQuery = kScoreCols * 128;
    static constexpr int kMisc = 3072;
    static constexpr int kQ = kMisc, kK = kQ + 2 * kQuery, kV = kK + kRing8 * kRaw, kVc = kV + kRing8 * kRaw,
                         kP = kVc + 2 * 2 * kRaw, kBytes = kP + 2 * kRaw;
    // O: the groups' first columns, and a whole product's columns
    static constexpr int kOutCols = (kRows8 + 15) / 16 * 16, kOut = 2 * kScoreCols;
    static constexpr uint32_t kCols = kOut + 2 * kOutCols <= 128 ? 128 : kOut + 2 * kOutCols <= 256 ? 256 : 512;
    static_assert(kBytes <= 227 * 1024 && kQ % 1024 == 0 && kQuery % 1024 == 0, "shared memory");
    static_assert(kOut + 2 * kOutCols <= 512, "tensor memory");
};

struct Attend8Shared {
    unsigned long long k_full[kRing8], k_empty[kRing8], v_full[kRing8], v_empty[kRing8];
    unsigned long long s_full[2], s_empty[2], vc_full[2], p_full[2], pv_done[2], q_full[2], q_empty[2], drain[2];
    unsigned long long piece_full[kPieces], piece_empty[kPieces];
    Piece pieces[kPieces];
    uint32_t tmem;
    int32_t dead, b0, last;
    float q_factor[2];          // power of two of a tile's queries, times the score scale
    int64_t skip;
    int64_t sums[kThreads8 / 32];
};
static_assert(sizeof(Attend8Shared) <= 1024, "misc region");

struct __align__(16) Attend8Rows {  // behind it, for each of the two groups
    float minus[2][kMaxRows8];     // minus the rows' references
    float factor[2][kMaxRows8];    // what a new reference makes of sums and outputs
    float across[2][4][kMaxRows8]; // its warps' maxima or sums
    int32_t exponent[2][4];        // its warps' largest scales
};
static_assert(sizeof(Attend8Rows) <= 2048, "misc region");

// As hold() of the 16-bit kernel.
template <uint64_t kLimitNs = kWaitLimitNs>
__device__ __forceinline__ bool hold8(Attend8Shared &sh, unsigned long long *bar, uint32_t parity,
                                      uint32_t *status) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try(bar, parity)) {
        if (*(volatile int32_t *)&sh.dead) return false;
        if (global_ns() - t0 > kLimitNs) {
            *(volatile int32_t *)&sh.dead = 1;
            atomicOr(status, SV_STATUS_TIMEOUT);
            return false;
        }
    }
    return true;
}

struct PieceReader8 {
    int k = 0;
    uint32_t turn = 0;
    // (all lanes) whether there is a piece; it is sh.pieces[k]
    __device__ __forceinline__ bool next(Attend8Shared &sh, uint32_t *status) {
        const bool ok = __all_sync(0xffffffffu, hold8(sh, &sh.piece_full[k], turn, status));
        return ok && sh.pieces[k].n >= 0;
    }
    __device__ __forceinline__ void done(Attend8Shared &sh, int lane) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.piece_empty[k]);
        if (++k == kPieces) {
            k = 0;
            turn ^= 1;
        }
    }
};
constexpr int kPieceReaders8 = 15;

// Barriers of the softmax's threads: a group's 128 (number 1 or 2), or all 256 (3).
// All of them come to each, whatever timed out.
template <int kCount>
__device__ __forceinline__ void softmax_barrier(int number) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(number), "n"(kCount) : "memory");
}
template <int kCount>
__device__ __forceinline__ bool softmax_any(int number, bool x) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred p, q; setp.ne.u32 q, %2, 0;\n"
        "barrier.cta.red.or.pred p, %1, %3, q; selp.u32 %0, 1, 0, p; }"
        : "=r"(r)
        : "r"(number), "r"((uint32_t)x), "n"(kCount)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}

// Joins each of 32 columns over a warp's lanes; lane i gets column i.
template <class F>
__device__ __forceinline__ float across_lanes(float (&v)[32], int lane, F join) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int c = 0; c < d; ++c) {
            const float keep = up ? v[c + d] : v[c], give = up ? v[c] : v[c + d];
            v[c] = join(keep, __shfl_xor_sync(0xffffffffu, give, d));
        }
    }
    return v[0];
}

// Four e4m3 codes as fp16.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Four floats to e5m2 codes, and what the codes leave of them.
__device__ __forceinline__ uint32_t split_off(float (&x)[4]) {
    uint16_t a, b;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(b) : "f"(x[3]), "f"(x[2]));
    const uint32_t w = (uint32_t)a | (uint32_t)b << 16;
    // an e5m2 number is the upper half of an fp16 one
    const uint32_t lo = __byte_perm(w, 0, 0x1404), hi = __byte_perm(w, 0, 0x3424);
    const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    x[0] -= u.x;
    x[1] -= u.y;
    x[2] -= v.x;
    x[3] -= v.y;
    return w;
}

template <class T, int kRows8>
__global__ void __launch_bounds__(kThreads8, 1)
    attend8_kernel(const __grid_constant__ Attend8Params P8, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
    typedef Attend8Smem<T, kRows8> L;
    constexpr int kParts = L::kParts;
    constexpr int kAtOnce = kRows8 < 32 ? kRows8 / 8 : 2;  // columns of scores by eight, as registers allow
    constexpr uint32_t kIdescS = tc::instr_desc_f8(kKeys, L::kScoreCols);
    // (bit 15: A's slots are its rows in memory, as B's)
    constexpr uint32_t kIdescO = tc::instr_desc(false, true, 128, L::kOutCols) | (1u << 15);
    extern __shared__ __align__(1024) char smem[];
    Attend8Shared &sh = *reinterpret_cast<Attend8Shared *>(smem);
    Attend8Rows &shared = *reinterpret_cast<Attend8Rows *>(smem + 1024);
    const AttendParams &A = P8.a;
    const int tid = threadIdx.x, warp = tc::uniform(tid / 32), lane = tid % 32;
    uint32_t *status = A.batch.status;
    const int D = A.head_dim;
    const bool wide = D > 64;  // both halves of 64 values are in use

    if (smem_u32(smem) & 1023) {  // the swizzle counts on it; no room is left to round up
        if (tid == 0) atomicOr(status, SV_STATUS_TIMEOUT);
        return;
    }
    if (warp == 13) tc::tmem_alloc(&sh.tmem, L::kCols);
    if (tid == 0) {
        for (int i = 0; i < kRing8; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], 4);
            mbar_init(&sh.vc_full[i], 4);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 9);
            mbar_init(&sh.drain[i], 1);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&sh.piece_full[i], 1);
            mbar_init(&sh.piece_empty[i], kPieceReaders8);
        }
        sh.dead = 0;
        sh.b0 = -1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // heads of up to 64 values: the other half of the values' rows is zero throughout
    if (!wide)
        for (int i = tid; i < 2 * kRaw / 16; i += kThreads8)
            *reinterpret_cast<uint4 *>(smem + L::kVc + (i / (kRaw / 16) * 2 + 1) * kRaw + i % (kRaw / 16) * 16) =
                make_uint4(0, 0, 0, 0);
    tc::fence_async_smem();
    wait_for_primary_grid();

    // the batch's blocks, and where this CTA's run of them begins
    int64_t c = 0, last_cost = 0;
    for (int32_t b0 = 0; b0 < A.batch.B; b0 += kThreads8) {
        const int32_t b = b0 + tid < A.batch.B ? b0 + tid : -1;
        last_cost = sequence_cost<kRows8, kTileCost8>(A, b, lane);
        c += last_cost;
        if (blockIdx.x == 0 && b >= 0 && load_sequence(A.batch, b).bad)
            atomicOr(status, SV_STATUS_BAD_LENGTH);
    }
    for (int d = 16; d > 0; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
    if (lane == 0) sh.sums[warp] = c;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    int64_t total = 0;
    for (int w = 0; w < kThreads8 / 32; ++w) total += sh.sums[w];
    const int32_t ctas = (int32_t)min((int64_t)gridDim.x, max((int64_t)1, total));
    const int64_t u0 = quotient((int64_t)blockIdx.x * total, ctas),
                  u1 = quotient(((int64_t)blockIdx.x + 1) * total, ctas);
    const bool idle = total == 0 || (int32_t)blockIdx.x >= ctas || u0 >= u1;
    if (!idle) {
        int64_t base = 0;
        for (int32_t b0 = 0; b0 < A.batch.B; b0 += kThreads8) {
            const int32_t b = b0 + tid < A.batch.B ? b0 + tid : -1;
            const int64_t own =
                A.batch.B <= kThreads8 ? last_cost : sequence_cost<kRows8, kTileCost8>(A, b, lane);
            int64_t inc = own;
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += o;
            }
            __syncthreads();
            if (lane == 31) sh.sums[warp] = inc;
            __syncthreads();
            int64_t at = base;
            for (int w = 0; w < kThreads8 / 32; ++w) {
                if (w < warp) at += sh.sums[w];
                base += sh.sums[w];
            }
            if (own > 0 && at + inc - own <= u0 && u0 < at + inc) {
                sh.b0 = b;
                sh.skip = u0 - (at + inc - own);
            }
            if (base > u0) break;
        }
        __syncthreads();
    }
    const uint32_t tmem = sh.tmem;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs8));
        if (warp == 15) {
            // ---- the schedule, and the queries of its pieces -------------------
            Walker<kRows8, kTileCost8> walk;
            walk.left = 0;
            if (!idle) walk.start(A, sh.b0, sh.skip, u0, u1 - u0, total, ctas, lane);
            int k = 0;
            uint32_t turn = 1, qn = 0;
            for (bool more = true; more;) {
                Piece p;
                more = walk.next(A, p);
                if (!more) p.n = -1;
                if (!__all_sync(0xffffffffu, hold8<kPieceLimitNs>(sh, &sh.piece_empty[k], turn, status))) break;
                if (lane == 0) {
                    sh.pieces[k] = p;
                    mbar_arrive(&sh.piece_full[k]);
                }
                __syncwarp();
                if (++k == kPieces) {
                    k = 0;
                    turn ^= 1;
                }
                if (p.n <= 0) continue;
                const int qb = qn & 1;
                if (!__all_sync(0xffffffffu, hold8<kPieceLimitNs>(sh, &sh.q_empty[qb], ((qn >> 1) & 1) ^ 1, status)))
                    break;
                ++qn;
                // four values to a lane, eight rows' loads in flight
                auto load = [&](int r) -> uint2 {
                    if (r >= p.rows || lane * 4 >= D || A.q_mode == 2) return make_uint2(0, 0);
                    const int pr = p.row + r, j = A.by_group.div(pr);
                    return __ldg(reinterpret_cast<const uint2 *>(
                        static_cast<const uint16_t *>(A.q) + (int64_t)(p.token + j) * A.q_st[0] +
                        (p.h * A.group + (pr - j * A.group)) * A.q_st[1] + lane * 4));
                };
                auto bits = [&](const float2 &f) -> uint32_t {  // of the larger finite magnitude
                    const uint32_t a = __float_as_uint(f.x) & 0x7fffffffu, b = __float_as_uint(f.y) & 0x7fffffffu;
                    return max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u);
                };
                uint32_t top = 0;
                for (int r0 = 0; r0 < p.rows; r0 += 8) {
                    uint2 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = load(r0 + i);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        top = max(top, max(bits(pair_of(x[i].x, T())), bits(pair_of(x[i].y, T()))));
                }
                for (int d = 16; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                // the largest is brought to 57344 (e5m2's) or less
                const int e = min(max((int)(top >> 23) - 127 - 15 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), -100), 120);
                const float f = A.q_mode == 1 ? -power_of_two(-e) : power_of_two(-e);
                char *to = smem + L::kQ + qb * L::kQuery;
                for (int r0 = 0; r0 < kRows8; r0 += 8) {
                    uint2 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = load(r0 + i);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 a = pair_of(x[i].x, T()), b = pair_of(x[i].y, T());
                        float y[4] = {a.x * f, a.y * f, b.x * f, b.y * f};
                        // an infinity makes its row NaN, as a NaN does
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            if (!(fabsf(y[m]) <= 57344.f)) y[m] = __uint_as_float(0x7fffffffu);
#pragma unroll
                        for (int part = 0; part < kParts; ++part)
                            *reinterpret_cast<uint32_t *>(to + (part * kRows8 + r0 + i) * 128 +
                                                          ((lane / 4) ^ i) * 16 + lane % 4 * 4) = split_off(y);
                    }
                }
                if (lane == 0) sh.q_factor[qb] = A.scale_log2 * power_of_two(e);
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full[qb]);
            }
        } else if (warp == 12) {
            // ---- copies of codes ------------------------------------------------
            const int boxes = kKeys / A.piece;
            const bool active = lane < boxes;
            int kn = 0, vn = 0;  // blocks copied so far
            PieceReader8 reader;
            bool ok = true;
            while (ok && reader.next(sh, status)) {
                const Piece p = sh.pieces[reader.k];
                reader.done(sh, lane);
                if (p.n == 0) continue;
                const int32_t *table = A.batch.pages + p.b * A.batch.pages_stride;
                const int first = A.window > 0 ? p.past + A.by_group.div(p.row) - A.window + 1 : 0;
                auto page_of = [&](int i) -> int {
                    const int s0 = (p.lo + i) * kKeys + lane * A.piece;
                    if (!active || i >= p.n || s0 >= p.end || s0 + A.piece <= first) return kNoPage;
                    return __ldg(table + A.by_page.div(s0));
                };
                auto checked = [&](int id) -> int {
                    if (id != kNoPage && (id < 0 || id >= A.batch.num_pages)) {
                        atomicOr(status, SV_STATUS_BAD_PAGE);
                        id = kNoPage;
                    }
                    return id;
                };
                auto load = [&](const CUtensorMap &map, int ring, unsigned long long *full, unsigned long long *empty,
                                int &n, int i, int id) {
                    const int st = n % kRing8;
                    ok = ok && __all_sync(0xffffffffu, hold8(sh, &empty[st], (n / kRing8 & 1) ^ 1, status));
                    if (ok) {
                        if (lane == 0) mbar_arrive_expect_tx(&full[st], kRaw);
                        __syncwarp();
                        if (active) {
                            const int s0 = (p.lo + i) * kKeys + lane * A.piece;
                            tc::load_box(smem + ring + st * kRaw + lane * A.piece * 128, &map, 0, p.h,
                                         s0 - A.by_page.div(s0) * A.batch.page_size, id, &full[st]);
                        }
                        ++n;
                    }
                    __syncwarp();
                };
                auto keys = [&](int i, int id) { load(kmap, L::kK, sh.k_full, sh.k_empty, kn, i, id); };
                // keys run a block ahead of values, page ids a block ahead of keys
                int id0 = checked(page_of(0)), id1 = page_of(1), id2 = page_of(2);
                keys(0, id0);
                for (int i = 0; i < p.n; ++i) {
                    const int id3 = page_of(i + 3);
                    id1 = checked(id1);
                    if (i + 1 < p.n) keys(i + 1, id1);
                    load(vmap, L::kV, sh.v_full, sh.v_empty, vn, i, id0);
                    id0 = id1;
                    id1 = id2;
                    id2 = id3;
                }
            }
            // the last copies have landed before the CTA may end
            for (int n = max(0, kn - kRing8); n < kn; ++n) mbar_wait(&sh.k_full[n % kRing8], n / kRing8 & 1);
            for (int n = max(0, vn - kRing8); n < vn; ++n) mbar_wait(&sh.v_full[n % kRing8], n / kRing8 & 1);
        } else if (warp == 13) {
            // ---- scores ---------------------------------------------------------
            const uint32_t tm = (uint32_t)tc::uniform((int)tmem);
            const uint64_t k_desc = tc::smem_desc(smem_u32(smem + L::kK), 16, 1024);
            const uint64_t q_desc = tc::smem_desc(smem_u32(smem + L::kQ), 16, 1024);
            const int steps = (D + 31) / 32;
            uint32_t n = 0, qn = 0, used[2] = {0, 0};  // blocks, tiles, blocks of each group
            PieceReader8 reader;
            bool ok = true;  // a wait gave up: nothing more is issued or handed back
            while (ok && reader.next(sh, status)) {
                const int blocks = tc::uniform(sh.pieces[reader.k].n);
                reader.done(sh, lane);
                if (blocks == 0) continue;
                const uint32_t qb = qn & 1;
                ok = ok && __all_sync(0xffffffffu, hold8<kPieceLimitNs>(sh, &sh.q_full[qb], (qn >> 1) & 1, status));
                ++qn;
                for (int i = 0; i < blocks && ok; ++i, ++n) {
                    const uint32_t st = n % kRing8, sb = i & 1;
                    const uint32_t turn = sb ? used[1]++ : used[0]++;
                    ok = __all_sync(0xffffffffu, hold8(sh, &sh.k_full[st], n / kRing8 & 1, status));
                    ok = ok && __all_sync(0xffffffffu, hold8(sh, &sh.s_empty[sb], (turn & 1) ^ 1, status));
                    if (!ok) break;
                    tc::fence_after();
                    if (tc::elect()) {
                        const uint64_t kd = k_desc + st * (kRaw / 16), qd = q_desc + qb * (L::kQuery / 16);
                        for (int s = 0; s < steps; ++s)
                            tc::mma_f8(tm + sb * L::kScoreCols, kd + s * 2, qd + s * 2, kIdescS, s > 0);
                        tc::commit(&sh.k_empty[st]);
                        tc::commit(&sh.s_full[sb]);
                        if (i + 1 == blocks) tc::commit(&sh.q_empty[qb]);
                    }
                    __syncwarp();
                }
            }
            if (tc::elect()) tc::commit(&sh.drain[0]);
            __syncwarp();
            mbar_wait(&sh.drain[0], 0);
        } else if (warp == 14) {
            // ---- outputs --------------------------------------------------------
            const uint32_t tm = (uint32_t)tc::uniform((int)tmem) + L::kOut;
            const uint64_t v_desc = tc::smem_desc(smem_u32(smem + L::kVc), kRaw, 1024);
            const uint64_t p_desc = tc::smem_desc(smem_u32(smem + L::kP), kRaw, 1024);
            uint32_t used[2] = {0, 0};
            PieceReader8 reader;
            bool ok = true;
            while (ok && reader.next(sh, status)) {
                const int blocks = tc::uniform(sh.pieces[reader.k].n);
                reader.done(sh, lane);
                for (int i = 0; i < blocks && ok; ++i) {
                    const uint32_t b = i & 1, turn = (b ? used[1]++ : used[0]++) & 1;
                    ok = __all_sync(0xffffffffu, hold8(sh, &sh.vc_full[b], turn, status));
                    ok = ok && __all_sync(0xffffffffu, hold8(sh, &sh.p_full[b], turn, status));
                    if (!ok) break;
                    tc::fence_after();
                    if (tc::elect()) {
                        const uint64_t vd = v_desc + b * (2 * kRaw / 16), pd = p_desc + b * (kRaw / 16);
#pragma unroll
                        for (int s = 0; s < kKeys / 16; ++s)
                            tc::mma_ss(tm + b * L::kOutCols, vd + s * (2048 / 16), pd + s * (2048 / 16), kIdescO, i > 1 || s > 0);
                        tc::commit(&sh.pv_done[b]);
                    }
                    __syncwarp();
                }
            }
            if (tc::elect()) tc::commit(&sh.drain[1]);
            __syncwarp();
            mbar_wait(&sh.drain[1], 0);
        } else {
            // ---- values to fp16 ---------------------------------------------------
            const int t = tid - 256;
            // a thread's chunk of 16 values and its slot of a group (eight lanes' chunks
            // lie in different banks)
            const int ch = wide ? t % 8 : t % 4, u = t / 4;
            const int slot0 = wide ? t / 8 : (u >> 3) * 8 + ((u & 1) << 2) + ((u >> 1) & 3);
            const int rounds = wide ? 8 : 4, per = wide ? 16 : 32;
            const bool odd_first = wide ? ch >= 4 : u & 1;
            uint32_t n = 0, used[2] = {0, 0};
            PieceReader8 reader;
            bool ok = true;
            while (ok && reader.next(sh, status)) {
                const int blocks = sh.pieces[reader.k].n;
                // slots from the tile's end on: whatever lies there, zeros
                const int end = sh.pieces[reader.k].end - sh.pieces[reader.k].lo * kKeys;
                reader.done(sh, lane);
                for (int i = 0; i < blocks && ok; ++i, ++n) {
                    const uint32_t st = n % kRing8, b = i & 1, turn = b ? used[1]++ : used[0]++;
                    const int here = end - i * kKeys;
                    ok = __all_sync(0xffffffffu, hold8(sh, &sh.v_full[st], n / kRing8 & 1, status));
                    if (ok && turn > 0)
                        ok = __all_sync(0xffffffffu, hold8(sh, &sh.pv_done[b], (turn - 1) & 1, status));
                    if (!ok) break;
                    const char *from = smem + L::kV + st * kRaw;
                    char *to = smem + L::kVc + b * 2 * kRaw + (ch / 4) * kRaw;
#pragma unroll 4
                    for (int k = 0; k < rounds; ++k) {
                        const int slot = k * per + slot0, x = slot & 7;
                        uint4 w = *reinterpret_cast<const uint4 *>(from + slot * 128 + ((ch ^ x) * 16));
                        if (slot >= here) w = make_uint4(0, 0, 0, 0);
                        uint4 lo, hi;
                        codes_to_half(w.x, lo.x, lo.y);
                        codes_to_half(w.y, lo.z, lo.w);
                        codes_to_half(w.z, hi.x, hi.y);
                        codes_to_half(w.w, hi.z, hi.w);
                        const int j = (ch % 4) * 2;
                        char *row = to + slot * 128;
                        *reinterpret_cast<uint4 *>(row + (((j + (odd_first ? 1 : 0)) ^ x) * 16)) = odd_first ? hi : lo;
                        *reinterpret_cast<uint4 *>(row + (((j + (odd_first ? 0 : 1)) ^ x) * 16)) = odd_first ? lo : hi;
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh.vc_full[b]);
                        mbar_arrive(&sh.v_empty[st]);
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs8));
        // ---- softmax: a slot to a thread ------------------------------------------
        const int g = warp / 4, gw = warp % 4, gt = gw * 32 + lane;
        const uint32_t lanes_at = tmem + ((uint32_t)(gw * 32) << 16);
        const uint32_t t_s = lanes_at + g * L::kScoreCols, t_o = lanes_at + L::kOut;
        uint32_t used = 0, others = 0, qn = 0;  // blocks of this group and of the other, tiles
        PieceReader8 reader;
        for (;;) {
            // (all eight warps go on, or none: they meet at barriers; and the last
            // tile's outputs have been read)
            if (softmax_any<256>(3, !reader.next(sh, status))) break;
            const Piece &p = sh.pieces[reader.k];
            const int blocks = p.n, past = p.past, row0 = p.row, rows = p.rows;
            const int mine = (blocks + 1 - g) / 2, theirs = blocks - mine;
            uint64_t sums[kRows8 / 2];  // this thread's slots', of rows 2 r and 2 r + 1
#pragma unroll
            for (int r = 0; r < kRows8 / 2; ++r) sums[r] = 0;
            int exponent = kNoScale;  // weights are times 2^-exponent
            if (gw == 0) shared.minus[g][lane] = kUnset;
            if (blocks > 0) {
                const uint32_t qb = qn & 1;
                hold8<kPieceLimitNs>(sh, &sh.q_full[qb], (qn >> 1) & 1, status);
                ++qn;
                const float q_factor = sh.q_factor[qb];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_empty[qb]);
                softmax_barrier<128>(1 + g);

                // scales: one of the group's blocks ahead, page ids two
                const int32_t *table = A.batch.pages + p.b * A.batch.pages_stride;
                const int lo = p.lo, end = p.end;
                const int j0 = A.by_group.div(row0), j1 = A.by_group.div(row0 + rows - 1);
                const int first_seen = A.window > 0 ? past + j0 - A.window + 1 : 0;
                const uint8_t *k_scales = P8.scales.k + p.h * P8.scales.k_st[2];
                const uint8_t *v_scales = P8.scales.v + p.h * P8.scales.v_st[2];
                auto slot_at = [&](int i) -> int { return (lo + 2 * i + g) * kKeys + gt; };
                auto page_of = [&](int i) -> int {
                    const int s = slot_at(i);
                    return i >= mine || s >= end || s < first_seen ? -1 : __ldg(table + A.by_page.div(s));
                };
                // (bytes as they come: nothing waits for them before the next block)
                uint32_t key_byte, value_byte, next_key, next_value;
                auto scales_of = [&](int i, int id) {
                    next_key = next_value = 127 + kMinScale;
                    if (id < 0 || id >= A.batch.num_pages) return;  // (no codes either)
                    const int s = slot_at(i);
                    const int64_t in = s - A.by_page.div(s) * A.batch.page_size;
                    next_key = __ldg(k_scales + id * P8.scales.k_st[0] + in * P8.scales.k_st[1]);
                    next_value = __ldg(v_scales + id * P8.scales.v_st[0] + in * P8.scales.v_st[1]);
                };
                scales_of(0, page_of(0));
                int next_page = page_of(1);
                for (int i = 0; i < mine; ++i, ++used) {
                    key_byte = next_key;
                    value_byte = next_value;
                    scales_of(i + 1, next_page);
                    next_page = page_of(i + 2);
                    hold8(sh, &sh.s_full[g], used & 1, status);
                    __syncwarp();
                    tc::fence_after();
                    uint64_t y[kRows8 / 2];  // of rows 2 r and 2 r + 1
                    const float key_scale = q_factor * scale_of(key_byte);
                    const int k0 = (lo + 2 * i + g) * kKeys;
                    const bool masked =
                        k0 + kKeys - 1 > past + j0 || (A.window > 0 && k0 <= past + j1 - A.window);
                    auto scores = [&]() {
                        const uint64_t key_scale2 = pair2(key_scale, key_scale);
#pragma unroll
                        for (int o0 = 0; o0 < kRows8 / 8; o0 += kAtOnce) {
                            uint32_t x[kParts][kAtOnce][8];
#pragma unroll
                            for (int o = 0; o < kAtOnce; ++o)
#pragma unroll
                                for (int part = 0; part < kParts; ++part)
                                    tc::ld8(x[part][o], t_s + part * kRows8 + (o0 + o) * 8);
                            tc::wait_ld();
#pragma unroll
                            for (int o = 0; o < kAtOnce; ++o)
#pragma unroll
                                for (int c = 0; c < 8; c += 2) {
                                    // the small parts first
                                    uint64_t sum = bits2(x[kParts - 1][o][c], x[kParts - 1][o][c + 1]);
#pragma unroll
                                    for (int part = kParts - 2; part >= 0; --part)
                                        sum = add2(sum, bits2(x[part][o][c], x[part][o][c + 1]));
                                    y[(o0 + o) * 4 + c / 2] = mul2(sum, key_scale2);
                                }
                        }
                        if (__builtin_expect(masked, 0)) {
                            // row r sees the slot when its token does: row0 + r >= t G, and
                            // < (t + window) G
                            const int64_t t = (int64_t)k0 + gt - past;
                            const int64_t from = t * A.group - row0;
                            const int64_t to = A.window > 0 ? from + (int64_t)A.window * A.group : kRows8;
                            const int r0 = (int)max((int64_t)0, min(from, (int64_t)kRows8));
                            const int r1 = (int)max((int64_t)0, min(to, (int64_t)kRows8));
#pragma unroll
                            for (int r = 0; r < kRows8 / 2; ++r) {
                                float a, b;
                                unpair2(y[r], a, b);
                                if (2 * r < r0 || 2 * r >= r1) a = -INFINITY;
                                if (2 * r + 1 < r0 || 2 * r + 1 >= r1) b = -INFINITY;
                                y[r] = pair2(a, b);
                            }
                        }
                    };
                    // scores relative to the references, and the largest of them
                    auto relative = [&]() -> float {
                        float top = -INFINITY;
#pragma unroll
                        for (int o = 0; o < kRows8 / 8; ++o) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float4 m = *reinterpret_cast<const float4 *>(&shared.minus[g][o * 8 + c * 4]);
                                const int r = o * 4 + c * 2;
                                y[r] = add2(y[r], pair2(m.x, m.y));
                                y[r + 1] = add2(y[r + 1], pair2(m.z, m.w));
                                float a, b;
                                unpair2(y[r], a, b);
                                top = max3(top, a, b);
                                unpair2(y[r + 1], a, b);
                                top = max3(top, a, b);
                            }
                        }
                        return top;
                    };
                    // (a byte of 255 is no scale: the vector is NaN)
                    const int e8 = value_byte == kScaleNan ? kNoScale : (int)value_byte - 127;
                    scores();
                    const float top = relative();
                    if (__builtin_expect(softmax_any<128>(1 + g, top > kRescaleAbove || e8 > exponent), 0)) {
                        // the rows' maxima over the block, and new references where they grew
                        scores();
                        {
                            float v[kMaxRows8];
#pragma unroll
                            for (int r = 0; r < kMaxRows8; ++r) v[r] = -INFINITY;
#pragma unroll
                            for (int r = 0; r < kRows8 / 2; ++r) unpair2(y[r], v[2 * r], v[2 * r + 1]);
                            shared.across[g][gw][lane] =
                                across_lanes(v, lane, [](float a, float b) { return fmaxf(a, b); });
                        }
                        const int largest = __reduce_max_sync(0xffffffffu, e8);
                        if (lane == 0) shared.exponent[g][gw] = largest;
                        softmax_barrier<128>(1 + g);
                        float high = shared.across[g][0][lane];
                        int most = shared.exponent[g][0];
#pragma unroll
                        for (int w = 1; w < 4; ++w) {
                            high = fmaxf(high, shared.across[g][w][lane]);
                            most = max(most, shared.exponent[g][w]);
                        }
                        // (one more, so that the next larger scale is no new reference)
                        const int now_e = most > exponent ? most + 1 : exponent;
                        const float old = shared.minus[g][lane];
                        const bool grow = high + old > kRescaleAbove;
                        const float now = grow ? -high : old;
                        const float f = !grow ? 1.f : old == kUnset ? 0.f : ex2(now - old);
                        const float fe = exponent == kNoScale ? 0.f : ex2((float)(exponent - now_e));
                        const bool scaled = __any_sync(0xffffffffu, grow && old != kUnset) || now_e != exponent;
                        exponent = now_e;
                        softmax_barrier<128>(1 + g);
                        if (gw == 0) {
                            shared.minus[g][lane] = now;
                            shared.factor[g][lane] = f;
                        }
                        softmax_barrier<128>(1 + g);
#pragma unroll
                        for (int o = 0; o < kRows8 / 4; ++o) {
                            const float4 m = *reinterpret_cast<const float4 *>(&shared.factor[g][o * 4]);
                            sums[2 * o] = mul2(sums[2 * o], pair2(m.x, m.y));
                            sums[2 * o + 1] = mul2(sums[2 * o + 1], pair2(m.z, m.w));
                        }
                        if (scaled && i > 0) {
                            hold8(sh, &sh.pv_done[g], (used - 1) & 1, status);
                            __syncwarp();
                            tc::fence_after();
#pragma unroll 1
                            for (int half = 0; half < L::kOutCols / 16; ++half) {
                                uint32_t o[16];
                                tc::ld16(o, t_o + g * L::kOutCols + half * 16);
                                tc::wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) *
                                                           (shared.factor[g][half * 16 + e] * fe));
                                tc::st16(t_o + g * L::kOutCols + half * 16, o);
                            }
                            tc::wait_st();
                        }
                        relative();
                    }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.s_empty[g]);
                    // a weight times its scale, in fp16's range (2^15 at most)
                    const int shift = e8 - exponent + (int)kHalfLift;
                    const float value_scale = shift < -126 ? 0.f : power_of_two(shift);
                    const uint64_t value_scale2 = pair2(value_scale, value_scale);
                    const bool any_nan = __any_sync(0xffffffffu, value_byte == kScaleNan);
                    if (used > 0) hold8(sh, &sh.pv_done[g], (used - 1) & 1, status);
                    __syncwarp();
                    char *row = smem + L::kP + g * kRaw + gt * 128;
#pragma unroll
                    for (int o = 0; o < kRows8 / 8; ++o) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = o * 4 + e;
                            float a, b;
                            unpair2(y[r], a, b);
                            const uint64_t x = pair2(ex2(a), ex2(b));
                            sums[r] = add2(sums[r], x);
                            unpair2(mul2(x, value_scale2), a, b);
                            if (__builtin_expect(any_nan, 0) && value_byte == kScaleNan) {  // for the rows that see it
                                float u, v;
                                unpair2(y[r], u, v);
                                a = u == -INFINITY ? 0.f : __uint_as_float(0x7fffffffu);
                                b = v == -INFINITY ? 0.f : __uint_as_float(0x7fffffffu);
                            }
                            w[e] = pack2<__half>(a, b);
                        }
                        *reinterpret_cast<uint4 *>(row + ((o ^ (gt & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_full[g]);
                }
                others += theirs;
                if (mine > 0) hold8(sh, &sh.pv_done[g], (used - 1) & 1, status);
                if (theirs > 0) hold8(sh, &sh.pv_done[1 - g], (others - 1) & 1, status);
                __syncwarp();
                tc::fence_after();
            }

            // ---- the groups' states, joined: lane r has row r's --------------------------
            {
                float v[kMaxRows8];
#pragma unroll
                for (int r = 0; r < kMaxRows8; ++r) v[r] = 0.f;
#pragma unroll
                for (int r = 0; r < kRows8 / 2; ++r) unpair2(sums[r], v[2 * r], v[2 * r + 1]);
                shared.across[g][gw][lane] = across_lanes(v, lane, [](float a, float b) { return a + b; });
                if (lane == 0) shared.exponent[g][gw] = exponent;
            }
            softmax_barrier<256>(3);
            float ref = -INFINITY, sum = 0.f, f[2];
            {
                float own_ref[2], own_sum[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float m = shared.minus[x][lane];
                    own_ref[x] = m == kUnset ? -INFINITY : -m;
                    own_sum[x] = (shared.across[x][0][lane] + shared.across[x][1][lane]) +
                                 (shared.across[x][2][lane] + shared.across[x][3][lane]);
                    ref = fmaxf(ref, own_ref[x]);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    f[x] = own_ref[x] == -INFINITY ? 0.f : ex2(own_ref[x] - ref);
                    sum += own_sum[x] * f[x];
                    const int e = shared.exponent[x][0];
                    f[x] *= e == kNoScale ? 0.f : ex2((float)(e - (int)kHalfLift));
                }
            }
            // thread d of group g has value d of rows 16 g .. 16 g + 15
            const int r0 = g * 16, here = min(16, rows - r0);
            float o[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) o[r] = 0.f;
            if (here > 0) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (blocks <= x) break;
                    uint32_t u[16];
                    tc::ld16(u, t_o + x * L::kOutCols + r0);
                    tc::wait_ld();
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        o[r] = fmaf(__shfl_sync(0xffffffffu, f[x], r0 + r), __uint_as_float(u[r]), o[r]);
                }
                tc::fence_before();
            }
            // rows of out, one after another
            const int j_first = A.by_group.div(row0 + r0);
            int head = row0 + r0 - j_first * A.group;
            T *out = static_cast<T *>(A.out) + (int64_t)(p.token + j_first) * A.o_st[0] +
                     ((int64_t)p.h * A.group + head) * A.o_st[1] + gt;
            const int64_t wrap = A.o_st[0] - A.group * A.o_st[1];
            auto store = [&](float y) {
                *out = from_f32<T>(y);
                out += A.o_st[1];
                if (++head == A.group) {
                    head = 0;
                    out += wrap;
                }
            };
            if (p.parts == 1) {
                // (a row that saw nothing has the sum 0, and zeros)
                const float norm = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float n = __shfl_sync(0xffffffffu, norm, r0 + r);
                    if (r < here && gt < D) store(n == 0.f ? 0.f : o[r] * n);
                }
            } else {
                const int slot = blockIdx.x * 2 + ((int)blockIdx.x == p.first ? 1 : 0);
                float2 *part_stats = reinterpret_cast<float2 *>(A.workspace + kAttendStats);
                float *part_out = reinterpret_cast<float *>(A.workspace + kAttendOut);
                constexpr int64_t kSlot = (int64_t)(kMaxHeadDim / 4) * 2 * kRows * 4;  // floats of a slot
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (r < here) part_out[slot * kSlot + (r0 + r) * 128 + gt] = o[r];
                if (warp == 0) part_stats[(int64_t)slot * 2 * kRows + lane] = make_float2(ref, sum);
                softmax_barrier<256>(3);
                if (tid == 0) {
                    __threadfence();  // all 256 threads' writes, after the barrier
                    uint32_t *count = reinterpret_cast<uint32_t *>(A.workspace + kAttendCounters) + 2 * p.first;
                    const uint32_t before = atomicAdd(count, 1u);
                    const bool last = before == (uint32_t)p.parts - 1;
                    if (last) *count = 0;
                    // no call leaves such a count: the workspace was not initialised
                    if (before >= (uint32_t)p.parts) atomicOr(status, SV_STATUS_OVERFLOW);
                    sh.last = last;
                }
                softmax_barrier<256>(3);
                if (sh.last && here > 0) {
                    __threadfence();
                    auto slot_of = [&](int i) -> int { return (p.first + i) * 2 + (i == 0 ? 1 : 0); };
                    // lane r: row r's reference and sum over the parts (as many loads in
                    // flight as a batch; one past the end is the last once more)
                    constexpr int kBatch = 8;
                    float top = -INFINITY, all = 0.f;
#pragma unroll 1
                    for (int i0 = 0; i0 < p.parts; i0 += kBatch) {
                        float2 x[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i)
                            x[i] = __ldcg(&part_stats[(int64_t)slot_of(min(i0 + i, p.parts - 1)) * 2 * kRows + lane]);
                        float m = top;
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) m = fmaxf(m, x[i].x);
                        all *= top == -INFINITY ? 0.f : ex2(top - m);
#pragma unroll
                        for (int i = 0; i < kBatch; ++i)
                            if (i0 + i < p.parts && x[i].y != 0.f) all += x[i].y * ex2(x[i].x - m);
                        top = m;
                    }
                    const float norm = all == 0.f ? 0.f : 1.f / all;
                    float acc[16];
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[r] = 0.f;
#pragma unroll 1
                    for (int i0 = 0; i0 < p.parts; i0 += 2) {
                        float x[2][16], m[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int64_t at = slot_of(min(i0 + i, p.parts - 1));
                            m[i] = __ldcg(&part_stats[at * 2 * kRows + lane]).x;
#pragma unroll
                            for (int r = 0; r < 16; ++r)
                                if (r < here) x[i][r] = __ldcg(&part_out[at * kSlot + (r0 + r) * 128 + gt]);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // (a NaN query leaves no reference, and NaN in O)
                            const float w = i0 + i >= p.parts || m[i] == -INFINITY ? 0.f : ex2(m[i] - top);
#pragma unroll
                            for (int r = 0; r < 16; ++r) {
                                const float fr = __shfl_sync(0xffffffffu, w, r0 + r);
                                if (r < here) acc[r] = fmaf(fr, x[i][r], acc[r]);
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float n = __shfl_sync(0xffffffffu, norm, r0 + r);
                        if (r < here && gt < D) store(n == 0.f ? 0.f : acc[r] * n);
                    }
                }
            }
            reader.done(sh, lane);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 13) {
        __syncwarp();
        tc::tmem_free(tmem, L::kCols);
    }
}

}  // namespace sv
