// sv_attend8.cuh -- attention of few new rows over a paged cache of 8-bit values,
// on the fifth-generation tensor cores.
//
// Rows are packed as in sv_attend.cuh (the G query heads of a kv head side by side),
// but the products are the transposed ones: a key block's 128 slots are the 128
// lanes of tensor memory and the tile's up to 32 rows its columns,
//   S^T = K Q^T,   O^T += V^T P^T.
// So a thread has one slot and all rows: the exponentials of a block are spread
// over four warps however few rows there are, a slot's scales are two numbers of
// its thread, and the tensor cores are not fed empty rows.
//
// Keys go to the tensor cores as the e4m3 codes they are.  The queries become 8-bit
// floats beside them: relative to a power of two of its row, each value is the
// sum of 3 (bf16) or 4 (fp16) e5m2 numbers, the nearest to what the ones before it
// left (3 significant bits each, 2 and the sign of the rest): exact down to 2^-23
// (fp16: 2^-20) of the row's largest, and good to 2^-31 of it below.  The parts are columns of their own
// (their products are added in fp32 by the softmax threads), so a block of keys is
// read from shared memory once.
// Values need their slots' axis contiguous for the second product, which 16-bit types
// have: four warps turn codes into fp16 (exact).  Their scales go into the weights, as
// logarithms beside the scores: weight times scale, relative to the row's reference, in
// fp16 is the one rounding between fp32 scores and the result (11 bits; what is below
// 2^-18 of the row's largest is rounded to steps of 2^-28 of it).  The sums take the
// scales out again, in fp32.
//
// Softmax: the reference of a row follows the largest weight times scale among the slots
// that it sees, and only when one would not fit fp16; whether any is so large, is one vote
// of the 128 threads per block, and finding the new references the rare way (a new one
// puts the largest at 2^4, with 2^11.9 of room above).  A row's numbers depend on no
// other row and on no slot that it does not see.  Two groups of
// four warps take the even and the odd blocks of a tile, each with scores, weights,
// outputs and references of its own, and join them at the tile's end.
//
// Work split, partial states and their join: as in sv_attend.cuh.
//
// Warps 0-7 softmax, 8-11 values to fp16, 12 copies (TMA boxes of page pieces), 13
// issues S, 14 issues O, 15 fetches scales, 16-19 walk the CTA's run, publish its
// pieces, prepare their queries and, while the next tile is under way, join a tile's
// groups and parts and write its rows.  Every wait is bounded, as there.
//
// Measured (32 query heads over 8 of 128, bf16, unless said otherwise):
//   rounds of 6 tokens over up to 4096 slots, 256 sequences: 279 us, 4.4 TB/s (16-bit
//     caches: 375).  The bound is a block's way through four softmax warps (latency: some
//     4000 cycles for two blocks at a time, a tenth of it instructions of one warp), which
//     the instruction cache feeds;
//   6 tokens over 131071 slots, 2 sequences, 16 over 4 heads of 64 in fp16: 76 us, with
//     pages of 64 slots instead of 16 (4 boxes a block instead of 16) 62.  A block of heads
//     of 64 takes as long as one of 128 at half the bytes: 16-bit caches take 66 and 59,
//     and are the faster ones for few rows of such heads over long contexts;
//   one token over 1000 slots: 12 us: launch, lookups, one block, join of the parts.
#pragma once

#include "sv_append8.cuh"
#include "sv_attend.cuh"

namespace sv {

constexpr int kMaxRows8 = 32;   // packed rows of a tile at most
// A tile's fixed cost in key blocks: 289 us for a round of 6 tokens over up to 4096 slots
// alone (302 with 3, 291 with 8), 138 over up to 500 (147 and 134).
constexpr int kTileCost8 = 5;
constexpr int kThreads8 = 640;
// Registers per thread after the roles part, of the 640 x 96 that the block is
// launched with.
constexpr int kSoftmaxRegs8 = 136, kValueRegs8 = 56, kIssueRegs8 = 56, kTileRegs8 = 96;
static_assert(128 * (2 * kSoftmaxRegs8 + kValueRegs8 + kIssueRegs8 + kTileRegs8) <= kThreads8 * 96, "register split");
constexpr int kRaw = kKeys * 128;     // a block of codes
constexpr int kScaleRing = 3;         // pairs of blocks of scales
// Weights are relative to a row's reference, their values' scales included: the logarithm
// of the largest that fp16 holds, and where a new reference puts the largest so far.
// (A round of 6 tokens over up to 4096 slots alone: 289 us, 310 with no more than 2^8.9 of
// room above a new reference's largest, 283 with 2^14.9, at 3 bits less below.)
constexpr float kGrowAbove = 15.9f, kTop = 4.f;
// Where references have steps of 8 and more, a new one may put the largest so far beside
// kTop; this far off it is corrected.
constexpr float kFarOff = 10.f, kCoarse = 0x1p26f;
constexpr int kMaxPasses = 8;
constexpr float kUnset = 3e38f;       // minus the reference of a row that has seen nothing
constexpr float kShift = 8.f;         // of scales' logarithms: those of values about 1 become 0
constexpr int kSumLift = 20;          // sums are so much smaller (log2), lest values of zeros' overflow
// A score is its codes' product (up to 2^32) times the key's scale times the row's power
// of two; the scale is taken 2^8 times smaller, and the power larger, lest the first
// product overflow.
constexpr int kKeyLift = 8;

struct Attend8Params {
    AttendParams a;
    Scales scales;
    // |scale| * log2(e) as a number from 1/2 to 1 and a power of two; the first goes into
    // the keys' scales, the second into the rows' factors
    float scale_part;
    int32_t scale_exponent;
};

template <class T, int kRows8>
struct Attend8Smem {
    static constexpr int kParts = __is_same(T, __nv_bfloat16) ? 3 : 4;
    // columns of scores: a whole product has a multiple of 16
    static constexpr int kScoreCols = (kParts * kRows8 + 15) / 16 * 16;
    static constexpr int kQuery = kScoreCols * 128;
    // Rings: blocks of keys and of values in flight, as room allows
    static constexpr int kMisc = 8192, kRoom = 227 * 1024;
    static constexpr int kFixed = kMisc + 2 * kQuery + 2 * 2 * kRaw + kRaw;
    static constexpr int kRingV = kFixed + 6 * kRaw <= kRoom ? 3 : 2, kRingK = kFixed + (4 + kRingV) * kRaw <= kRoom ? 4 : 3;
    static constexpr int kQ = kMisc, kK = kQ + 2 * kQuery, kV = kK + kRingK * kRaw, kVc = kV + kRingV * kRaw,
                         kP = kVc + 2 * 2 * kRaw, kBytes = kP + kRaw;
    // O of two tiles' two groups: first column, and a whole product's columns
    static constexpr int kOutCols = (kRows8 + 15) / 16 * 16, kOut = 2 * kScoreCols;
    static constexpr uint32_t kCols = kOut + 4 * kOutCols <= 128 ? 128 : kOut + 4 * kOutCols <= 256 ? 256 : 512;
    static_assert(kBytes <= 227 * 1024 && kQ % 1024 == 0 && kQuery % 1024 == 0, "shared memory");
    static_assert(kOut + 4 * kOutCols <= 512, "tensor memory");
};

constexpr int kPieceReaders8 = 20;

struct Attend8Shared {
    unsigned long long k_full[4], k_empty[4], v_full[4], v_empty[4];
    unsigned long long scale_full[kScaleRing], scale_empty[kScaleRing];
    unsigned long long s_full[2], s_empty[2], vc_full[2], p_full[2], pv_done[2], q_full[2], q_empty[2], drain[2];
    unsigned long long state_full[2], state_empty[2], o_full[2], o_empty[2];
    unsigned long long piece_full[kPieces], piece_empty[kPieces];
    Piece pieces[kPieces];
    uint32_t tmem;
    int32_t dead, b0, last;
    int64_t skip;
    int64_t sums[kThreads8 / 32];
};

struct __align__(16) GroupState {   // of a softmax group
    float minus[kMaxRows8], base[kMaxRows8];  // minus the rows' references; 0 where there is none
    float factor[kMaxRows8];        // root of what a new reference makes of sums and outputs
    float across[4][kMaxRows8];     // its warps' maxima
};

struct __align__(16) TileState {    // what the softmax leaves of a tile
    float minus[2][kMaxRows8], sums[2][4][kMaxRows8];
    float shift[2];
};

struct __align__(16) Attend8Misc {
    Attend8Shared sh;
    GroupState group[2];
    TileState tile[2];
    float q_factor[2][kMaxRows8];  // powers of two of a tile's rows, with the call's scale's and kKeyLift
    uint8_t scales[kScaleRing][2][2 * kKeys];  // of keys and values
};
static_assert(sizeof(Attend8Misc) <= 8192, "misc region");

// A wait that gives up for the whole CTA, as hold() of the 16-bit kernel; the kernel's
// end reports it.  Every wait of every warp is a copy of this, and code that does not
// fit the instruction cache costs a third of the time: 32 bits of the timer do.  (Short
// waits give up after 0.25 s; long ones, which wait for whole pieces, count 2^32 ns: 24
// of them are 103 s.)
template <bool kLong = false>
__device__ __forceinline__ bool hold8(Attend8Shared &sh, unsigned long long *bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return true;
    auto now = []() -> uint32_t {
        uint32_t t;
        if (kLong) asm volatile("mov.u32 %0, %%globaltimer_hi;" : "=r"(t));
        else asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
        return t;
    };
    const uint32_t t0 = now();
    while (!mbar_try(bar, parity)) {
        if (now() - t0 > (kLong ? 24u : (uint32_t)kWaitLimitNs)) *(volatile int32_t *)&sh.dead = 1;
        if (*(volatile int32_t *)&sh.dead) return false;
    }
    return true;
}

// Where a warp is in a ring of stages.
template <int kStages>
struct RingPlace {
    int st = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next() {
        if (++st == kStages) {
            st = 0;
            turn ^= 1;
        }
    }
};

struct PieceReader8 {
    int k = 0;
    uint32_t turn = 0;
    // (all lanes) whether there is a piece; it is sh.pieces[k]
    __device__ __forceinline__ bool next(Attend8Shared &sh) {
        const bool ok = __all_sync(0xffffffffu, hold8(sh, &sh.piece_full[k], turn));
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

// Barriers of the 128 threads of a softmax group (number 1 or 2) or of the tile warps
// (3).  All of them come to each, whatever timed out.
__device__ __forceinline__ void group_barrier(int number) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(number) : "memory");
}
__device__ __forceinline__ bool group_any(int number, bool x) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred p, q; setp.ne.u32 q, %2, 0;\n"
        "barrier.cta.red.or.pred p, %1, 128, q; selp.u32 %0, 1, 0, p; }"
        : "=r"(r)
        : "r"(number), "r"((uint32_t)x)
        : "memory");
    return r != 0;
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

// How far reference a lies above b, each given as minus it and its group's shift.  (kUnset
// lies below every other, and as far from itself as 0.)
__device__ __forceinline__ float above(float a_minus, float a_shift, float b_minus, float b_shift) {
    return (b_minus - a_minus) + (b_shift - a_shift);
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
    // parts of scores loaded at once, as registers allow
    constexpr int kAtOnce = kParts * kRows8 <= 72 ? kParts : kRows8 <= 24 ? 2 : 1;
    constexpr uint32_t kIdescS = tc::instr_desc_f8(kKeys, L::kScoreCols);
    // (bit 15: A's slots are its rows in memory, as B's)
    constexpr uint32_t kIdescO = tc::instr_desc(false, true, 128, L::kOutCols) | (1u << 15);
    extern __shared__ __align__(1024) char smem[];
    Attend8Misc &misc = *reinterpret_cast<Attend8Misc *>(smem);
    Attend8Shared &sh = misc.sh;
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
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_empty[i], 4);
        }
        for (int i = 0; i < kScaleRing; ++i) {
            mbar_init(&sh.scale_full[i], 1);
            mbar_init(&sh.scale_empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], 4);
            mbar_init(&sh.vc_full[i], 4);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.q_full[i], 4);
            mbar_init(&sh.q_empty[i], 9);
            mbar_init(&sh.state_full[i], 8);
            mbar_init(&sh.state_empty[i], 4);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.o_empty[i], 4);
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
            const int64_t own = A.batch.B <= kThreads8 ? last_cost : sequence_cost<kRows8, kTileCost8>(A, b, lane);
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

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTileRegs8));
        // ---- tiles: their pieces and queries ahead, their rows behind the softmax ------
        const int tw = warp - 16, tt = tid - 512;
        const uint32_t t_o = tmem + ((uint32_t)(tw * 32) << 16) + L::kOut;
        Walker<kRows8, kTileCost8> walk;
        walk.left = 0;
        if (tw == 0 && !idle) walk.start(A, sh.b0, sh.skip, u0, u1 - u0, total, ctas, lane);
        uint32_t ready = 0, done = 0, qn = 0;  // pieces published and finished, tiles with queries
        bool more = true;                      // pieces may follow
        // Publishes the next piece and prepares its queries (all four warps; false after
        // a wait gave up).
        auto prepare = [&]() -> bool {
            if (SV_STALL && ready == 1 && blockIdx.x % 2 == 1) return false;
            const int k = ready % kPieces;
            bool ok = true;
            if (tw == 0) {
                Piece p;
                if (!walk.next(A, p)) p.n = -1;
                ok = __all_sync(0xffffffffu, hold8<true>(sh, &sh.piece_empty[k], (ready / kPieces & 1) ^ 1));
                if (ok && lane == 0) {
                    sh.pieces[k] = p;
                    mbar_arrive(&sh.piece_full[k]);
                }
                __syncwarp();
            }
            ok = ok && __all_sync(0xffffffffu, hold8<true>(sh, &sh.piece_full[k], ready / kPieces & 1));
            if (group_any(3, !ok)) return false;
            const Piece &p = sh.pieces[k];
            if (p.n < 0) {
                more = false;
                return true;
            }
            ++ready;
            if (p.n == 0) return true;
            const int qb = qn & 1;
            ok = __all_sync(0xffffffffu, hold8<true>(sh, &sh.q_empty[qb], (qn >> 1 & 1) ^ 1));
            ++qn;
            // four values to a lane, rows tw, tw + 4, ... to a warp
            constexpr int kMine = kRows8 / 4;
            const int rows = p.rows;
            auto load = [&](int i) -> uint2 {
                const int r = tw + 4 * i;
                if (r >= rows || lane * 4 >= D || A.q_mode == 2) return make_uint2(0, 0);
                const int pr = p.row + r, j = A.by_group.div(pr);
                return __ldg(reinterpret_cast<const uint2 *>(
                    static_cast<const uint16_t *>(A.q) + (int64_t)(p.token + j) * A.q_st[0] +
                    (p.h * A.group + (pr - j * A.group)) * A.q_st[1] + lane * 4));
            };
            auto bits = [&](const float2 &f) -> uint32_t {  // of the larger finite magnitude
                const uint32_t a = __float_as_uint(f.x) & 0x7fffffffu, b = __float_as_uint(f.y) & 0x7fffffffu;
                return max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u);
            };
            // (all rows' loads in flight; the second time they come from near by)
            uint32_t tops = 0;  // lane i: bits of the i-th row's largest magnitude
            {
                uint2 x[kMine];
#pragma unroll
                for (int i = 0; i < kMine; ++i) x[i] = load(i);
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const uint32_t top =
                        __reduce_max_sync(0xffffffffu, max(bits(pair_of(x[i].x, T())), bits(pair_of(x[i].y, T()))));
                    if (lane == i) tops = top;
                }
            }
            char *to = smem + L::kQ + qb * L::kQuery;
#pragma unroll 1
            for (int i = 0; i < kMine; ++i) {
                const int r = tw + 4 * i;
                const uint2 x = load(i);
                // the row's largest is brought to 57344 (e5m2's) or less
                const uint32_t top = __shfl_sync(0xffffffffu, tops, i);
                const int e =
                    min(max((int)(top >> 23) - 127 - 15 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), -126), 120);
                const float f = A.q_mode == 1 ? -power_of_two(-e) : power_of_two(-e);
                if (lane == 0) misc.q_factor[qb][r] = power_of_two(min(max(e + kKeyLift + P8.scale_exponent, -126), 127));
                const float2 a = pair_of(x.x, T()), b = pair_of(x.y, T());
                float y[4] = {a.x * f, a.y * f, b.x * f, b.y * f};
                // an infinity makes its row NaN, as a NaN does
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (!(fabsf(y[m]) <= 57344.f)) y[m] = __uint_as_float(0x7fffffffu);
#pragma unroll 1
                for (int part = 0; part < kParts; ++part)
                    *reinterpret_cast<uint32_t *>(to + (part * kRows8 + r) * 128 + ((lane / 4) ^ (r & 7)) * 16 +
                                                  lane % 4 * 4) = split_off(y);
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full[qb]);
            return !group_any(3, !ok);
        };
        bool ok = true;
        for (;;) {
            while (ok && more && ready < done + 2) ok = prepare();  // two tiles ahead
            if (!ok || done == ready) break;
            const Piece &p = sh.pieces[done % kPieces];
            const uint32_t tb = done & 1, turn = done >> 1 & 1;
            const int blocks = p.n, row0 = p.row, rows = p.rows;
            ok = __all_sync(0xffffffffu, hold8<true>(sh, &sh.state_full[tb], turn));
            ok = ok && __all_sync(0xffffffffu, hold8<true>(sh, &sh.o_full[tb], turn));
            ok = !group_any(3, !ok);
            if (!ok) break;
            tc::fence_after();
            // the groups' states, joined: lane r has row r's
            const TileState &st = misc.tile[tb];
            // (references may be 2^200 apart beside sums that are as far: factors in two steps)
            float minus = kUnset, shift = 0.f, sum = 0.f, f[2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (above(st.minus[x][lane], st.shift[x], minus, shift) > 0.f)
                    minus = st.minus[x][lane], shift = st.shift[x];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float h = ex2(0.5f * above(st.minus[x][lane], st.shift[x], minus, shift));
                sum += ((st.sums[x][0][lane] + st.sums[x][1][lane]) + (st.sums[x][2][lane] + st.sums[x][3][lane])) * h * h;
                f[x] = h * h * (1.f / (1 << kSumLift));
            }
            // (a row that saw nothing has the sum 0, and zeros)
            const bool whole = p.parts == 1;
            if (whole) {
                const float norm = sum == 0.f ? 0.f : 1.f / sum;
                f[0] *= norm;
                f[1] *= norm;
            }
            const int slot = blockIdx.x * 2 + ((int)blockIdx.x == p.first ? 1 : 0);
            float2 *part_stats = reinterpret_cast<float2 *>(A.workspace + kAttendStats);
            float *part_out = reinterpret_cast<float *>(A.workspace + kAttendOut);
            constexpr int64_t kSlot = (int64_t)(kMaxHeadDim / 4) * 2 * kRows * 4;  // floats of a slot
            // rows of out, one after another; thread d has value d
            const int j_first = A.by_group.div(row0);
            int head = row0 - j_first * A.group;
            T *out = static_cast<T *>(A.out) + (int64_t)(p.token + j_first) * A.o_st[0] +
                     ((int64_t)p.h * A.group + head) * A.o_st[1] + tt;
            const int64_t wrap = A.o_st[0] - A.group * A.o_st[1];
            // (a row at a time: what this loop is long, the softmax's leaves the cache)
#pragma unroll 1
            for (int r = 0; r < rows; ++r) {
                uint32_t u0 = 0, u1 = 0;  // (a group that had no block left none)
                if (blocks > 0) u0 = tc::ld1(t_o + tb * 2 * L::kOutCols + r);
                if (blocks > 1) u1 = tc::ld1(t_o + (tb * 2 + 1) * L::kOutCols + r);
                tc::wait_ld();
                const float f0 = __shfl_sync(0xffffffffu, f[0], r), f1 = __shfl_sync(0xffffffffu, f[1], r);
                const float o = fmaf(f1, __uint_as_float(u1), f0 * __uint_as_float(u0));
                if (whole) {
                    if (tt < D) *out = from_f32<T>(o);
                } else {
                    part_out[slot * kSlot + r * 128 + tt] = o;
                }
                out += A.o_st[1];
                if (++head == A.group) {
                    head = 0;
                    out += wrap;
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.o_empty[tb]);
                mbar_arrive(&sh.state_empty[tb]);
            }
            if (!whole) {
                if (tw == 0) {
                    part_stats[(int64_t)slot * 2 * kRows + lane] = make_float2(minus, sum);
                    part_stats[(int64_t)slot * 2 * kRows + kMaxRows8 + lane] = make_float2(shift, 0.f);
                }
                group_barrier(3);
                if (tt == 0) {
                    __threadfence();  // all 128 threads' writes, after the barrier
                    uint32_t *count = reinterpret_cast<uint32_t *>(A.workspace + kAttendCounters) + 2 * p.first;
                    const uint32_t before = atomicAdd(count, 1u);
                    const bool last = before == (uint32_t)p.parts - 1;
                    if (last) *count = 0;
                    // no call leaves such a count: the workspace was not initialised
                    if (before >= (uint32_t)p.parts) atomicOr(status, SV_STATUS_OVERFLOW);
                    sh.last = last;
                }
                group_barrier(3);
                if (sh.last) {
                    __threadfence();
                    const int parts = p.parts, first = p.first;
                    auto slot_of = [&](int i) -> int64_t { return (first + i) * 2 + (i == 0 ? 1 : 0); };
                    // lane r: row r's reference and sum over the parts (as many loads in
                    // flight as a batch; one past the end is the last once more)
                    constexpr int kBatch = 8;
                    float all = 0.f;
                    minus = kUnset, shift = 0.f;
#pragma unroll 1
                    for (int i0 = 0; i0 < parts; i0 += kBatch) {
                        float2 x[kBatch];
                        float n[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const float2 *at = &part_stats[slot_of(min(i0 + i, parts - 1)) * 2 * kRows + lane];
                            x[i] = __ldcg(at);
                            n[i] = __ldcg(at + kMaxRows8).x;
                        }
                        const float old_minus = minus, old_shift = shift;
#pragma unroll
                        for (int i = 0; i < kBatch; ++i)
                            if (above(x[i].x, n[i], minus, shift) > 0.f) minus = x[i].x, shift = n[i];
                        const float h = ex2(0.5f * above(old_minus, old_shift, minus, shift));
                        all *= h * h;
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const float g = ex2(0.5f * above(x[i].x, n[i], minus, shift));
                            if (i0 + i < parts) all += x[i].y * g * g;
                        }
                    }
                    const float over = 1.f / all;
                    // four values to a lane, one row to a warp, or two of up to 64 values
                    const int per = wide ? 1 : 2, d0 = (wide ? lane : lane % 16) * 4;
                    const int64_t base = (int64_t)p.token * A.o_st[0] + (int64_t)p.h * A.group * A.o_st[1];
#pragma unroll 1
                    for (int r0 = tw * per; r0 < rows; r0 += 4 * per) {
                        const int r = min(r0 + (wide ? 0 : lane / 16), rows - 1);
                        const float row_minus = __shfl_sync(0xffffffffu, minus, r);
                        const float row_shift = __shfl_sync(0xffffffffu, shift, r);
                        const float row_all = __shfl_sync(0xffffffffu, all, r);
                        const float row_over = __shfl_sync(0xffffffffu, over, r);
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                        for (int i0 = 0; i0 < parts; i0 += kBatch) {
                            float4 x[kBatch];
                            float m[kBatch];
#pragma unroll
                            for (int i = 0; i < kBatch; ++i) {
                                const int64_t at = slot_of(min(i0 + i, parts - 1));
                                m[i] = above(__ldcg(&part_stats[at * 2 * kRows + r]).x,
                                             __ldcg(&part_stats[at * 2 * kRows + kMaxRows8 + r]).x, row_minus, row_shift);
                                x[i] = __ldcg(reinterpret_cast<const float4 *>(part_out + at * kSlot + r * 128 + d0));
                            }
#pragma unroll
                            for (int i = 0; i < kBatch; ++i) {
                                const float w = ex2(m[i]);
                                if (i0 + i < parts) {
                                    acc.x = fmaf(w, x[i].x, acc.x);
                                    acc.y = fmaf(w, x[i].y, acc.y);
                                    acc.z = fmaf(w, x[i].z, acc.z);
                                    acc.w = fmaf(w, x[i].w, acc.w);
                                }
                            }
                        }
                        if (d0 < D && (wide || r0 + lane / 16 < rows)) {
                            const int pr = row0 + r, j = A.by_group.div(pr);
                            uint2 y;
                            y.x = pack2<T>(acc.x * row_over, acc.y * row_over);
                            y.y = pack2<T>(acc.z * row_over, acc.w * row_over);
                            if (row_all == 0.f) y = make_uint2(0, 0);
                            *reinterpret_cast<uint2 *>(static_cast<T *>(A.out) + base + j * A.o_st[0] +
                                                       (pr - j * A.group) * A.o_st[1] + d0) = y;
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.piece_empty[done % kPieces]);
            ++done;
        }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs8));
        if (warp == 12) {
            // ---- copies of codes ------------------------------------------------
            const int boxes = kKeys / A.piece;
            const bool active = lane < boxes;
            RingPlace<L::kRingK> kp;
            RingPlace<L::kRingV> vp;
            int kn = 0, vn = 0;  // blocks copied so far, as far as a ring goes
            PieceReader8 reader;
            bool ok = true;
            while (ok && reader.next(sh)) {
                const Piece &q = sh.pieces[reader.k];
                const int blocks = q.n, lo = q.lo, end = q.end, h = q.h;
                const int32_t *table = A.batch.pages + q.b * A.batch.pages_stride;
                const int first = A.window > 0 ? q.past + A.by_group.div(q.row) - A.window + 1 : 0;
                reader.done(sh, lane);
                if (blocks == 0) continue;
                // page ids of 32 boxes at a time, the next ones on their way
                auto pages_of = [&](int box) -> int {
                    if (box + lane >= blocks * boxes) return kNoPage;  // (slots past 2^31 among them)
                    const int s0 = lo * kKeys + (box + lane) * A.piece;
                    return s0 >= end || s0 + A.piece <= first ? kNoPage : __ldg(table + A.by_page.div(s0));
                };
                auto checked = [&](int id) -> int {
                    if (id != kNoPage && (id < 0 || id >= A.batch.num_pages)) {
                        atomicOr(status, SV_STATUS_BAD_PAGE);
                        id = kNoPage;
                    }
                    return id;
                };
                // keys run a block ahead of values
                int ids = 0, next_ids = pages_of(0), key_id = kNoPage, value_id;
#pragma unroll 1
                for (int i = -1; i < blocks && ok; ++i) {
                    const int box = (i + 1) * boxes;
                    if (box % 32 == 0) {
                        ids = next_ids;
                        next_ids = pages_of(box + 32);
                    }
                    value_id = key_id;
                    key_id = checked(__shfl_sync(0xffffffffu, ids, box % 32 + lane % boxes));
#pragma unroll 1
                    for (int of = 0; of < 2; ++of) {  // keys of block i + 1, values of block i
                        const int x = of ? i : i + 1;
                        if (x < 0 || x >= blocks) continue;
                        const int st = of ? vp.st : kp.st;
                        unsigned long long *full = of ? &sh.v_full[st] : &sh.k_full[st];
                        unsigned long long *empty = of ? &sh.v_empty[st] : &sh.k_empty[st];
                        ok = ok && __all_sync(0xffffffffu, hold8(sh, empty, (of ? vp.turn : kp.turn) ^ 1));
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(full, kRaw);
                        __syncwarp();
                        if (active) {
                            const int s0 = (lo + x) * kKeys + lane * A.piece;
                            tc::load_box(smem + (of ? L::kV : L::kK) + st * kRaw + lane * A.piece * 128,
                                         of ? &vmap : &kmap, 0, h, s0 - A.by_page.div(s0) * A.batch.page_size,
                                         of ? value_id : key_id, full);
                        }
                        if (of) vp.next(), vn = min(vn + 1, L::kRingV);
                        else kp.next(), kn = min(kn + 1, L::kRingK);
                    }
                }
            }
            // the last copies have landed before the CTA may end
            for (int n = 0; n < kn; ++n) {  // (stages from kp.st on are the turn before)
                const int st = (kp.st + L::kRingK - 1 - n) % L::kRingK;
                mbar_wait(&sh.k_full[st], st < kp.st ? kp.turn : kp.turn ^ 1);
            }
            for (int n = 0; n < vn; ++n) {
                const int st = (vp.st + L::kRingV - 1 - n) % L::kRingV;
                mbar_wait(&sh.v_full[st], st < vp.st ? vp.turn : vp.turn ^ 1);
            }
        } else if (warp == 13) {
            // ---- scores ---------------------------------------------------------
            const uint32_t tm = (uint32_t)tc::uniform((int)tmem);
            const uint64_t k_desc = tc::smem_desc(smem_u32(smem + L::kK), 16, 1024);
            const uint64_t q_desc = tc::smem_desc(smem_u32(smem + L::kQ), 16, 1024);
            const int steps = (D + 31) / 32;
            uint32_t qn = 0, used[2] = {0, 0};  // tiles, blocks of each group
            RingPlace<L::kRingK> at;
            PieceReader8 reader;
            bool ok = true;  // a wait gave up: nothing more is issued or handed back
            while (ok && reader.next(sh)) {
                const int blocks = tc::uniform(sh.pieces[reader.k].n);
                reader.done(sh, lane);
                if (blocks == 0) continue;
                const uint32_t qb = qn & 1;
                ok = ok && __all_sync(0xffffffffu, hold8<true>(sh, &sh.q_full[qb], (qn >> 1) & 1));
                ++qn;
                for (int i = 0; i < blocks && ok; ++i, at.next()) {
                    const uint32_t st = at.st, sb = i & 1;
                    const uint32_t turn = sb ? used[1]++ : used[0]++;
                    ok = __all_sync(0xffffffffu, hold8(sh, &sh.k_full[st], at.turn));
                    ok = ok && __all_sync(0xffffffffu, hold8(sh, &sh.s_empty[sb], (turn & 1) ^ 1));
                    if (!ok) break;
                    tc::fence_after();
                    if (tc::elect()) {
                        const uint64_t kd = k_desc + st * (kRaw / 16), qd = q_desc + qb * (L::kQuery / 16);
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            if (s < steps)
                                tc::mma_f8(tm + sb * L::kScoreCols, kd + s * 2, qd + s * 2, kIdescS, s > 0);
                        tc::commit(&sh.k_empty[st]);
                        // (both groups' at once: their warps then run the same code together,
                        // and share its fetching: 289 instead of 295 us for a round alone)
                        if (sb == 1) tc::commit(&sh.s_full[0]);
                        if (sb == 1 || i + 1 == blocks) tc::commit(&sh.s_full[sb]);
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
            uint32_t used[2] = {0, 0}, tile = 0;
            PieceReader8 reader;
            bool ok = true;
            while (ok && reader.next(sh)) {
                const int blocks = tc::uniform(sh.pieces[reader.k].n);
                reader.done(sh, lane);
                const uint32_t tb = tile & 1;
                ok = __all_sync(0xffffffffu, hold8<true>(sh, &sh.o_empty[tb], (tile >> 1 & 1) ^ 1));
                ++tile;
                for (int i = 0; i < blocks && ok; ++i) {
                    const uint32_t b = i & 1, turn = (b ? used[1]++ : used[0]++) & 1;
                    ok = __all_sync(0xffffffffu, hold8(sh, &sh.vc_full[b], turn));
                    ok = ok && __all_sync(0xffffffffu, hold8(sh, &sh.p_full[b], turn));
                    if (!ok) break;
                    tc::fence_after();
                    if (tc::elect()) {
                        const uint64_t vd = v_desc + b * (2 * kRaw / 16), pd = p_desc + b * 4;  // (64 bytes)
#pragma unroll
                        for (int s = 0; s < kKeys / 16; ++s)
                            tc::mma_ss(tm + (tb * 2 + b) * L::kOutCols, vd + s * (2048 / 16), pd + s * (2048 / 16),
                                       kIdescO, i > 1 || s > 0);
                        tc::commit(&sh.pv_done[b]);
                    }
                    __syncwarp();
                }
                if (tc::elect() && ok) tc::commit(&sh.o_full[tb]);
                __syncwarp();
            }
            if (tc::elect()) tc::commit(&sh.drain[1]);
            __syncwarp();
            mbar_wait(&sh.drain[1], 0);
        } else {
            // ---- scales of two blocks at a time, eight slots to a lane ---------------
            const Scales &S = P8.scales;
            RingPlace<kScaleRing> at;
            PieceReader8 reader;
            bool ok = true;
            while (ok && reader.next(sh)) {
                const Piece &q = sh.pieces[reader.k];
                const int pairs = (q.n + 1) / 2, begin = q.lo * kKeys + lane * 8, end = min(q.end, (q.lo + q.n) * kKeys);
                const int32_t *table = A.batch.pages + q.b * A.batch.pages_stride;
                const int first = A.window > 0 ? q.past + A.by_group.div(q.row) - A.window + 1 : 0;
                const uint8_t *ks = S.k + q.h * S.k_st[2], *vs = S.v + q.h * S.v_st[2];
                reader.done(sh, lane);
                auto page_of = [&](int i) -> int {
                    if (i >= pairs) return -1;
                    const int s0 = begin + i * 2 * kKeys;
                    return s0 >= end || s0 + 8 <= first ? -1 : __ldg(table + A.by_page.div(s0));
                };
                // bytes are loaded a pair ahead of their use (and put together then), page
                // ids two
                uint32_t key[8], value[8];
                int id = page_of(0);
#pragma unroll 1
                for (int i = -1; i < pairs; ++i) {
                    if (i >= 0) {
                        ok = __all_sync(0xffffffffu, hold8(sh, &sh.scale_empty[at.st], at.turn ^ 1));
                        if (!ok) break;
                        auto four = [](const uint32_t *x) { return x[0] | x[1] << 8 | x[2] << 16 | x[3] << 24; };
                        *reinterpret_cast<uint2 *>(&misc.scales[at.st][0][lane * 8]) = make_uint2(four(key), four(key + 4));
                        *reinterpret_cast<uint2 *>(&misc.scales[at.st][1][lane * 8]) =
                            make_uint2(four(value), four(value + 4));
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.scale_full[at.st]);
                        at.next();
                    }
                    const int s0 = begin + (i + 1) * 2 * kKeys;
                    const int64_t in = s0 - A.by_page.div(s0) * A.batch.page_size;
                    const bool known = id >= 0 && id < A.batch.num_pages;
                    const uint8_t *k = ks + id * S.k_st[0] + in * S.k_st[1], *v = vs + id * S.v_st[0] + in * S.v_st[1];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        key[e] = value[e] = 127 + kMinScale;  // no page, no codes
                        if (known) {
                            key[e] = __ldg(k + e * S.k_st[1]);
                            value[e] = __ldg(v + e * S.v_st[1]);
                        }
                    }
                    id = page_of(i + 2);
                }
            }
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kValueRegs8));
        // ---- values to fp16 ---------------------------------------------------
        const int t = tid - 256;
        // a thread's chunk of 16 values and its slot of a group (eight lanes' chunks
        // lie in different banks)
        const int ch = wide ? t % 8 : t % 4, u = t / 4;
        const int slot0 = wide ? t / 8 : (u >> 3) * 8 + ((u & 1) << 2) + ((u >> 1) & 3);
        const int rounds = wide ? 8 : 4, per = wide ? 16 : 32;
        // (lanes of the upper half, or of odd slots, write their second eight values first)
        const bool odd_first = wide ? ch >= 4 : u & 1;
        // (per is a multiple of 8: all of a thread's slots share their place in a swizzle)
        const int x = slot0 & 7, j = (ch % 4) * 2;
        const int src = slot0 * 128 + ((ch ^ x) * 16), dst = (ch / 4) * kRaw + slot0 * 128;
        const int first = dst + (((j + (odd_first ? 1 : 0)) ^ x) * 16);
        const int second = dst + (((j + (odd_first ? 0 : 1)) ^ x) * 16);
        uint32_t used[2] = {0, 0};
        RingPlace<L::kRingV> at;
        PieceReader8 reader;
        bool ok = true;
        while (ok && reader.next(sh)) {
            const int blocks = sh.pieces[reader.k].n;
            const int end = sh.pieces[reader.k].end - sh.pieces[reader.k].lo * kKeys;
            reader.done(sh, lane);
            for (int i = 0; i < blocks && ok; ++i, at.next()) {
                const uint32_t b = i & 1, turn = b ? used[1]++ : used[0]++;
                ok = __all_sync(0xffffffffu, hold8(sh, &sh.v_full[at.st], at.turn));
                if (ok && turn > 0) ok = __all_sync(0xffffffffu, hold8(sh, &sh.pv_done[b], (turn - 1) & 1));
                if (!ok) break;
                char *raw = smem + L::kV + at.st * kRaw, *to = smem + L::kVc + b * 2 * kRaw;
                const int here = end - i * kKeys;
                if (here < kKeys) {
                    // slots from the tile's end on: whatever lies there, zeros
#pragma unroll 1
                    for (int k = 0; k < rounds; ++k)
                        if (k * per + slot0 >= here)
                            *reinterpret_cast<uint4 *>(raw + src + k * per * 128) = make_uint4(0, 0, 0, 0);
                }
                // (not unrolled, for the instruction cache's sake: 289 us for a round of 6 tokens
                // over up to 4096 slots alone, 296 by four, 377 by eight)
#pragma unroll 1
                for (int k = 0; k < rounds; ++k) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(raw + src + k * per * 128);
                    uint4 y, z;
                    codes_to_half(odd_first ? w.z : w.x, y.x, y.y);
                    codes_to_half(odd_first ? w.w : w.y, y.z, y.w);
                    codes_to_half(odd_first ? w.x : w.z, z.x, z.y);
                    codes_to_half(odd_first ? w.y : w.w, z.z, z.w);
                    *reinterpret_cast<uint4 *>(to + first + k * per * 128) = y;
                    *reinterpret_cast<uint4 *>(to + second + k * per * 128) = z;
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.vc_full[b]);
                    mbar_arrive(&sh.v_empty[at.st]);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs8));
        // ---- softmax: a slot to a thread ------------------------------------------
        const int g = warp / 4, gw = warp % 4, gt = gw * 32 + lane;
        const uint32_t lanes_at = tmem + ((uint32_t)(gw * 32) << 16);
        const uint32_t t_s = lanes_at + g * L::kScoreCols;
        GroupState &own = misc.group[g];
        uint32_t used = 0, qn = 0, tile = 0;  // the group's blocks, tiles with queries, tiles
        RingPlace<kScaleRing> sc;
        PieceReader8 reader;
        for (;;) {
            // (nothing that the last tile left is read any more)
            if (gw == 0) {
                own.minus[lane] = kUnset;
                own.base[lane] = 0.f;
            }
            // (all four warps go on, or none: they meet at barriers)
            if (group_any(1 + g, !reader.next(sh))) break;
            const Piece &p = sh.pieces[reader.k];
            const int blocks = p.n, past = p.past, row0 = p.row, rows = p.rows, lo = p.lo;
            const int mine = (blocks + 1 - g) / 2;
            const int j0 = A.by_group.div(row0), j1 = A.by_group.div(row0 + rows - 1);
            reader.done(sh, lane);
            uint64_t sums[kRows8 / 2];  // this thread's slots', of rows 2 r and 2 r + 1
#pragma unroll
            for (int r = 0; r < kRows8 / 2; ++r) sums[r] = 0;
            float minus = kUnset;       // lane r: minus row r's reference
            float shift = kShift;
            const uint32_t tb = tile & 1;
            if (blocks > 0) {
                const uint32_t qb = qn & 1;
                hold8<true>(sh, &sh.q_full[qb], (qn >> 1) & 1);
                ++qn;
                const float *q_factor = misc.q_factor[qb];
                const uint32_t t_o = lanes_at + L::kOut + (tb * 2 + g) * L::kOutCols;
                for (int i = 0; i < mine; ++i, ++used) {
                    const int k0 = (lo + 2 * i + g) * kKeys;
                    hold8(sh, &sh.scale_full[sc.st], sc.turn);
                    const uint32_t key_byte = misc.scales[sc.st][0][g * kKeys + gt],
                                   value_byte = misc.scales[sc.st][1][g * kKeys + gt];
                    hold8(sh, &sh.s_full[g], used & 1);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.scale_empty[sc.st]);
                    sc.next();
                    tc::fence_after();
                    uint64_t y[kRows8 / 2];  // scores over their rows' factors, of rows 2 r and 2 r + 1
                    const float key_scale = scale_of(key_byte) * (P8.scale_part / (1 << kKeyLift));
                    const bool masked =
                        k0 + kKeys - 1 > past + j0 || (A.window > 0 && k0 <= past + j1 - A.window);
                    // rows [r0, r1) see the slot: row r does when its token does, row0 + r >=
                    // t G, and < (t + window) G (none past the tile's last, which would see
                    // what lies behind its end)
                    int r0 = 0, r1 = kRows8;
                    if (__builtin_expect(masked, 0)) {
                        const int64_t from = ((int64_t)k0 + gt - past) * A.group - row0;
                        const int64_t to = A.window > 0 ? from + (int64_t)A.window * A.group : kRows8;
                        r0 = (int)max((int64_t)0, min(from, (int64_t)rows));
                        r1 = (int)max((int64_t)0, min(to, (int64_t)rows));
                    }
                    auto sees = [&](int r) -> bool { return r >= r0 && r < r1; };
                    auto scores = [&]() {
                        // the small parts first
                        uint32_t x[kAtOnce * kRows8];
#pragma unroll
                        for (int p0 = (kParts - 1) / kAtOnce * kAtOnce; p0 >= 0; p0 -= kAtOnce) {
                            constexpr int kRest = kParts % kAtOnce ? kParts % kAtOnce : kAtOnce;
                            const bool rest = p0 + kAtOnce > kParts;
                            if (rest) tc::ld_columns<kRest * kRows8>(x, t_s + p0 * kRows8);
                            else tc::ld_columns<kAtOnce * kRows8>(x, t_s + p0 * kRows8);
                            tc::wait_ld();
#pragma unroll
                            for (int r = 0; r < kRows8 / 2; ++r) {
#pragma unroll
                                for (int part = (rest ? kRest : kAtOnce) - 1; part >= 0; --part) {
                                    const uint64_t z = bits2(x[part * kRows8 + 2 * r], x[part * kRows8 + 2 * r + 1]);
                                    y[r] = p0 + part == kParts - 1 ? z : add2(y[r], z);
                                }
                            }
                        }
                        const uint64_t key_scale2 = pair2(key_scale, key_scale);
#pragma unroll
                        for (int r = 0; r < kRows8 / 2; ++r) y[r] = mul2(y[r], key_scale2);
                        if (__builtin_expect(masked, 0)) {
#pragma unroll
                            for (int r = 0; r < kRows8 / 2; ++r) {
                                float a, b;
                                unpair2(y[r], a, b);
                                if (!sees(2 * r)) a = -INFINITY;
                                if (!sees(2 * r + 1)) b = -INFINITY;
                                y[r] = pair2(a, b);
                            }
                        }
                    };
                    // (a byte of 255 is no scale: the vector is NaN)
                    const int e8 = value_byte == kScaleNan ? 0 : (int)value_byte - 127;
                    // (once more, from tensor memory, where references grow; the first block
                    // has none to begin with)
                    bool fresh = false;  // lane r: row r's reference is of the pass before
                    for (int pass = i == 0 ? 0 : -1;; ++pass) {
                        bool again = false;
                        scores();
                        if (__builtin_expect(pass >= 0, 0)) {
                            // the rows' maxima over the block, and new references where they grew
                            {
                                float v[kMaxRows8];
#pragma unroll
                                for (int r = 0; r < kMaxRows8; ++r) v[r] = -INFINITY;
                                const uint64_t value2 = pair2((float)e8 + shift, (float)e8 + shift);
#pragma unroll
                                for (int o = 0; o < kRows8 / 4; ++o) {
                                    const float4 f = *reinterpret_cast<const float4 *>(&q_factor[o * 4]);
                                    const float4 m = *reinterpret_cast<const float4 *>(&own.base[o * 4]);
                                    unpair2(add2(fma2(y[2 * o], pair2(f.x, f.y), pair2(m.x, m.y)), value2), v[4 * o],
                                            v[4 * o + 1]);
                                    unpair2(add2(fma2(y[2 * o + 1], pair2(f.z, f.w), pair2(m.z, m.w)), value2),
                                            v[4 * o + 2], v[4 * o + 3]);
                                }
                                own.across[gw][lane] =
                                    across_lanes(v, lane, [](float a, float b) { return fmaxf(a, b); });
                            }
                            group_barrier(1 + g);
                            float high = own.across[0][lane];
#pragma unroll
                            for (int w = 1; w < 4; ++w) high = fmaxf(high, own.across[w][lane]);
                            const bool unset = minus == kUnset;
                            const bool grow = high > (unset ? -INFINITY : kGrowAbove) || (fresh && high < kTop - kFarOff);
                            const float from = unset ? 0.f : minus;
                            float to = grow ? from - (high - kTop) : minus, by = 0.f;
                            // References from 2^26 on have steps of 4 and more, which may
                            // swallow a value's scale: the next pass has small numbers and
                            // finds out.  What a step is too large for, the group's shift
                            // takes, and the other rows' references take the shift back.
                            const float off = (to - from) + (high - kTop);
                            const unsigned far = __ballot_sync(0xffffffffu, grow && fabsf(off) > kFarOff);
                            if (__builtin_expect(far != 0, 0)) {
                                by = -__shfl_sync(0xffffffffu, off, __ffs(far) - 1);
                                shift += by;
                                if (!(far >> lane & 1)) to -= by;
                            }
                            fresh = grow && fabsf(to) >= kCoarse;
                            again = __any_sync(0xffffffffu, fresh) && pass < kMaxPasses;
                            const float h = unset ? 0.f : ex2(0.5f * ((to - from) + by));
                            const bool scaled = __any_sync(0xffffffffu, grow && !unset) || far != 0;
                            minus = to;
                            if (gw == 0) {
                                own.minus[lane] = minus;
                                own.base[lane] = minus == kUnset ? 0.f : minus;
                                own.factor[lane] = h;
                            }
                            group_barrier(1 + g);
                            if (i > 0) {
#pragma unroll
                                for (int o = 0; o < kRows8 / 4; ++o) {
                                    const float4 m = *reinterpret_cast<const float4 *>(&own.factor[o * 4]);
                                    const uint64_t a = pair2(m.x, m.y), b = pair2(m.z, m.w);
                                    sums[2 * o] = mul2(mul2(sums[2 * o], a), a);
                                    sums[2 * o + 1] = mul2(mul2(sums[2 * o + 1], b), b);
                                }
                                if (scaled) {
                                    hold8(sh, &sh.pv_done[g], (used - 1) & 1);
                                    __syncwarp();
                                    tc::fence_after();
#pragma unroll 1
                                    for (int part = 0; part < L::kOutCols / 8; ++part) {
                                        uint32_t o[8];
                                        tc::ld8(o, t_o + part * 8);
                                        tc::wait_ld();
#pragma unroll
                                        for (int e = 0; e < 8; ++e) {
                                            const float f = own.factor[part * 8 + e];
                                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f * f);
                                        }
                                        tc::st8(t_o + part * 8, o);
                                    }
                                    tc::wait_st();
                                }
                            }
                        }
                        // logarithms of weights times scales, and the largest of them
                        float top = -INFINITY;
                        const uint64_t value2 = pair2((float)e8 + shift, (float)e8 + shift);
#pragma unroll
                        for (int o = 0; o < kRows8 / 4; ++o) {
                            const float4 m = *reinterpret_cast<const float4 *>(&own.minus[o * 4]);
                            const float4 f = *reinterpret_cast<const float4 *>(&q_factor[o * 4]);
                            // (the products are exact: the factors are powers of two)
                            y[2 * o] = add2(fma2(y[2 * o], pair2(f.x, f.y), pair2(m.x, m.y)), value2);
                            y[2 * o + 1] = add2(fma2(y[2 * o + 1], pair2(f.z, f.w), pair2(m.z, m.w)), value2);
                            float a, b;
                            unpair2(y[2 * o], a, b);
                            top = max3(top, a, b);
                            unpair2(y[2 * o + 1], a, b);
                            top = max3(top, a, b);
                        }
                        if (pass >= 0 ? !again : !group_any(1 + g, top > kGrowAbove)) break;
                    }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.s_empty[g]);
                    // (what takes the scale out of a weight for the sums)
                    const float inv = power_of_two(max(-(e8 + kSumLift), -126));
                    const uint64_t inv2 = pair2(inv, inv);
                    if (used > 0) hold8(sh, &sh.pv_done[g], (used - 1) & 1);
                    __syncwarp();
                    char *row = smem + L::kP + gt * 128;  // the group's half of it
#pragma unroll
                    for (int o = 0; o < kRows8 / 8; ++o) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = o * 4 + e;
                            float a, b;
                            unpair2(y[r], a, b);
                            const uint64_t x = pair2(ex2(a), ex2(b));
                            sums[r] = fma2(x, inv2, sums[r]);
                            unpair2(x, a, b);
                            w[e] = pack2<__half>(a, b);
                        }
                        *reinterpret_cast<uint4 *>(row + (((4 * g + o) ^ (gt & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (__builtin_expect(value_byte == kScaleNan, 0)) {  // NaN for the rows that see it
#pragma unroll 1
                        for (int o = 0; o < kRows8 / 8; ++o) {
                            uint4 *at = reinterpret_cast<uint4 *>(row + (((4 * g + o) ^ (gt & 7)) * 16));
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int r = o * 8 + 2 * e;
                                w[e] = (sees(r) ? 0x7fffu : 0u) | (sees(r + 1) ? 0x7fff0000u : 0u);
                            }
                            *at = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_full[g]);
                }
                // (the rows' factors have been read for the last time)
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_empty[qb]);
                if (g == 1 && (blocks & 1)) {  // a last pair's second block that there is none of
                    if (lane == 0) mbar_arrive(&sh.scale_empty[sc.st]);
                    sc.next();
                }
            }
            // the tile's state, for the warps that finish it
            {
                float v[kMaxRows8];
#pragma unroll
                for (int r = 0; r < kMaxRows8; ++r) v[r] = 0.f;
#pragma unroll
                for (int r = 0; r < kRows8 / 2; ++r) unpair2(sums[r], v[2 * r], v[2 * r + 1]);
                const float sum = across_lanes(v, lane, [](float a, float b) { return a + b; });
                hold8<true>(sh, &sh.state_empty[tb], (tile >> 1 & 1) ^ 1);
                TileState &st = misc.tile[tb];
                st.sums[g][gw][lane] = sum;
                if (gw == 0) {
                    st.minus[g][lane] = minus;
                    if (lane == 0) st.shift[g] = shift;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.state_full[tb]);
                ++tile;
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (tid == 0 && sh.dead) atomicOr(status, SV_STATUS_TIMEOUT);
    if (warp == 13) {
        __syncwarp();
        tc::tmem_free(tmem, L::kCols);
    }
}

}  // namespace sv
