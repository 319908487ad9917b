// sv_attend.cuh -- attention of new tokens over the paged cache, on the
// fifth-generation tensor cores.
//
// Rows.  A kv head's queries are packed token by token, the G = q_heads /
// kv_heads heads of a token side by side: packed row j * G + g.  Every key and
// value is then read once for all G heads.  A tile is up to 256 packed rows of
// one (sequence, kv head), worked by two softmax groups of 128 threads, one
// thread per row:
//   pair tiles (more than 128 rows): group g has rows 128 g .. 128 g + 127 and
//     both walk all key blocks;
//   split tiles (up to 128 rows, rounds and single tokens): both groups have
//     the same rows and take the even and the odd key blocks; their softmax
//     states are joined at the end.
// A key block is 128 slots.  Per group and block: S = Q K^T (128 x 128 fp32 in
// tensor memory), the group's threads turn their rows of S into weights P
// (running maximum and sum in registers, fp32), written over S in 16 bits, and
// O += P V accumulates in tensor memory.  While one group computes weights the
// tensor cores work for the other.
//
// Running maximum.  Weights are taken relative to a reference that follows the
// maximum only when it has grown by more than 2^8: up to that the weights stay
// below 256 (fp16: below 2^15, see kHalfLift), which no type here overflows, and the
// 128 x head_dim rescaling of O is skipped for nearly all blocks.  P rounded to 16 bits is the one
// rounding between fp32 scores and the result; the sum is of the unrounded
// weights.
//
// Work split.  A tile costs its key blocks.  The batch's blocks in a fixed
// order (sequence, tile, head, block) are cut into equal runs, one per CTA, so
// every SM gets the same number of blocks whatever the lengths.  A tile cut
// between CTAs leaves partial states (unnormalised O, reference, sum) in the
// workspace, and the last CTA of a tile to arrive joins them in order: results
// do not depend on timing.
//
// Warps 0-7 softmax, 8 copies of keys and values (one TMA box per page piece and
// 64 values of a head, 128-byte swizzle), 9 issues the products, 10 copies of
// queries, 11 walks the CTA's run and publishes its pieces.  Every wait is
// bounded; when one gives up the CTA's warps leave at the next piece they miss,
// without further waits or copies, and the call reports SV_STATUS_TIMEOUT.
//
// Measured (32 query heads over 8 of 128, bf16, unless said otherwise):
//   rounds of 6 tokens over up to 4096 slots, 256 sequences: 367 us, 6.5 TB/s:
//     bound by memory;
//   6 tokens over 131071 slots, 2 sequences, 16 over 4 heads of 64 in fp16:
//     65 us, 4.1 TB/s: only 24 of 128 rows are used, so that one warp of each
//     group turns scores into weights, and its latency per key block shows;
//   two prompts of 8192 tokens: 0.73 ms in short bursts, 0.79 under sustained
//     load (1.5 and 1.4 PFLOP/s of the causal half): the softmax of a pair of
//     key blocks takes a group 2800 cycles where the products take 2048;
//   five chunks of up to 1025 tokens over up to 7000: 159 us (1.16 PFLOP/s):
//     the same, and each tile's start, end and joining;
//   one token over 1000 slots: 12.5 us, mostly latency (launch, table lookups,
//     one block after another, join).
#pragma once

#include <type_traits>

#include "sv_append.cuh"
#include "sv_cache.cuh"
#include "sv_pairs.cuh"
#include "sv_tc.cuh"

// 1: a build for the test of the bounded waits.  Every other CTA's scheduler stops
// after its first piece, without a word: the other warps wait for what never comes.
#ifndef SV_STALL
#define SV_STALL 0
#endif

namespace sv {

constexpr int kAttendThreads = 384;
// Registers per thread after the roles part: 256 softmax threads and 128 others
// share the 384 x 168 that the block is launched with.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kAttendThreads * 168, "register split");
constexpr int kRows = 128;           // packed rows per softmax group
constexpr int kKeys = 128;           // slots per key block
constexpr int kAttendMaxCtas = 160;  // partial states the workspace holds room for
constexpr uint32_t kTmemCols = 512;
constexpr int kNoPage = 0x7fffffff;  // outside every cache: its boxes read zeros
// fp16 weights are taken 2^7 times as large (2^15 at most): numbers below 2^-14 are
// held in steps of 2^-24, and without this what a key far below the reference weighs
// vanished (20,000 of 2^-25 beside one of 1: all of their 0.0005).
constexpr float kHalfLift = 7.f;
constexpr float kRescaleAbove = 8.f;  // log2 (0: 0.90 instead of 0.79 ms for two prompts of 8192)

// Workspace: header (status), tile counters [ctas][2], partial statistics
// [ctas * 2 slots][2 groups][128 rows] (reference, sum), partial O
// [ctas * 2][32 column quads][256 rows] float4.
constexpr size_t kAttendCounters = 256;
constexpr size_t kAttendStats = kAttendCounters + 2 * 4 * 256;
constexpr size_t kAttendOut = kAttendStats + (size_t)kAttendMaxCtas * 2 * 2 * kRows * sizeof(float2);
constexpr size_t kAttendWorkspace =
    kAttendOut + (size_t)kAttendMaxCtas * 2 * (kMaxHeadDim / 4) * 2 * kRows * sizeof(float4);

struct AttendParams {
    Batch batch;
    FastDiv by_group, by_page;
    const void *q;
    void *out;
    int64_t q_st[2], o_st[2];
    int32_t q_heads, kv_heads, group, head_dim, window;
    int32_t piece;      // slots per copied box: the largest power of two in page_size, <= 128
    float scale_log2;   // |scale| * log2(e); the sign goes into q
    int32_t q_mode;     // 0: q, 1: -q, 2: zeros (scale 0)
    int32_t wide_out;   // rows of out start on 32 bytes
    int32_t q_boxes;    // queries come by TMA boxes (else the softmax threads load them)
    char *workspace;
};

template <int DP>
struct AttendSmem {
    static constexpr int kTile = kRows * DP * 2;  // a Q tile, a K or V block
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr int kStats = 1024;               // states of the two groups
    static constexpr int kMisc = kStats + 2 * kRows * 8;
    static constexpr int kBytes = kMisc + (2 + kStages) * kTile;
};

// ---------------------------------------------------------------------------
// the split of the work

// a / b for a, b >= 0: most quotients here are of small numbers, and a 64-bit
// division costs hundreds of cycles.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// A tile's fixed cost (queries in, states joined, rows out) in key blocks: 2
// and 4 measure alike, 0 takes 1.05 instead of 0.79 ms for two prompts of 8192
// tokens (CTAs with many short tiles finish late).
constexpr int kTileCost = 2;

// (kTileRows: packed rows of a tile; kFixed: its fixed cost.)
template <int kTileRows, int kFixed>
struct SeqCost {
    int32_t n, len, row0, tiles, packed;  // packed: rows n * G
    __device__ __forceinline__ void load(const AttendParams &A, int32_t b) {
        const Sequence s = load_sequence(A.batch, b);
        n = s.n;
        len = s.len;
        row0 = s.row0;
        packed = n * A.group;  // the host checks that it fits
        tiles = (packed + kTileRows - 1) / kTileRows;
    }
    __device__ __forceinline__ int rows(int t) const { return min(kTileRows, packed - t * kTileRows); }
    // key blocks [lo, hi) that tile t's rows see, and one past its last slot
    __device__ __forceinline__ void blocks(const AttendParams &A, int t, int &lo, int &hi,
                                           int &end) const {
        const int r0 = t * kTileRows;
        end = max(0, len - n + A.by_group.div(r0 + rows(t) - 1) + 1);
        hi = (end + kKeys - 1) / kKeys;
        lo = A.window > 0 ? max(0, len - n + A.by_group.div(r0) - A.window + 1) / kKeys : 0;
        lo = min(lo, hi);
    }
    __device__ __forceinline__ int cost(const AttendParams &A, int t) const {
        int lo, hi, end;
        blocks(A, t, lo, hi, end);
        return kFixed + max(1, hi - lo);
    }
};

// One CTA's part of a tile, as the scheduler warp publishes it.
struct Piece {
    int32_t n;                  // its key blocks; -1: no more pieces
    int32_t lo;                 // the first of them
    int32_t n1;                 // blocks of group 1 (group 0 has the others)
    int32_t split;              // split tile
    int32_t b, h;
    int32_t row, rows;          // first packed row of the tile, rows of the tile
    int32_t end;                // one past the tile's last slot
    int32_t token;              // first token row of the sequence
    int32_t past;               // slots before its new tokens
    int32_t first, parts;       // CTA that holds the tile's first block, CTAs that share the tile
    int32_t pad[3];
};

// Walks one CTA's run of the work (a whole warp).
template <int kTileRows, int kFixed>
struct Walker {
    SeqCost<kTileRows, kFixed> s;
    int32_t b, t, h, off;
    int64_t left, unit, total;
    int32_t ctas;

    __device__ __forceinline__ void start(const AttendParams &A, int32_t b0, int64_t skip,
                                          int64_t unit0, int64_t count, int64_t total_,
                                          int32_t ctas_, int lane) {
        b = b0;
        left = count;
        unit = unit0;
        total = total_;
        ctas = ctas_;
        t = h = off = 0;
        if (left <= 0) return;
        s.load(A, b);
        for (;; t += 32) {  // the tile that unit `skip` of the sequence lies in
            const int64_t own = t + lane < s.tiles ? (int64_t)s.cost(A, t + lane) * A.kv_heads : 0;
            int64_t inc = own;
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += o;
            }
            const unsigned at = __ballot_sync(0xffffffffu, inc > skip);
            if (at || t + 32 >= s.tiles) {
                const int w = at ? __ffs(at) - 1 : 31;
                skip -= __shfl_sync(0xffffffffu, inc - own, w);
                t += w;
                break;
            }
            skip -= __shfl_sync(0xffffffffu, inc, 31);
        }
        const int c = s.cost(A, t);
        h = (int32_t)quotient(skip, c);
        off = (int32_t)(skip - (int64_t)h * c);
    }

    __device__ __forceinline__ int32_t cta_of(int64_t u) const {
        return (int32_t)quotient((u + 1) * ctas - 1, total);
    }

    __device__ __forceinline__ bool next(const AttendParams &A, Piece &p) {
        while (left > 0) {
            while (t >= s.tiles) {
                if (++b >= A.batch.B) return false;
                s.load(A, b);
                t = h = off = 0;
            }
            int lo, hi, end;
            s.blocks(A, t, lo, hi, end);
            const int cost = kFixed + max(1, hi - lo);
            const int from = off, to = (int)min((int64_t)cost, off + left);
            p.b = b;
            p.h = h;
            p.row = t * kTileRows;
            p.rows = s.rows(t);
            p.end = end;
            p.token = s.row0;
            p.past = s.len - s.n;
            const int64_t unit_of_tile = unit - off;
            left -= to - from;
            unit += to - from;
            off = to;
            if (to == cost) {
                off = 0;
                if (++h >= A.kv_heads) {
                    h = 0;
                    ++t;
                }
            }
            if (to <= kFixed) continue;  // the run ends before the tile's first block
            p.lo = lo + max(0, from - kFixed);
            p.n = hi > lo ? to - max(from, kFixed) : 0;
            p.split = p.rows <= kRows;
            p.n1 = p.split ? p.n / 2 : p.n;
            p.first = from <= kFixed ? (int32_t)blockIdx.x : cta_of(unit_of_tile + kFixed);
            p.parts = (to == cost ? (int32_t)blockIdx.x : cta_of(unit_of_tile + cost - 1)) - p.first + 1;
            return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------------------

constexpr int kPieces = 4;  // pieces the scheduler may be ahead
// arrivals that free a piece: softmax warps, keys and values, queries, products
constexpr int kPieceReaders = 11;

struct AttendShared {
    unsigned long long full[8], empty[8];
    unsigned long long s_full[2], p_full[2][2], o_full[2], q_full[2], q_free[2], drain;
    unsigned long long piece_full[kPieces], piece_empty[kPieces];
    unsigned long long group_sync[2], both_sync;
    Piece pieces[kPieces];
    uint32_t tmem;
    int32_t dead, b0, last[2];
    int64_t skip;
    int64_t sums[kAttendThreads / 32];
};
static_assert(sizeof(AttendShared) <= 1024, "misc region");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 32 values of a row (those below `left`), in 32-byte stores where the rows
// allow: a thread has a row of its own, so a store touches as many lines as it
// has lanes, and half the stores take half the time.
__device__ __forceinline__ void store_row(uint16_t *to, const uint32_t (&y)[16], int left,
                                          bool wide) {
#pragma unroll
    for (int e = 0; e < 16; e += 8) {
        if (wide && 2 * e + 16 <= left) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 2 * e),
                         "r"(y[e]), "r"(y[e + 1]), "r"(y[e + 2]), "r"(y[e + 3]), "r"(y[e + 4]),
                         "r"(y[e + 5]), "r"(y[e + 6]), "r"(y[e + 7])
                         : "memory");
        } else {
            if (2 * e < left)
                *reinterpret_cast<uint4 *>(to + 2 * e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            if (2 * e + 8 < left)
                *reinterpret_cast<uint4 *>(to + 2 * e + 8) =
                    make_uint4(y[e + 4], y[e + 5], y[e + 6], y[e + 7]);
        }
    }
}

// A wait that gives up for the whole CTA.
template <uint64_t kLimitNs = kWaitLimitNs>
__device__ __forceinline__ bool hold(AttendShared &sh, unsigned long long *bar, uint32_t parity,
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

// The scheduler and the queries' warp wait for whole pieces, whose millions of slots
// may well take seconds (2^31 of them half a minute); the others wait for a key
// block at most, and when one of them gives up these see it.  (A limit that any
// progress renews: 2 us of 65 for 6 tokens over 131071 slots.)
constexpr uint64_t kPieceLimitNs = 100000000000ull;

// The pieces as a reader warp sees them, in order.
struct PieceReader {
    int k = 0;
    uint32_t turn = 0;
    template <uint64_t kLimitNs = kWaitLimitNs>
    __device__ __forceinline__ const Piece *next(AttendShared &sh, uint32_t *status) {
        const bool ok = __all_sync(0xffffffffu, hold<kLimitNs>(sh, &sh.piece_full[k], turn, status));
        return ok && sh.pieces[k].n >= 0 ? &sh.pieces[k] : nullptr;
    }
    __device__ __forceinline__ void done(AttendShared &sh, int lane) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.piece_empty[k]);
        if (++k == kPieces) {
            k = 0;
            turn ^= 1;
        }
    }
};

// A barrier among warps, by an mbarrier so that the wait is bounded: no warp
// hangs when another has left after a timeout.
__device__ __forceinline__ void meet(AttendShared &sh, unsigned long long *bar, uint32_t &turn,
                                     int lane, uint32_t *status) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    hold(sh, bar, turn, status);
    __syncwarp();
    turn ^= 1;
}

// Cost of sequence b's tiles over all heads, for each lane's own b (< 0: none).
template <int kTileRows, int kFixed>
__device__ __forceinline__ int64_t sequence_cost(const AttendParams &A, int32_t b, int lane) {
    SeqCost<kTileRows, kFixed> s;
    s.n = s.len = s.tiles = s.packed = 0;
    if (b >= 0) s.load(A, b);
    int64_t c = 0;
    if (s.tiles <= 2)
        for (int t = 0; t < s.tiles; ++t) c += s.cost(A, t);
    // long prompts: the whole warp adds up one lane's tiles
    unsigned long_ones = __ballot_sync(0xffffffffu, s.tiles > 2);
    while (long_ones) {
        const int who = __ffs(long_ones) - 1;
        long_ones &= long_ones - 1;
        SeqCost<kTileRows, kFixed> o;
        o.n = __shfl_sync(0xffffffffu, s.n, who);
        o.len = __shfl_sync(0xffffffffu, s.len, who);
        o.tiles = __shfl_sync(0xffffffffu, s.tiles, who);
        o.packed = __shfl_sync(0xffffffffu, s.packed, who);
        int64_t x = 0;
        for (int t = lane; t < o.tiles; t += 32) x += o.cost(A, t);
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (lane == who) c = x;
    }
    return c * A.kv_heads;
}

template <class T, int DP>
__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ AttendParams A, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
    typedef AttendSmem<DP> L;
    constexpr bool kBf16 = sizeof(T) == 2 && __is_same(T, __nv_bfloat16);
    constexpr float kLift = kBf16 ? 0.f : kHalfLift;
    constexpr int kHalves = DP / 64;
    constexpr int kHalfBytes = kKeys * 128;
    constexpr uint32_t kIdescS = tc::instr_desc(kBf16, false, kRows, kKeys);
    constexpr uint32_t kIdescO = tc::instr_desc(kBf16, true, kRows, DP);
    extern __shared__ __align__(1024) char smem[];
    AttendShared &sh = *reinterpret_cast<AttendShared *>(smem);
    char *sq = smem + L::kMisc;
    char *ring = sq + 2 * L::kTile;
    const int tid = threadIdx.x, warp = tc::uniform(tid / 32), lane = tid % 32;
    uint32_t *status = A.batch.status;

    if (smem_u32(smem) & 1023) {  // the swizzle counts on it; no room is left to round up
        if (tid == 0) atomicOr(status, SV_STATUS_TIMEOUT);
        return;
    }
    if (warp == 9) tc::tmem_alloc(&sh.tmem, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&sh.s_full[g], 1);
            mbar_init(&sh.p_full[g][0], 4);
            mbar_init(&sh.p_full[g][1], 4);
            mbar_init(&sh.o_full[g], 1);
            mbar_init(&sh.q_full[g], A.q_boxes ? 1 : 4);
            mbar_init(&sh.q_free[g], 1);
        }
        mbar_init(&sh.drain, 1);
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&sh.piece_full[i], 1);
            mbar_init(&sh.piece_empty[i], kPieceReaders);
        }
        mbar_init(&sh.group_sync[0], 4);
        mbar_init(&sh.group_sync[1], 4);
        mbar_init(&sh.both_sync, 8);
        sh.dead = 0;
        sh.b0 = -1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    wait_for_primary_grid();

    // the batch's blocks, and where this CTA's run of them begins
    int64_t c = 0, last_cost = 0;
    for (int32_t b0 = 0; b0 < A.batch.B; b0 += kAttendThreads) {
        const int32_t b = b0 + tid < A.batch.B ? b0 + tid : -1;
        last_cost = sequence_cost<2 * kRows, kTileCost>(A, b, lane);
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
    for (int w = 0; w < kAttendThreads / 32; ++w) total += sh.sums[w];
    const int32_t ctas = (int32_t)min((int64_t)gridDim.x, max((int64_t)1, total));
    const int64_t u0 = quotient((int64_t)blockIdx.x * total, ctas),
                  u1 = quotient(((int64_t)blockIdx.x + 1) * total, ctas);
    const bool idle = total == 0 || (int32_t)blockIdx.x >= ctas || u0 >= u1;
    if (!idle) {
        int64_t base = 0;
        for (int32_t b0 = 0; b0 < A.batch.B; b0 += kAttendThreads) {
            const int32_t b = b0 + tid < A.batch.B ? b0 + tid : -1;
            const int64_t own = A.batch.B <= kAttendThreads ? last_cost : sequence_cost<2 * kRows, kTileCost>(A, b, lane);
            int64_t inc = own;
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += o;
            }
            __syncthreads();
            if (lane == 31) sh.sums[warp] = inc;
            __syncthreads();
            int64_t at = base;
            for (int w = 0; w < kAttendThreads / 32; ++w) {
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
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 11) {
            // ---- the schedule ---------------------------------------------
            Walker<2 * kRows, kTileCost> walk;
            walk.left = 0;
            if (!idle) walk.start(A, sh.b0, sh.skip, u0, u1 - u0, total, ctas, lane);
            int k = 0;
            uint32_t turn = 1;
            for (bool more = true; more;) {
                Piece p;
                more = walk.next(A, p);
                if (!more) p.n = -1;
                if (SV_STALL && k == 1 && blockIdx.x % 2 == 1) break;
                // (after a timeout the readers stop at the first piece they miss)
                if (!__all_sync(0xffffffffu, hold<kPieceLimitNs>(sh, &sh.piece_empty[k], turn, status))) break;
                if (lane == 0) {
                    sh.pieces[k] = p;
                    mbar_arrive(&sh.piece_full[k]);
                }
                __syncwarp();
                if (++k == kPieces) {
                    k = 0;
                    turn ^= 1;
                }
            }
        } else if (warp == 8) {
            // ---- copies of keys and values --------------------------------
            const int pieces = kKeys / A.piece;
            const int mine = lane % pieces, half = lane / pieces;
            const bool active = half < kHalves;
            char *dst = ring + half * kHalfBytes + mine * A.piece * 128;
            int it = 0, st = 0;
            uint32_t turn = 1;  // parity of the stage's last release
            PieceReader reader;
            while (const Piece *pp = reader.next(sh, status)) {
                const Piece p = *pp;
                reader.done(sh, lane);
                if (p.n == 0) continue;
                const int32_t *table = A.batch.pages + p.b * A.batch.pages_stride;
                const int first = A.window > 0 ? p.past + A.by_group.div(p.row) - A.window + 1 : 0;
                // this lane's slots of block i: page id, or one outside the cache
                // (its box reads zeros) where no row looks
                auto page_of = [&](int i) -> int {
                    const int s0 = (p.lo + i) * kKeys + mine * A.piece;
                    if (!active || i >= p.n || s0 >= p.end || s0 + A.piece <= first) return kNoPage;
                    return __ldg(table + A.by_page.div(s0));
                };
                auto load = [&](const CUtensorMap &map, int i, int id) {
                    if (__all_sync(0xffffffffu, hold(sh, &sh.empty[st], turn, status))) {
                        if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], L::kTile);
                        __syncwarp();
                        if (active) {
                            const int s0 = (p.lo + i) * kKeys + mine * A.piece;
                            tc::load_box(dst + st * L::kTile, &map, half * 64, p.h,
                                         s0 - A.by_page.div(s0) * A.batch.page_size, id,
                                         &sh.full[st]);
                        }
                        ++it;
                        if (++st == L::kStages) {
                            st = 0;
                            turn ^= 1;
                        }
                    }
                    __syncwarp();
                };
                auto checked = [&](int id) -> int {
                    if (id != kNoPage && (id < 0 || id >= A.batch.num_pages)) {
                        atomicOr(status, SV_STATUS_BAD_PAGE);
                        id = kNoPage;
                    }
                    return id;
                };
                // keys run ahead of values by one block (pair) or two (split);
                // page ids are fetched one block further ahead
                const int ahead = p.split ? 2 : 1;
                int id0 = page_of(0), id1 = page_of(1), id2 = page_of(2);
                id0 = checked(id0);
                load(kmap, 0, id0);
                id1 = checked(id1);
                if (ahead == 2 && p.n > 1) load(kmap, 1, id1);
                for (int i = 0; i < p.n; ++i) {
                    const int id3 = page_of(i + 3);
                    load(vmap, i, id0);
                    id2 = checked(id2);
                    if (i + ahead < p.n) load(kmap, i + ahead, ahead == 2 ? id2 : id1);
                    id0 = id1;
                    id1 = id2;
                    id2 = id3;
                }
            }
            // the last fills must have been taken before the CTA may end; after a
            // wait gave up, here or elsewhere, they must at least have landed
            for (int k = max(0, it - L::kStages); k < it; ++k)
                hold(sh, &sh.empty[k % L::kStages], (k / L::kStages) & 1, status);
            if (*(volatile int32_t *)&sh.dead)
                for (int k = max(0, it - L::kStages); k < it; ++k)
                    mbar_wait(&sh.full[k % L::kStages], (k / L::kStages) & 1);
        } else if (warp == 9) {
            // ---- products -----------------------------------------------------
            const uint32_t tm = (uint32_t)tc::uniform((int)tmem);
            int st = 0;
            uint32_t turn = 0, qn0 = 0, qn1 = 0, pn0 = 0, pn1 = 0;
            const uint32_t ring_at = smem_u32(ring);
            const uint64_t q_desc = tc::smem_desc(smem_u32(sq), 16, 1024);
            const uint64_t k_desc = tc::smem_desc(ring_at, 16, 1024);
            const uint64_t v_desc = tc::smem_desc(ring_at, kHalfBytes, 1024);
            // (a descriptor's start address is in units of 16 bytes)
            // Once a fill did not come, nothing is handed back any more: a stage or a
            // query tile that is still being filled must not be filled again.
            // (Each lane's own; the elected one's counts.)
            bool filled = true;
            auto acquire = [&]() -> int {  // the next stage, filled
                const int x = st;
                if (!hold(sh, &sh.full[x], turn, status)) filled = false;
                if (++st == L::kStages) {
                    st = 0;
                    turn ^= 1;
                }
                return x;
            };
            auto release = [&](int x) {
                if (tc::elect() && filled) tc::commit(&sh.empty[x]);
            };
            auto scores = [&](auto gc, int x, bool last) {  // S_g = Q_g K^T
                constexpr int g = decltype(gc)::value;
                tc::fence_after();
                if (tc::elect()) {
                    const uint64_t kd = k_desc + (uint32_t)(x * (L::kTile / 16));
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        const uint32_t at = ((k / 4) * kHalfBytes + (k % 4) * 32) / 16;
                        tc::mma_ss(tm + g * kKeys, q_desc + (g * (L::kTile / 16) + at), kd + at, kIdescS,
                                   k > 0);
                    }
                    tc::commit(&sh.s_full[g]);
                    if (last && filled) tc::commit(&sh.q_free[g]);
                }
                __syncwarp();
            };
            auto values = [&](auto gc, int x, bool add) {  // O_g (+)= P_g V
                constexpr int g = decltype(gc)::value;
                const uint32_t phase = (g ? pn1++ : pn0++) & 1;
                const uint64_t vd = v_desc + (uint32_t)(x * (L::kTile / 16));
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // the weights come in two halves
                    hold(sh, &sh.p_full[g][half], phase, status);
                    tc::fence_after();
                    if (tc::elect()) {
#pragma unroll
                        for (int k = half * (kKeys / 32); k < (half + 1) * (kKeys / 32); ++k)
                            tc::mma_ts(tm + 2 * kKeys + g * 128, tm + g * kKeys + k * 8,
                                       vd + k * (2048 / 16), kIdescO, add || k > 0);
                    }
                    __syncwarp();
                }
            };
            const std::integral_constant<int, 0> g0{};
            const std::integral_constant<int, 1> g1{};
            // slots past the tile's last one in a page that holds it: their weights
            // are zero, and zero times whatever lies there must be zero
            auto clear_tail = [&](int st, int kb, int end) {
                const int r0 = end - kb * kKeys;
                if (r0 >= kKeys || r0 <= 0) return;
                const int r1 = min(kKeys, (r0 + A.piece - 1) / A.piece * A.piece);
                if (r0 == r1) return;
                char *v = ring + st * L::kTile;
                for (int i = lane; i < (r1 - r0) * 8 * kHalves; i += 32) {
                    const int half = i / ((r1 - r0) * 8), x = i - half * (r1 - r0) * 8;
                    *reinterpret_cast<uint4 *>(v + half * kHalfBytes + r0 * 128 + x * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                tc::fence_async_smem();
                __syncwarp();
            };
            PieceReader reader;
            while (const Piece *p = reader.next(sh, status)) {
                const int blocks = tc::uniform(p->n), lo = tc::uniform(p->lo), n1 = tc::uniform(p->n1);
                const int end = tc::uniform(p->end);
                const bool split = tc::uniform(p->split);
                reader.done(sh, lane);
                if (blocks == 0) continue;
                if (!hold(sh, &sh.q_full[0], qn0++ & 1, status)) filled = false;
                if (split) {
                    int x = acquire();
                    scores(g0, x, blocks <= 2);
                    release(x);
                    if (n1 > 0) {
                        if (!hold(sh, &sh.q_full[1], qn1++ & 1, status)) filled = false;
                        x = acquire();
                        scores(g1, x, blocks <= 3);
                        release(x);
                    }
                    auto step = [&](auto gc, int i) {  // block i of the tile's run
                        constexpr int g = decltype(gc)::value;
                        x = acquire();
                        clear_tail(x, lo + i, end);
                        values(gc, x, i > 1);
                        release(x);
                        if (i + 2 < blocks) {
                            x = acquire();
                            scores(gc, x, i + 4 >= blocks);
                            release(x);
                        } else if (tc::elect()) {
                            tc::commit(&sh.o_full[g]);
                        }
                    };
                    for (int i = 0; i < blocks; i += 2) {
                        step(g0, i);
                        if (i + 1 < blocks) step(g1, i + 1);
                    }
                } else {
                    if (!hold(sh, &sh.q_full[1], qn1++ & 1, status)) filled = false;
                    int ks = acquire();
                    scores(g0, ks, blocks == 1);
                    scores(g1, ks, blocks == 1);
                    release(ks);
                    for (int i = 0; i < blocks; ++i) {
                        const int vs = acquire();
                        clear_tail(vs, lo + i, end);
                        const bool more = i + 1 < blocks;
                        values(g0, vs, i > 0);
                        if (more) {
                            ks = acquire();
                            scores(g0, ks, i + 2 == blocks);
                        } else if (tc::elect()) {
                            tc::commit(&sh.o_full[0]);
                        }
                        values(g1, vs, i > 0);
                        release(vs);
                        if (more) {
                            scores(g1, ks, i + 2 == blocks);
                            release(ks);
                        } else if (tc::elect()) {
                            tc::commit(&sh.o_full[1]);
                        }
                    }
                }
                __syncwarp();
            }
            if (tc::elect()) tc::commit(&sh.drain);
            __syncwarp();
            mbar_wait(&sh.drain, 0);
        } else if (A.q_boxes) {
            // ---- copies of queries: a tile's boxes as soon as the last scores
            // of the tile before it are done
            uint32_t qn0 = 0, qn1 = 0;
            PieceReader reader;
            while (const Piece *pp = reader.next<kPieceLimitNs>(sh, status)) {
                const Piece p = *pp;
                reader.done(sh, lane);
                if (p.n == 0) continue;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (g == 1 && p.n1 == 0) continue;
                    const uint32_t turn = ((g ? qn1 : qn0) & 1) ^ 1;
                    if (!__all_sync(0xffffffffu, hold<kPieceLimitNs>(sh, &sh.q_free[g], turn, status))) continue;
                    const int r0 = p.row + (p.split ? 0 : g * kRows);
                    if (lane == 0) mbar_arrive_expect_tx(&sh.q_full[g], L::kTile);
                    __syncwarp();
                    if (lane < kHalves)
                        tc::load_box(sq + g * L::kTile + lane * kHalfBytes, &qmap, lane * 64, 0, p.h,
                                     p.token + A.by_group.div(r0), &sh.q_full[g]);
                    if (g) ++qn1;
                    else ++qn0;
                }
            }
            // every box has landed before the CTA may end
            if (qn0 > 0) mbar_wait(&sh.q_full[0], (qn0 - 1) & 1);
            if (qn1 > 0) mbar_wait(&sh.q_full[1], (qn1 - 1) & 1);
        } else {
            PieceReader reader;
            while (reader.next<kPieceLimitNs>(sh, status)) reader.done(sh, lane);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---- softmax ------------------------------------------------------
        const int g = warp / 4, gw = warp % 4, gt = gw * 32 + lane;
        const uint32_t t_s = tmem + ((uint32_t)(gw * 32) << 16) + g * kKeys;
        const uint32_t t_o = tmem + ((uint32_t)(gw * 32) << 16) + 2 * kKeys;  // group 0's O
        float2 *stats = reinterpret_cast<float2 *>(smem + L::kStats);
        const int D = A.head_dim;
        uint32_t sn = 0, own_n = 0, other_n = 0, group_turn = 0, both_turn = 0;
        PieceReader reader;
        while (const Piece *pp = reader.next(sh, status)) {
            const Piece &p = *pp;
            const bool split = p.split != 0;
            const int steps = g == 0 && split ? p.n - p.n1 : p.n1;
            const int r_base = p.row + (split ? 0 : g * kRows);
            const int rows = split ? p.rows : min(kRows, p.rows - g * kRows);
            if (steps > 0 && !A.q_boxes) {
                // eight loads in flight per thread
                char *q_s = sq + g * L::kTile;
                constexpr int kChunks = DP / 8, kStep = 128 / kChunks;
                const int ch = gt % kChunks;
                const uint32_t flip = A.q_mode == 1 ? 0x80008000u : 0u;
                for (int r0 = gt / kChunks; r0 < rows; r0 += 8 * kStep) {
                    uint4 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r0 + i * kStep;
                        x[i] = make_uint4(0, 0, 0, 0);
                        if (r < rows && ch * 8 < D && A.q_mode != 2) {
                            const int pr = r_base + r, j = A.by_group.div(pr);
                            const int hq = p.h * A.group + (pr - j * A.group);
                            x[i] = __ldg(reinterpret_cast<const uint4 *>(
                                static_cast<const uint16_t *>(A.q) +
                                (int64_t)(p.token + j) * A.q_st[0] + hq * A.q_st[1] + ch * 8));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r0 + i * kStep;
                        if (r < rows)
                            *reinterpret_cast<uint4 *>(q_s + (ch / 8) * kHalfBytes + r * 128 +
                                                       (((ch % 8) ^ (r & 7)) * 16)) =
                                make_uint4(x[i].x ^ flip, x[i].y ^ flip, x[i].z ^ flip, x[i].w ^ flip);
                    }
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full[g]);
            }
            const bool mine = gt < rows;        // this thread's row exists
            const bool any = gw * 32 < rows;    // one of the warp's does
            float ref = -INFINITY, sum = 0.f;
            {
                // last slot the row sees, relative to the block at hand
                int limit = mine ? p.past + A.by_group.div(r_base + gt) : 0x7fffff00;
                const int k0 = (p.lo + (split ? g : 0)) * kKeys;
                limit -= k0;
                const int stride = split ? 2 * kKeys : kKeys;
                const int span = A.window > 0 ? A.window : 0x7fffffff;  // slots a row may see
                for (int i = 0; i < steps; ++i, limit -= stride) {
                    hold(sh, &sh.s_full[g], sn++ & 1, status);
                    __syncwarp();
                    if (!any) {
                        if (lane == 0) {
                            mbar_arrive(&sh.p_full[g][0]);
                            mbar_arrive(&sh.p_full[g][1]);
                        }
                        continue;
                    }
                    tc::fence_after();
                    uint32_t x[4][32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc::ld32(x[q], t_s + 32 * q);
                    tc::wait_ld();
                    if (__any_sync(0xffffffffu, mine && (limit < kKeys - 1 || limit >= span))) {
                        const int lo = max(limit, -1) - span + 1;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * q + e > limit || 32 * q + e < lo) x[q][e] = 0xff800000u;
                    }
                    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            m[q] = max3(m[q], __uint_as_float(x[q][e]), __uint_as_float(x[q][e + 1]));
                    const float top = fmaxf(max3(m[0], m[1], m[2]), m[3]) * A.scale_log2;
                    const bool grow =
                        mine && (top > ref + kRescaleAbove || (ref == -INFINITY && top > ref));
                    if (__any_sync(0xffffffffu, grow)) {
                        const float to = grow ? top : ref;
                        const float f = grow ? (ref == -INFINITY ? 0.f : ex2(ref - to)) : 1.f;
                        if (i > 0 && __any_sync(0xffffffffu, grow && ref != -INFINITY)) {
#pragma unroll 1
                            for (int q = 0; q < DP / 16; ++q) {
                                uint32_t o[16];
                                tc::ld16(o, t_o + g * 128 + 16 * q);
                                tc::wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::st16(t_o + g * 128 + 16 * q, o);
                            }
                        }
                        sum *= f;
                        ref = to;
                    }
                    const float minus = ref == -INFINITY ? 0.f : kLift - ref;
                    const uint64_t scale2 = pair2(A.scale_log2, A.scale_log2), minus2 = pair2(minus, minus);
                    uint64_t sums = 0;  // of even and odd columns
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int q = 2 * half; q < 2 * half + 2; ++q) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float a, b;
                                unpair2(fma2(bits2(x[q][2 * e], x[q][2 * e + 1]), scale2, minus2), a, b);
                                a = ex2(a);
                                b = ex2(b);
                                sums = add2(sums, pair2(a, b));
                                w[e] = pack2<T>(a, b);
                            }
                            tc::st16(t_s + 16 * q, w);
                        }
                        tc::wait_st();
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.p_full[g][half]);
                    }
                    float even, odd;
                    unpair2(sums, even, odd);
                    sum += even + odd;
                }
            }
            const int other_steps = g == 0 ? (split ? p.n1 : 0) : (split ? p.n - p.n1 : 0);
            float own_f = 1.f, other_f = 0.f;  // factors of the two groups' O
            if (split) {
                // join the groups' states; group g then has half the columns
                if (steps > 0) hold(sh, &sh.o_full[g], own_n++ & 1, status);
                if (other_steps > 0) hold(sh, &sh.o_full[1 - g], other_n++ & 1, status);
                stats[g * kRows + gt] = make_float2(ref, sum);
                meet(sh, &sh.both_sync, both_turn, lane, status);
                const float2 o = stats[(1 - g) * kRows + gt];
                const float to = fmaxf(ref, o.x);
                own_f = ref == -INFINITY ? 0.f : ex2(ref - to);
                other_f = o.x == -INFINITY ? 0.f : ex2(o.x - to);
                sum = sum * own_f + o.y * other_f;
                ref = to;
            } else if (steps > 0) {
                hold(sh, &sh.o_full[g], own_n++ & 1, status);
                // the other group's accumulators went through a phase too; this
                // group next waits for them in a split tile, where its own
                // phase (or the other's, for group 1) comes later in the
                // order of the products
                ++other_n;
            }
            __syncwarp();
            tc::fence_after();
            const int c0 = split ? g * (DP / 2) : 0;      // this group's columns
            const int c1 = split ? c0 + DP / 2 : DP;
            const int part_row = split ? 0 : g * kRows;
            const int slot = blockIdx.x * 2 + ((int)blockIdx.x == p.first ? 1 : 0);
            auto row_of = [&](int r) -> uint16_t * {      // row r of the group in out
                const int pr = r_base + r, j = A.by_group.div(pr);
                return static_cast<uint16_t *>(A.out) + (int64_t)(p.token + j) * A.o_st[0] +
                       (p.h * A.group + (pr - j * A.group)) * A.o_st[1];
            };
            if (any) {
                const float inv = sum > 0.f ? 1.f / sum : 0.f;
                uint16_t *out = row_of(gt);
                float4 *part = reinterpret_cast<float4 *>(A.workspace + kAttendOut) +
                               (int64_t)slot * (kMaxHeadDim / 4) * 256 + part_row + gt;
#pragma unroll 1
                for (int cc = c0; cc < c1; cc += 32) {
                    float v[32];
                    uint32_t o[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                    if (steps > 0) {
                        tc::ld32(o, t_o + g * 128 + cc);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = own_f * __uint_as_float(o[e]);
                    }
                    if (split && other_steps > 0) {
                        tc::ld32(o, t_o + (1 - g) * 128 + cc);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = fmaf(other_f, __uint_as_float(o[e]), v[e]);
                    }
                    if (p.parts > 1) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            part[(cc + e) / 4 * 256] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    } else if (mine) {
                        uint32_t y[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            y[e] = sum == 0.f ? 0u : pack2<T>(v[2 * e] * inv, v[2 * e + 1] * inv);
                        store_row(out + cc, y, D - cc, A.wide_out);
                    }
                }
                tc::fence_before();
            }
            if (p.parts > 1) {
                float2 *part_stats = reinterpret_cast<float2 *>(A.workspace + kAttendStats);
                const float4 *part_out = reinterpret_cast<const float4 *>(A.workspace + kAttendOut);
                part_stats[(slot * 2 + g) * kRows + gt] = make_float2(ref, sum);
                meet(sh, &sh.group_sync[g], group_turn, lane, status);
                if (gt == 0) {
                    __threadfence();   // the group's writes, after the meeting
                    uint32_t *c = reinterpret_cast<uint32_t *>(A.workspace + kAttendCounters) +
                                  2 * p.first + g;
                    const uint32_t before = atomicAdd(c, 1u);
                    const bool last = before == (uint32_t)p.parts - 1;
                    if (last) *c = 0;
                    // no call leaves such a count: the workspace was not initialised
                    if (before >= (uint32_t)p.parts) atomicOr(status, SV_STATUS_OVERFLOW);
                    sh.last[g] = last;
                }
                meet(sh, &sh.group_sync[g], group_turn, lane, status);
                if (sh.last[g]) {
                    __threadfence();
                    // warps share the 32-row strips; a strip's warps share its columns
                    const int strips = (rows + 31) / 32;
                    const int per = strips == 1 ? 4 : strips == 2 ? 2 : 1;
                    const int strip = gw / per, share = gw % per;
                    const int wide = (c1 - c0) / per;
                    const int r = strip * 32 + lane;
                    auto slot_of = [&](int i) -> int { return (p.first + i) * 2 + (i == 0 ? 1 : 0); };
                    if (strip < strips) {
                        uint16_t *co = row_of(r);
                        // kBatch parts' loads in flight; a part past the last
                        // one is the last once more, with no weight.  (A part
                        // whose row saw nothing has the sum 0; a query of NaN
                        // leaves a sum of NaN and no reference.)
                        constexpr int kBatch = 8;
                        float top = -INFINITY, all = 0.f;
#pragma unroll 1
                        for (int i0 = 0; i0 < p.parts; i0 += kBatch) {
                            float2 x[kBatch];
#pragma unroll
                            for (int i = 0; i < kBatch; ++i)
                                x[i] = __ldcg(&part_stats[(slot_of(min(i0 + i, p.parts - 1)) * 2 + g) * kRows + r]);
                            float m = top;
#pragma unroll
                            for (int i = 0; i < kBatch; ++i) m = fmaxf(m, x[i].x);
                            all *= top == -INFINITY ? 0.f : ex2(top - m);
#pragma unroll
                            for (int i = 0; i < kBatch; ++i)
                                if (i0 + i < p.parts && x[i].y != 0.f) all += x[i].y * ex2(x[i].x - m);
                            top = m;
                        }
                        const float norm = all > 0.f ? 1.f / all : 0.f;
#pragma unroll 1
                        for (int cc = c0 + share * wide; cc < c0 + (share + 1) * wide; cc += 16) {
                            const int quads = min(4, (c0 + (share + 1) * wide - cc) / 4);
                            float4 v[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                            for (int i0 = 0; i0 < p.parts; i0 += kBatch / 2) {
                                float m[kBatch / 2];
                                float4 a[kBatch / 2][4];
#pragma unroll
                                for (int i = 0; i < kBatch / 2; ++i) {
                                    const int s = slot_of(min(i0 + i, p.parts - 1));
                                    m[i] = __ldcg(&part_stats[(s * 2 + g) * kRows + r]).x;
                                    const float4 *at = part_out +
                                                       ((int64_t)s * (kMaxHeadDim / 4) + cc / 4) * 256 +
                                                       part_row + r;
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (e < quads) a[i][e] = __ldcg(at + e * 256);
                                }
#pragma unroll
                                for (int i = 0; i < kBatch / 2; ++i) {
                                    const float f =
                                        i0 + i >= p.parts || m[i] == -INFINITY ? 0.f : ex2(m[i] - top);
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (e < quads) {
                                            v[e].x = fmaf(f, a[i][e].x, v[e].x);
                                            v[e].y = fmaf(f, a[i][e].y, v[e].y);
                                            v[e].z = fmaf(f, a[i][e].z, v[e].z);
                                            v[e].w = fmaf(f, a[i][e].w, v[e].w);
                                        }
                                }
                            }
                            if (r < rows) {
#pragma unroll
                                for (int e = 0; e < 4; e += 2)
                                    if (e < quads && cc + 4 * e < D) {
                                        uint4 y;
                                        y.x = pack2<T>(v[e].x * norm, v[e].y * norm);
                                        y.y = pack2<T>(v[e].z * norm, v[e].w * norm);
                                        y.z = pack2<T>(v[e + 1].x * norm, v[e + 1].y * norm);
                                        y.w = pack2<T>(v[e + 1].z * norm, v[e + 1].w * norm);
                                        if (all == 0.f) y = make_uint4(0, 0, 0, 0);
                                        *reinterpret_cast<uint4 *>(co + cc + 4 * e) = y;
                                    }
                            }
                        }
                    }
                }
            }
            // the joined states and accumulators have been read before the next
            // piece writes its own
            if (split) meet(sh, &sh.both_sync, both_turn, lane, status);
            reader.done(sh, lane);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 9) {
        __syncwarp();
        tc::tmem_free(tmem, kTmemCols);
    }
}

}  // namespace sv
