// cache8.cu -- host side of the calls on caches of 8-bit values and of the append
// with norms (sv_append_kv_normed, sv_read_kv, sv_paged_attention_scaled): argument
// checks and launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "specverify.h"
#include "sv_append8.cuh"
#include "sv_attend8.cuh"
#include "sv_cache_host.cuh"

namespace {

constexpr int kSms = 152;

using namespace svhost;

bool token_type(int32_t dtype) { return dtype == SV_BF16 || dtype == SV_F16; }

// A cache of 16-bit values of the tokens' type, or of 8-bit values with scales.
int check_either(const sv_paged_cache *c, const sv_cache_scales *s, int32_t dtype) {
    const int rc = check_cache(c, s != nullptr);
    if (rc != SV_OK) return rc;
    if (!token_type(dtype) || (!s && c->dtype != dtype)) return SV_EINVAL;
    if (!s || c->B == 0 || c->tokens == 0) return SV_OK;
    if (!s->k || !s->v) return SV_EINVAL;
    for (int i = 0; i < 3; ++i)
        if (s->k_stride[i] < 0 || s->v_stride[i] < 0) return SV_EINVAL;
    return SV_OK;
}

// Whether no two of a cache's vectors share a scale's byte by a stride of zero.
bool own_bytes(const sv_paged_cache *c, const sv_cache_scales *s) {
    const int32_t sizes[3] = {c->num_pages, c->page_size, c->kv_heads};
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && (s->k_stride[i] == 0 || s->v_stride[i] == 0)) return false;
    return true;
}

bool holds_scales(const CurrentDevice &here, const sv_cache_scales *s) {
    return !s || (here.holds(s->k) && here.holds(s->v));
}

sv::Scales device_scales(const sv_cache_scales *s) {
    sv::Scales d{};
    if (!s) return d;
    d.k = s->k;
    d.v = s->v;
    for (int i = 0; i < 3; ++i) {
        d.k_st[i] = s->k_stride[i];
        d.v_st[i] = s->v_stride[i];
    }
    return d;
}

template <class... P, class... A>
int launch(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return SV_ECUDA;
    g_last_grid = grid;
    g_last_kernels = 1;
    return SV_OK;
}

template <class T, bool kEight>
int launch_append(const sv::AppendNormParams &A, bool interleaved, cudaStream_t st) {
    const int rot = A.a.rot_dim;
    int lanes = 1;
    while (lanes * 16 < A.a.head_dim) lanes *= 2;
    const int tokens = A.a.batch.tokens;
    const int per_block = (int)std::min<int64_t>(
        sv::kNormTokens, std::max<int64_t>(1, ((int64_t)tokens + kSms * 4 - 1) / (kSms * 4)));
    const unsigned grid = (unsigned)((tokens + per_block - 1) / per_block);
    // as many warps as share a token's vectors evenly
    const int vectors = A.a.q_heads + 2 * A.a.kv_heads, per_warp = 32 / lanes;
    const int warps = (vectors + per_warp - 1) / per_warp;
    const int rounds = (warps + sv::kAppendThreads / 32 - 1) / (sv::kAppendThreads / 32);
    const int threads = (warps + rounds - 1) / rounds * 32;
    auto kernel = interleaved || rot == 0 ? sv::append_norm_kernel<T, kEight, sv::kAdjacentTurn>
                  : rot % 16 == 0         ? sv::append_norm_kernel<T, kEight, sv::kPackTurn>
                                          : sv::append_norm_kernel<T, kEight, sv::kPairTurn>;
    return launch(kernel, grid, threads, 0, st, A, per_block, lanes);
}

template <class T, bool kPages>
int launch_read(const sv::ReadParams &A, bool eight, int64_t rows, int per_block, cudaStream_t st) {
    const int64_t grid = (rows + per_block - 1) / per_block;
    if (grid > INT32_MAX) return SV_ETOOLARGE;
    auto kernel = eight ? sv::read_kernel<T, true, kPages> : sv::read_kernel<T, false, kPages>;
    return launch(kernel, (unsigned)grid, sv::kReadThreads, 0, st, A, per_block);
}

// The parameters of read_kernel that do not depend on where the rows go.
sv::ReadParams read_params(const sv_paged_cache *c, const sv_cache_scales *s) {
    sv::ReadParams A{};
    A.k_cache = c->k;
    A.v_cache = c->v;
    for (int i = 0; i < 3; ++i) {
        A.kc_st[i] = c->k_stride[i];
        A.vc_st[i] = c->v_stride[i];
    }
    A.scales = device_scales(s);
    A.kv_heads = c->kv_heads;
    A.head_dim = c->head_dim;
    A.chunks = (c->head_dim + 15) / 16;
    A.by_page.set((uint32_t)c->page_size);
    A.by_chunks.set((uint32_t)A.chunks);
    A.by_heads.set((uint32_t)c->kv_heads);
    return A;
}

// Room for the batch's sequences in 16 bits: keys and values, in pages of their own with
// a page table (page i of sequence b is page b * max_pages + i), or, where the cache has
// fewer pages than the table has entries, in its pages under their own numbers.
struct Scratch {
    bool own_pages;
    size_t half, table, bytes;
    explicit Scratch(const sv_paged_cache *c) {  // (can_read_back)
        const int64_t entries = (int64_t)c->B * c->max_pages;
        own_pages = entries <= c->num_pages;
        const size_t rows = (size_t)std::min<int64_t>(entries, c->num_pages) * c->page_size;
        half = round_up(rows * c->kv_heads * c->head_dim * 2);
        table = 2 * half;
        bytes = table + (own_pages ? round_up((size_t)entries * sizeof(int32_t)) : 0);
    }
};

// A map of one cache of codes for boxes of 128 values x one head x `piece` slots of
// a page: [pages][slots][heads][values], whatever their order in memory.  Values
// past head_dim and pages outside the cache read as zeros.
int code_map(CUtensorMap *map, const sv_paged_cache *c, void *base, const int64_t *stride, int piece) {
    const EncodeTiled encode = encoder();
    if (!encode) return SV_ECUDA;
    const cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->kv_heads, (cuuint64_t)c->page_size,
                                (cuuint64_t)c->num_pages};
    cuuint64_t bytes[3] = {(cuuint64_t)stride[2], (cuuint64_t)stride[1], (cuuint64_t)stride[0]};
    // the stride of an axis of length 1 means nothing: any valid one will do
    for (int i = 0; i < 3; ++i)
        if (dims[i + 1] == 1) bytes[i] = (cuuint64_t)c->head_dim;
    const cuuint32_t box[4] = {128, 1, (cuuint32_t)piece, 1}, step[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, bytes, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SV_OK : SV_EINVAL;
}

template <class T, int kRows>
int launch_attend8(const sv::Attend8Params &A, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SV_ECUDA;
    constexpr int bytes = sv::Attend8Smem<T, kRows>::kBytes;
    static std::atomic<int> raised[64];
    if (!raised[dev].load()) {
        if (cudaFuncSetAttribute(sv::attend8_kernel<T, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
            cudaSuccess)
            return SV_ECUDA;
        raised[dev].store(1);
    }
    const int sms = sm_count();
    if (sms <= 0) return SV_ECUDA;
    const unsigned grid = (unsigned)std::min(sms, sv::kAttendMaxCtas);
    return launch(sv::attend8_kernel<T, kRows>, grid, sv::kThreads8, bytes, st, A, kmap, vmap);
}

// Up to so many packed rows of a sequence and kv head attention goes over the codes
// directly, above it (and with room for it) the sequences are read back to 16 bits
// first.  32 sequences of 4096 slots, 32 heads over 8 of 128, bf16: 89 against 252 us
// for 8 tokens each (32 rows), 253 against 259 for 32, 304 against 272 for 40, 881
// against 379 for 128; 4 of 32768: 225 against 259 for 32, 279 against 270 for 40.
//
// The rule and the tiles' width go by the batch's average (the lengths are known on the
// device alone), which suits sequences with like numbers of new tokens.  One long one
// among short ones fares badly: a chunk of 2048 tokens over 4096 slots takes 113 us,
// 127 single tokens over 512 to 4096 slots 124, both in one call 552; a chunk of 4096 and
// 255 single tokens 145, 230 and 1243 (over the codes, in narrow tiles); with 62 single
// tokens beside the chunk of 2048 the whole batch is read back, 379 for 113 and 65.  Calls
// of their own for the long ones and for the short ones take the sum.
constexpr int64_t kDirectRows = 128;
// Reading back looks at every slot of the page table (a block for 16 of them, most of
// which end at once where sequences are short): not past a table whose slots would be so
// many bytes in 16 bits.
constexpr size_t kMaxTable = (size_t)16 << 30;
constexpr int32_t kMaxReadHeads = 1 << 16;  // (a block's items are numbered by 32 bits)

// Whether the sequences may be read back.
bool can_read_back(const sv_paged_cache *c) {
    const unsigned __int128 slots = (unsigned __int128)c->B * c->max_pages * c->page_size;
    return c->kv_heads <= kMaxReadHeads && slots * c->kv_heads * c->head_dim * 4 <= kMaxTable;
}

// Packed rows of a sequence and kv head, on average and rounded up.
int64_t average_rows(const sv_paged_cache *c, int32_t q_heads) {
    return ((int64_t)c->tokens * (q_heads / c->kv_heads) + c->B - 1) / c->B;
}

template <class T>
int launch_attend8(const sv::Attend8Params &A, int64_t rows, const CUtensorMap &kmap, const CUtensorMap &vmap,
                   cudaStream_t st) {
    // as few tiles as hold them, and as few columns to a tile
    const int64_t tiles = (rows + sv::kMaxRows8 - 1) / sv::kMaxRows8;
    rows = (rows + tiles - 1) / tiles;
    if (rows <= 8) return launch_attend8<T, 8>(A, kmap, vmap, st);
    if (rows <= 16) return launch_attend8<T, 16>(A, kmap, vmap, st);
    if (rows <= 24) return launch_attend8<T, 24>(A, kmap, vmap, st);
    return launch_attend8<T, 32>(A, kmap, vmap, st);
}

}  // namespace

extern "C" {

int sv_append_kv_normed(const sv_paged_cache *cache, const sv_cache_scales *scales, int32_t dtype,
                        const void *k, const int64_t *k_stride, const void *v, const int64_t *v_stride,
                        const void *q, const int64_t *q_stride, void *q_out, const int64_t *q_out_stride,
                        int32_t q_heads, const void *q_norm, const void *k_norm, int32_t norm_dtype, float eps,
                        const double *inv_freq, int32_t rot_dim, int32_t interleaved, const int32_t *positions,
                        void *workspace, size_t workspace_bytes, sv_stream_t stream) {
    sv::AppendNormParams P{};
    int rc = check_either(cache, scales, dtype);
    if (rc != SV_OK) return rc;
    if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 4 != 0 || (rot_dim > 0 && !inv_freq) ||
        q_heads < 0 || q_heads > (1 << 16) || cache->kv_heads > (1 << 16))
        return SV_EINVAL;
    if ((q_norm || k_norm) &&
        ((norm_dtype != SV_F32 && norm_dtype != dtype) || !(eps >= 0.f) || !std::isfinite(eps)))
        return SV_EINVAL;
    if (cache->B == 0 || cache->tokens == 0) return SV_OK;
    if ((q == nullptr) != (q_heads == 0) || (q_norm && !q)) return SV_EINVAL;
    if (!k || !v || !k_stride || !v_stride || !vec_ok(k, k_stride, 2) || !vec_ok(v, v_stride, 2))
        return SV_EINVAL;
    if (q && (!q_out || !q_stride || !q_out_stride || !vec_ok(q, q_stride, 2) ||
              !vec_ok(q_out, q_out_stride, 2)))
        return SV_EINVAL;
    if (scales && !own_bytes(cache, scales)) return SV_EINVAL;
    const CurrentDevice here;
    sv::AppendParams &A = P.a;
    if ((rc = bind_cache(here, cache, workspace, workspace_bytes, A.batch)) != SV_OK) return rc;
    if (!here.holds(k) || !here.holds(v) || (q && (!here.holds(q) || !here.holds(q_out))) ||
        !here.holds_or_null(inv_freq) || !here.holds_or_null(positions) || !here.holds_or_null(q_norm) ||
        !here.holds_or_null(k_norm) || !holds_scales(here, scales))
        return SV_EINVAL;
    A.k = k;
    A.v = v;
    A.q = q;
    A.q_out = q_out;
    A.k_cache = cache->k;
    A.v_cache = cache->v;
    for (int i = 0; i < 2; ++i) {
        A.k_st[i] = k_stride[i];
        A.v_st[i] = v_stride[i];
        if (q) {
            A.q_st[i] = q_stride[i];
            A.o_st[i] = q_out_stride[i];
        }
    }
    for (int i = 0; i < 3; ++i) {
        A.kc_st[i] = cache->k_stride[i];
        A.vc_st[i] = cache->v_stride[i];
    }
    A.inv_freq = inv_freq;
    A.by_page.set((uint32_t)cache->page_size);
    A.positions = positions;
    A.q_heads = q_heads;
    A.kv_heads = cache->kv_heads;
    A.head_dim = cache->head_dim;
    A.rot_dim = rot_dim;
    P.scales = device_scales(scales);
    P.q_norm = q_norm;
    P.k_norm = k_norm;
    P.norm_f32 = norm_dtype == SV_F32;
    P.eps = eps;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool turn = interleaved != 0;
    if (dtype == SV_BF16)
        return scales ? launch_append<__nv_bfloat16, true>(P, turn, st) : launch_append<__nv_bfloat16, false>(P, turn, st);
    return scales ? launch_append<__half, true>(P, turn, st) : launch_append<__half, false>(P, turn, st);
}

int sv_read_kv(const sv_paged_cache *cache, const sv_cache_scales *scales, int32_t dtype, void *k_out,
               const int64_t *k_out_stride, void *v_out, const int64_t *v_out_stride, void *workspace,
               size_t workspace_bytes, sv_stream_t stream) {
    int rc = check_either(cache, scales, dtype);
    if (rc != SV_OK) return rc;
    if (cache->kv_heads > kMaxReadHeads) return SV_EINVAL;
    if (cache->B == 0 || cache->tokens == 0) return SV_OK;
    if (!k_out || !v_out || !k_out_stride || !v_out_stride || !vec_ok(k_out, k_out_stride, 2) ||
        !vec_ok(v_out, v_out_stride, 2))
        return SV_EINVAL;
    const CurrentDevice here;
    sv::ReadParams A = read_params(cache, scales);
    if ((rc = bind_cache(here, cache, workspace, workspace_bytes, A.batch)) != SV_OK) return rc;
    if (!here.holds(k_out) || !here.holds(v_out) || !holds_scales(here, scales)) return SV_EINVAL;
    A.k = k_out;
    A.v = v_out;
    for (int i = 0; i < 2; ++i) {
        A.k_st[i] = k_out_stride[i];
        A.v_st[i] = v_out_stride[i];
    }
    const int per_block = (int)std::min<int64_t>(
        sv::kReadRows, std::max<int64_t>(1, ((int64_t)cache->tokens + kSms * 4 - 1) / (kSms * 4)));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == SV_BF16 ? launch_read<__nv_bfloat16, false>(A, scales != nullptr, cache->tokens, per_block, st)
                            : launch_read<__half, false>(A, scales != nullptr, cache->tokens, per_block, st);
}

size_t sv_paged_attention_scratch_size(const sv_paged_cache *cache, int32_t q_heads) {
    if (check_cache(cache, true) != SV_OK || q_heads < 1 || cache->B == 0 || cache->tokens == 0) return 0;
    if (q_heads % cache->kv_heads != 0 || average_rows(cache, q_heads) <= kDirectRows) return 0;
    return can_read_back(cache) ? Scratch(cache).bytes : 0;
}

int sv_paged_attention_scaled(const sv_paged_cache *cache, const sv_cache_scales *scales, int32_t dtype,
                        const void *q, const int64_t *q_stride, void *out, const int64_t *out_stride,
                        int32_t q_heads, float scale, int32_t window, void *scratch, size_t scratch_bytes,
                        void *workspace, size_t workspace_bytes, sv_stream_t stream) {
    int rc = check_cache(cache, true);
    if (rc != SV_OK) return rc;
    if (!scales) return SV_EINVAL;
    if ((rc = check_either(cache, scales, dtype)) != SV_OK) return rc;
    if (q_heads < 1 || q_heads % cache->kv_heads != 0 || !std::isfinite(scale) || window < 0 ||
        (int64_t)cache->tokens * (q_heads / cache->kv_heads) > INT32_MAX - 1024)
        return SV_EINVAL;
    if (cache->B == 0 || cache->tokens == 0) return SV_OK;
    if (!q || !out || !q_stride || !out_stride || !vec_ok(q, q_stride, 2) || !vec_ok(out, out_stride, 2))
        return SV_EINVAL;
    if (scratch && !can_read_back(cache)) return SV_EINVAL;
    const CurrentDevice here;
    sv::Batch batch{};
    if ((rc = bind_cache(here, cache, workspace, workspace_bytes, batch)) != SV_OK) return rc;
    if (!here.holds(q) || !here.holds(out) || !holds_scales(here, scales)) return SV_EINVAL;
    if (window >= (int64_t)cache->max_pages * cache->page_size) window = 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!scratch) {
        sv::Attend8Params P{};
        sv::AttendParams &A = P.a;
        A.batch = batch;
        A.q = q;
        A.out = out;
        for (int i = 0; i < 2; ++i) {
            A.q_st[i] = q_stride[i];
            A.o_st[i] = out_stride[i];
        }
        A.q_heads = q_heads;
        A.kv_heads = cache->kv_heads;
        A.group = q_heads / cache->kv_heads;
        A.by_group.set((uint32_t)A.group);
        A.by_page.set((uint32_t)cache->page_size);
        A.head_dim = cache->head_dim;
        A.window = window;
        A.piece = 8;
        while (A.piece < sv::kKeys && cache->page_size % (2 * A.piece) == 0) A.piece *= 2;
        A.q_mode = scale == 0.f ? 2 : scale < 0.f ? 1 : 0;
        A.workspace = static_cast<char *>(workspace);
        P.scales = device_scales(scales);
        P.scale_part = scale == 0.f ? 1.f
                                    : (float)std::frexp(std::fabs((double)scale) * 1.4426950408889634, &P.scale_exponent);
        CUtensorMap kmap, vmap;
        if ((rc = code_map(&kmap, cache, cache->k, cache->k_stride, A.piece)) != SV_OK) return rc;
        if ((rc = code_map(&vmap, cache, cache->v, cache->v_stride, A.piece)) != SV_OK) return rc;
        const int64_t rows = average_rows(cache, q_heads);
        return dtype == SV_BF16 ? launch_attend8<__nv_bfloat16>(P, rows, kmap, vmap, st)
                                : launch_attend8<__half>(P, rows, kmap, vmap, st);
    }
    // many rows: the sequences back to 16 bits, and the attention over those
    const Scratch room(cache);
    if (scratch_bytes < room.bytes || (reinterpret_cast<uintptr_t>(scratch) % kAlign) != 0 || !here.holds(scratch))
        return SV_EWORKSPACE;
    sv::ReadParams A = read_params(cache, scales);
    A.batch = batch;
    char *base = static_cast<char *>(scratch);
    A.k = base;
    A.v = base + room.half;
    A.table = room.own_pages ? reinterpret_cast<int32_t *>(base + room.table) : nullptr;
    A.window = window;
    for (int64_t *s : {A.k_st, A.v_st}) {
        s[0] = (int64_t)cache->kv_heads * cache->head_dim;
        s[1] = cache->head_dim;
    }
    const int64_t rows = (int64_t)cache->B * cache->max_pages * cache->page_size;
    const int per_block = cache->page_size % 16 == 0 ? 16 : 8;
    rc = dtype == SV_BF16 ? launch_read<__nv_bfloat16, true>(A, true, rows, per_block, st)
                          : launch_read<__half, true>(A, true, rows, per_block, st);
    if (rc != SV_OK) return rc;
    sv_paged_cache plain = *cache;
    plain.k = A.k;
    plain.v = A.v;
    plain.dtype = dtype;
    for (int64_t *s : {plain.k_stride, plain.v_stride}) {
        s[0] = (int64_t)cache->page_size * cache->kv_heads * cache->head_dim;
        s[1] = (int64_t)cache->kv_heads * cache->head_dim;
        s[2] = cache->head_dim;
    }
    if (room.own_pages) {
        plain.num_pages = cache->B * cache->max_pages;
        plain.pages = A.table;
        plain.pages_stride = cache->max_pages;
    }
    rc = sv_paged_attention(&plain, q, q_stride, out, out_stride, q_heads, scale, window, workspace,
                            workspace_bytes, stream);
    if (rc == SV_OK) g_last_kernels = 2;
    return rc;
}

}  // extern "C"
