// cache.cu -- host side of the paged-cache calls (sv_append_kv,
// sv_paged_attention): argument checks and launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "specverify.h"
#include "sv_append.cuh"
#include "sv_attend.cuh"
#include "sv_cache_host.cuh"

namespace {

constexpr int kSms = 152;

using namespace svhost;

template <class T, int kVec>
int launch_append(sv::AppendParams &A, bool interleaved, unsigned grid, int per_block,
                  cudaStream_t st) {
    const int turned = A.rot_dim / 2 / kVec + (A.head_dim - A.rot_dim) / kVec;
    const int per_value = A.head_dim / kVec;
    // as many threads as share a token's items evenly (for 16 + 16 + 16 heads of
    // 64, half of it rotated: 67 us for 25400 tokens, 82 with 256 threads)
    const int items = (A.q_heads + A.kv_heads) * turned + A.kv_heads * per_value;
    const int rounds = (items + sv::kAppendThreads - 1) / sv::kAppendThreads;
    const int threads = std::max(32, ((items + rounds - 1) / rounds + 31) / 32 * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg,
                              interleaved ? sv::append_kernel<T, kVec, true>
                                          : sv::append_kernel<T, kVec, false>,
                              A, per_block) == cudaSuccess
               ? SV_OK
               : SV_ECUDA;
}

template <class T>
int launch_append(sv::AppendParams &A, bool interleaved, unsigned grid, int per_block,
                  cudaStream_t st) {
    // both halves of a rotated pair start on a pack: 16, 8 or 4 bytes
    const int half = A.rot_dim / 2;
    if (half % 8 == 0) return launch_append<T, 8>(A, interleaved, grid, per_block, st);
    if (half % 4 == 0) return launch_append<T, 4>(A, interleaved, grid, per_block, st);
    return launch_append<T, 2>(A, interleaved, grid, per_block, st);
}

// A map of one cache for boxes of 64 values x one head x `piece` slots of a
// page: [pages][slots][heads][values], whatever their order in memory.
// Values past head_dim and pages outside the cache read as zeros.
int box_map(CUtensorMap *map, const sv_paged_cache *c, void *base, const int64_t *stride,
            int piece) {
    const EncodeTiled encode = encoder();
    if (!encode) return SV_ECUDA;
    const cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->kv_heads,
                                (cuuint64_t)c->page_size, (cuuint64_t)c->num_pages};
    cuuint64_t bytes[3] = {(cuuint64_t)stride[2] * 2, (cuuint64_t)stride[1] * 2,
                           (cuuint64_t)stride[0] * 2};
    // the stride of an axis of length 1 means nothing: any valid one will do
    for (int i = 0; i < 3; ++i)
        if (dims[i + 1] == 1) bytes[i] = (cuuint64_t)c->head_dim * 2;
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)piece, 1}, step[4] = {1, 1, 1, 1};
    const CUresult r = encode(
        map, c->dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
        4, base, dims, bytes, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SV_OK : SV_EINVAL;
}

// A map of the queries for boxes of 64 values x the group's heads x the tokens
// that make 128 packed rows: [tokens][kv heads][group][values].
int query_map(CUtensorMap *map, const sv_paged_cache *c, const void *q, const int64_t *stride,
              int group) {
    const EncodeTiled encode = encoder();
    if (!encode) return SV_ECUDA;
    const cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)group, (cuuint64_t)c->kv_heads,
                                (cuuint64_t)c->tokens};
    cuuint64_t bytes[3] = {(cuuint64_t)stride[1] * 2, (cuuint64_t)stride[1] * 2 * group,
                           (cuuint64_t)stride[0] * 2};
    for (int i = 0; i < 3; ++i)
        if (dims[i + 1] == 1) bytes[i] = (cuuint64_t)c->head_dim * 2;
    const cuuint32_t box[4] = {64, (cuuint32_t)group, 1, (cuuint32_t)(sv::kRows / group)},
                     step[4] = {1, 1, 1, 1};
    const CUresult r = encode(
        map, c->dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
        4, const_cast<void *>(q), dims, bytes, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SV_OK : SV_EINVAL;
}

template <class T, int DP>
int launch_attend(const sv::AttendParams &A, const CUtensorMap &kmap, const CUtensorMap &vmap,
                  const CUtensorMap &qmap, cudaStream_t st) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SV_ECUDA;
    constexpr int bytes = sv::AttendSmem<DP>::kBytes;
    static std::atomic<int> raised[64];
    if (!raised[dev].load()) {
        if (cudaFuncSetAttribute(sv::attend_kernel<T, DP>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return SV_ECUDA;
        raised[dev].store(1);
    }
    const int sms = sm_count();
    if (sms <= 0) return SV_ECUDA;
    const unsigned grid = (unsigned)std::min(sms, sv::kAttendMaxCtas);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(sv::kAttendThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, sv::attend_kernel<T, DP>, A, kmap, vmap, qmap) != cudaSuccess)
        return SV_ECUDA;
    g_last_grid = grid;
    g_last_kernels = 1;
    return SV_OK;
}

}  // namespace

extern "C" {

size_t sv_cache_workspace_size(void) { return round_up(sv::kAttendWorkspace); }

int sv_append_kv(const sv_paged_cache *cache, const void *k, const int64_t *k_stride,
                 const void *v, const int64_t *v_stride, const void *q, const int64_t *q_stride,
                 void *q_out, const int64_t *q_out_stride, int32_t q_heads,
                 const double *inv_freq, int32_t rot_dim, int32_t interleaved,
                 const int32_t *positions, void *workspace, size_t workspace_bytes,
                 sv_stream_t stream) {
    sv::AppendParams A{};
    int rc = check_cache(cache);
    if (rc != SV_OK) return rc;
    if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 4 != 0 || (rot_dim > 0 && !inv_freq) ||
        q_heads < 0 || q_heads > (1 << 16) || cache->kv_heads > (1 << 16) ||
        (q == nullptr) != (q_heads == 0))
        return SV_EINVAL;
    if (cache->B == 0 || cache->tokens == 0) return SV_OK;
    if (!k || !v || !k_stride || !v_stride || !vec_ok(k, k_stride, 2) || !vec_ok(v, v_stride, 2))
        return SV_EINVAL;
    if (q && (!q_out || !q_stride || !q_out_stride || !vec_ok(q, q_stride, 2) ||
              !vec_ok(q_out, q_out_stride, 2)))
        return SV_EINVAL;
    const CurrentDevice here;
    if ((rc = bind_cache(here, cache, workspace, workspace_bytes, A.batch)) != SV_OK) return rc;
    if (!here.holds(k) || !here.holds(v) || (q && (!here.holds(q) || !here.holds(q_out))) ||
        !here.holds_or_null(inv_freq) || !here.holds_or_null(positions))
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
    // Tokens per block: one wave of eight blocks to an SM where that suffices.
    // (1536 tokens of 32 + 8 + 8 heads of 128: 11.8 us with two, 14.6 with one,
    // 13.7 with four; 25400 tokens of 16 + 16 + 16 heads of 64: 67 us with four,
    // 94 with one.)
    const int per_block = (int)std::min<int64_t>(
        sv::kAppendTokens, std::max<int64_t>(1, ((int64_t)cache->tokens + kSms * 8 - 1) / (kSms * 8)));
    const unsigned grid = (unsigned)((cache->tokens + per_block - 1) / per_block);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    rc = cache->dtype == SV_BF16
             ? launch_append<__nv_bfloat16>(A, interleaved != 0, grid, per_block, st)
             : launch_append<__half>(A, interleaved != 0, grid, per_block, st);
    if (rc != SV_OK) return rc;
    g_last_grid = grid;
    g_last_kernels = 1;
    return SV_OK;
}

int sv_paged_attention(const sv_paged_cache *cache, const void *q, const int64_t *q_stride,
                       void *out, const int64_t *out_stride, int32_t q_heads, float scale,
                       int32_t window, void *workspace, size_t workspace_bytes,
                       sv_stream_t stream) {
    sv::AttendParams A{};
    int rc = check_cache(cache);
    if (rc != SV_OK) return rc;
    if (q_heads < 1 || q_heads % cache->kv_heads != 0 || !std::isfinite(scale) || window < 0 ||
        (int64_t)cache->tokens * (q_heads / cache->kv_heads) > INT32_MAX - 1024)
        return SV_EINVAL;
    if (cache->B == 0 || cache->tokens == 0) return SV_OK;
    if (!q || !out || !q_stride || !out_stride || !vec_ok(q, q_stride, 2) ||
        !vec_ok(out, out_stride, 2))
        return SV_EINVAL;
    const CurrentDevice here;
    if ((rc = bind_cache(here, cache, workspace, workspace_bytes, A.batch)) != SV_OK) return rc;
    if (!here.holds(q) || !here.holds(out)) return SV_EINVAL;
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
    A.window = window < (int64_t)cache->max_pages * cache->page_size ? window : 0;
    A.piece = 8;
    while (A.piece < sv::kKeys && cache->page_size % (2 * A.piece) == 0) A.piece *= 2;
    A.scale_log2 = scale == 0.f ? 1.f : std::fabs(scale) * 1.44269504f;
    A.q_mode = scale == 0.f ? 2 : scale < 0.f ? 1 : 0;
    A.workspace = static_cast<char *>(workspace);
    CUtensorMap kmap, vmap;
    if ((rc = box_map(&kmap, cache, cache->k, cache->k_stride, A.piece)) != SV_OK) return rc;
    if ((rc = box_map(&vmap, cache, cache->v, cache->v_stride, A.piece)) != SV_OK) return rc;
    // Queries by TMA boxes of 128 packed rows when whole tokens make them up.
    // (Two prompts of 8192 tokens: 0.79 ms, 1.00 when threads load them; rounds
    // of 6 over 4096 slots 367 against 380 us.)
    A.q_boxes = A.q_mode == 0 && sv::kRows % A.group == 0;
    CUtensorMap qmap = kmap;  // unused otherwise
    if (A.q_boxes && (rc = query_map(&qmap, cache, q, q_stride, A.group)) != SV_OK) return rc;
    // (rows stored 32 bytes at a time: the prompts 0.79 ms, 0.86 by 16)
    A.wide_out = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 && out_stride[0] % 16 == 0 &&
                 out_stride[1] % 16 == 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = cache->dtype == SV_BF16;
    if (cache->head_dim > 64)
        return bf16 ? launch_attend<__nv_bfloat16, 128>(A, kmap, vmap, qmap, st)
                    : launch_attend<__half, 128>(A, kmap, vmap, qmap, st);
    return bf16 ? launch_attend<__nv_bfloat16, 64>(A, kmap, vmap, qmap, st)
                : launch_attend<__half, 64>(A, kmap, vmap, qmap, st);
}

}  // extern "C"
