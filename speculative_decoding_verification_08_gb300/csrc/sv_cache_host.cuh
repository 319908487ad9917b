// sv_cache_host.cuh -- what the host sides of the paged-cache calls share:
// checks of a cache descriptor, the driver's tensor-map encoder, the SM count.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "specverify.h"
#include "sv_cache.cuh"
#include "sv_host.cuh"

namespace svhost {

// A base on 16 bytes and strides of whole 16-byte packs (`unit` elements).
inline bool vec_ok(const void *p, const int64_t *st, int n, int unit = 8) {
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return false;
    for (int i = 0; i < n; ++i)
        if (st[i] < 0 || st[i] % unit != 0) return false;
    return true;
}

// What can be told from the cache descriptor's values alone.  (eight: a cache of
// 8-bit values; a pack of 16 bytes then holds 16 of them.)
inline int check_cache(const sv_paged_cache *c, bool eight = false) {
    if (!c) return SV_EINVAL;
    const int unit = eight ? 16 : 8;
    if (c->B < 0 || c->tokens < 0 || c->kv_heads < 1 || c->head_dim < unit ||
        c->head_dim > sv::kMaxHeadDim || c->head_dim % unit != 0 || c->page_size < 8 ||
        c->page_size % 8 != 0 || c->num_pages < 1 || c->max_pages < 1 ||
        (eight ? c->dtype != SV_E4M3 : c->dtype != SV_BF16 && c->dtype != SV_F16))
        return SV_EINVAL;
    if ((int64_t)c->max_pages * c->page_size > (int64_t)INT32_MAX - 1024) return SV_EINVAL;
    if (c->B == 0 || c->tokens == 0) return SV_OK;
    if (!c->k || !c->v || !c->pages || !c->q_start || !c->kv_len || c->pages_stride < c->max_pages)
        return SV_EINVAL;
    return vec_ok(c->k, c->k_stride, 3, unit) && vec_ok(c->v, c->v_stride, 3, unit) ? SV_OK : SV_EINVAL;
}

// Checks where the workspace and the cache's arrays live, and fills in the
// batch the device sees.
inline int bind_cache(const CurrentDevice &here, const sv_paged_cache *c, void *ws, size_t ws_bytes, sv::Batch &b) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0 ||
        ws_bytes < sv_cache_workspace_size())
        return SV_EWORKSPACE;
    if (!here.holds(ws)) return SV_EWORKSPACE;
    if (!here.holds(c->k) || !here.holds(c->v) || !here.holds(c->pages) || !here.holds(c->q_start) ||
        !here.holds(c->kv_len))
        return SV_EINVAL;
    b.pages = c->pages;
    b.pages_stride = c->pages_stride;
    b.q_start = c->q_start;
    b.kv_len = c->kv_len;
    b.B = c->B;
    b.tokens = c->tokens;
    b.num_pages = c->num_pages;
    b.page_size = c->page_size;
    b.max_pages = c->max_pages;
    b.status = static_cast<uint32_t *>(ws);
    return SV_OK;
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (looked up once; the library does not link
// libcuda).
inline EncodeTiled encoder() {
    static const EncodeTiled f = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                             &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            fn = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(fn);
    }();
    return f;
}

// SM count of the current device, queried once.
inline int sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    static std::atomic<int> cached[64];
    int n = cached[dev].load();
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cached[dev].store(n);
    }
    return n;
}

}  // namespace svhost
