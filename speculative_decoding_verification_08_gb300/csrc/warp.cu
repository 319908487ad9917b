// warp.cu -- host side of sv_warp_sample: argument checks and launch.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "specverify.h"
#include "sv_host.cuh"
#include "sv_warp.cuh"

namespace {

constexpr int kSms = 152;
constexpr int kThreads = 256;
// Slices of more than this many words (64 KB and one) leave room for two CTAs of an
// SM at most, and soon for one: 1024 threads then, not 256 (64 rows of 262144 fp32
// with top-p: 162 against 199 us).
constexpr int kSharedWords = 4096 + 1;
// 16-byte words of a slice that shared memory holds beside WarpShared
constexpr int kMaxWords = (227 * 1024 - (int)sizeof(sv::WarpShared)) / 16;

using svhost::kAlign;

int launch_clusters(void (*kernel)(sv::WarpParams), const sv::WarpParams &A, int c, int threads, size_t bytes,
                    cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(A.R * c));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, A) != cudaSuccess)
        return SV_ECUDA;
    svhost::g_last_grid = (int64_t)A.R * c;
    svhost::g_last_kernels = 1;
    return SV_OK;
}

template <class T>
int launch(sv::WarpParams &A, cudaStream_t st) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SV_ECUDA;
    const bool plain = !A.top_k && !A.top_p && !A.min_p;
    // Cluster: as many CTAs as keep a slice within 64 KB (three of them then
    // share an SM and hide one another's barriers: 256 rows of 128256 fp32 with
    // top-k 107 us, 141 with slices of 128 KB and one CTA to an SM; a slice of 64 KB
    // itself, with the word that alignment may take, is rounded up to one more round
    // of the block and leaves two: 131072 logits take 1.2 to 1.3 times as long as
    // 128256), and more
    // while the whole batch has fewer CTAs than SMs, down to 2048 elements each.
    // Rows without filters keep to the same rule (768 rows of 128256 bf16: 226,
    // 180, 167 and 181 us with 1, 2, 4 and 8 CTAs).
    const int64_t row = A.V * (int64_t)sizeof(T);
    int c = 1;
    while (c < sv::kWarpMaxCluster &&
           ((row + c - 1) / c > 65536 || ((int64_t)A.R * c * 2 <= kSms && A.V / (2 * c) >= 2048)))
        c *= 2;
    A.slice = (int32_t)(((A.V + c - 1) / c + 15) / 16 * 16);
    if ((int64_t)A.R * c > INT32_MAX) return SV_EINVAL;
    if (plain) return launch_clusters(sv::plain_kernel<T>, A, c, sv::kPlainThreads, 0, st);
    const int per_word = 16 / (int)sizeof(T);
    const bool wide = (int64_t)A.slice / per_word + 1 > kSharedWords;
    const int threads = wide ? 1024 : kThreads;
    // words of a slice (one more where rows do not start on one), in whole rounds
    // of the block
    const int64_t words = ((int64_t)A.slice / per_word + 1 + threads - 1) / threads * threads;
    const bool held = words <= kMaxWords;
    A.cached = (int32_t)std::min<int64_t>(words, kMaxWords);
    const size_t bytes = sizeof(sv::WarpShared) + (size_t)A.cached * 16;
    auto *kernel = !held ? sv::warp_kernel<T, false, 1024>
                   : wide ? sv::warp_kernel<T, true, 1024>
                          : sv::warp_kernel<T, true, kThreads>;
    static std::atomic<int> raised[64];
    if (!raised[dev].load()) {
        const int most = (int)(sizeof(sv::WarpShared) + (size_t)kMaxWords * 16);
        for (auto *k : {sv::warp_kernel<T, false, 1024>, sv::warp_kernel<T, true, 1024>,
                        sv::warp_kernel<T, true, kThreads>})
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
                return SV_ECUDA;
        raised[dev].store(1);
    }
    return launch_clusters(kernel, A, c, threads, bytes, st);
}

}  // namespace

extern "C" int sv_warp_sample(const void *z, int64_t z_row_stride, int32_t z_dtype, int32_t R,
                              int64_t V, const float *temperature, const int32_t *top_k,
                              const float *top_p, const float *min_p, const double *u,
                              int32_t *token, float *probs, int64_t probs_row_stride,
                              void *workspace, size_t workspace_bytes, sv_stream_t stream) {
    if (R < 0 || V < 1 || V > INT32_MAX ||
        (z_dtype != SV_F32 && z_dtype != SV_BF16 && z_dtype != SV_F16))
        return SV_EINVAL;
    if (R == 0) return SV_OK;
    if (!z || z_row_stride < V || (!token && !probs) || (token && !u) ||
        (probs && probs_row_stride < V))
        return SV_EINVAL;
    const svhost::CurrentDevice here;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
        workspace_bytes < sv_cache_workspace_size() || !here.holds(workspace))
        return SV_EWORKSPACE;
    for (const void *p : {z, (const void *)temperature, (const void *)top_k, (const void *)top_p, (const void *)min_p,
                          (const void *)u, (const void *)token, (const void *)probs})
        if (!here.holds_or_null(p)) return SV_EINVAL;
    sv::WarpParams A{};
    A.z = z;
    A.zs = z_row_stride;
    A.V = V;
    A.temperature = temperature;
    A.top_k = top_k;
    A.top_p = top_p;
    A.min_p = min_p;
    A.u = token ? u : nullptr;
    A.token = token;
    A.probs = probs;
    A.ps = probs_row_stride;
    A.status = static_cast<uint32_t *>(workspace);
    A.R = R;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    switch (z_dtype) {
        case SV_F32: return launch<float>(A, st);
        case SV_BF16: return launch<__nv_bfloat16>(A, st);
        default: return launch<__half>(A, st);
    }
}
