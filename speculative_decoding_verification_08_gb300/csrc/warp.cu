// warp.cu -- host side of sv_warp_sample: argument checks and launch.
#include <cuda_runtime.h>
#include <stdint.h>

#include "specverify.h"
#include "sv_host.cuh"
#include "sv_warp.cuh"

namespace {

using svhost::kAlign;
using svhost::kOnDevice;
using svhost::place;

bool on_device(const void *p) {
    const void *x = p;
    return place(x) == kOnDevice;  // true for null: optional arrays
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
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
        workspace_bytes < sv_cache_workspace_size() || !on_device(workspace))
        return SV_EWORKSPACE;
    if (!on_device(z) || !on_device(temperature) || !on_device(top_k) || !on_device(top_p) ||
        !on_device(min_p) || !on_device(u) || !on_device(token) || !on_device(probs))
        return SV_EINVAL;
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
        case SV_F32: sv::warp_kernel<float><<<R, sv::kWarpThreads, 0, st>>>(A); break;
        case SV_BF16: sv::warp_kernel<__nv_bfloat16><<<R, sv::kWarpThreads, 0, st>>>(A); break;
        default: sv::warp_kernel<__half><<<R, sv::kWarpThreads, 0, st>>>(A); break;
    }
    if (cudaGetLastError() != cudaSuccess) return SV_ECUDA;
    svhost::g_last_grid = R;
    svhost::g_last_kernels = 1;
    return SV_OK;
}
