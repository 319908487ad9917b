// sv_host.cuh -- what the host sides of the library's translation units share:
// workspace alignment, where a caller's pointer lives, dependent launches, and
// the launch counters behind sv_last_grid_size and sv_last_kernel_count.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "specverify.h"

namespace svhost {

constexpr size_t kAlign = 256;

inline size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

extern thread_local int64_t g_last_grid;
extern thread_local int32_t g_last_kernels;

// Launches kernel on stream st as a programmatic dependent of the previous
// launch: it may be scheduled while that grid's CTAs retire and waits on the
// device (griddepcontrol.wait) before it reads their results.
template <class Kernel, class Args>
int launch_dependent(Kernel kernel, unsigned grid, unsigned threads, size_t smem,
                     const Args &P, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? SV_OK : SV_ECUDA;
}

// Where a pointer lives, as the runtime knows it: device (or managed) memory,
// page-locked host memory the GPU reads over the host link, or neither
// (pageable host memory, which the kernels must not be given).
enum Residence { kOnDevice = 0, kOnHost = 1, kUnusable = 2 };

template <class T>
Residence place(T *&ptr) {
    if (!ptr) return kOnDevice;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
        cudaGetLastError();
        return kUnusable;
    }
    if (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged) return kOnDevice;
    if (a.type != cudaMemoryTypeHost || !a.devicePointer) return kUnusable;
    // the address the device uses for this page-locked block
    const char *base = static_cast<const char *>(a.hostPointer);
    const ptrdiff_t off = reinterpret_cast<const char *>(ptr) - base;
    ptr = reinterpret_cast<T *>(static_cast<char *>(a.devicePointer) + off);
    return kOnHost;
}

// The device that this thread's launches go to.  A kernel there is handed memory
// of that device (or managed memory, which is every device's) and no other's.
struct CurrentDevice {
    int id = -1;
    CurrentDevice() {
        if (cudaGetDevice(&id) != cudaSuccess) {
            cudaGetLastError();
            id = -1;
        }
    }
    bool holds(const void *p) const {
        if (!p || id < 0) return false;
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        return a.type == cudaMemoryTypeManaged || (a.type == cudaMemoryTypeDevice && a.device == id);
    }
    bool holds_or_null(const void *p) const { return !p || holds(p); }
};

}  // namespace svhost
