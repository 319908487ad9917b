"""The pointer check of the target pass's calls, against a stand-in for the CUDA
runtime that knows two devices (host code only: compiled and run without one)."""
import os
import shutil
import subprocess

import pytest

import speculative_decoding_verification_08_gb300 as sv
from speculative_decoding_verification_08_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include "sv_host.cuh"

static int g_current = 0, g_errors = 0;
thread_local int64_t svhost::g_last_grid = 0;
thread_local int32_t svhost::g_last_kernels = 0;

// addresses 0x1000.. lie on device 0, 0x2000.. on 1, 0x3000.. are managed by 1,
// 0x4000.. page-locked, 0x5000.. pageable; the rest is refused
cudaError_t fake_device(int *d) {
    *d = g_current < 0 ? 0 : g_current;
    return g_current < 0 ? cudaErrorNoDevice : cudaSuccess;
}
cudaError_t fake_attributes(cudaPointerAttributes *a, const void *p) {
    switch (reinterpret_cast<uintptr_t>(p) >> 12) {
        case 1: a->type = cudaMemoryTypeDevice; a->device = 0; return cudaSuccess;
        case 2: a->type = cudaMemoryTypeDevice; a->device = 1; return cudaSuccess;
        case 3: a->type = cudaMemoryTypeManaged; a->device = 1; return cudaSuccess;
        case 4: a->type = cudaMemoryTypeHost; a->device = 0; return cudaSuccess;
        case 5: a->type = cudaMemoryTypeUnregistered; a->device = 0; return cudaSuccess;
    }
    return cudaErrorInvalidValue;
}
extern "C" {
cudaError_t CUDARTAPI cudaGetDevice(int *d) { return fake_device(d); }
cudaError_t CUDARTAPI cudaPointerGetAttributes(cudaPointerAttributes *a, const void *p) { return fake_attributes(a, p); }
cudaError_t CUDARTAPI cudaGetLastError(void) { ++g_errors; return cudaSuccess; }
}

int main() {
    for (g_current = -1; g_current < 2; ++g_current) {
        const svhost::CurrentDevice here;
        for (uintptr_t p = 0; p < 7; ++p)
            std::printf("%d", (int)here.holds(reinterpret_cast<const void *>(p << 12)));
        std::printf("%d ", (int)here.holds_or_null(nullptr));
    }
    std::printf("%d\n", g_errors);
}
"""


def test_only_memory_of_the_current_device_is_taken(tmp_path):
    cxx = os.environ.get("CXX", "g++")
    if not shutil.which(cxx):
        pytest.skip("no host compiler")
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    subprocess.run([cxx, "-std=c++17", "-I", _build.CSRC, "-I", _build.INCLUDE, "-I", cuda, str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    # null, device 0, device 1, managed, page-locked, pageable, unknown; null where that is allowed
    assert out == ["00000001", "01010001", "00110001", "3"]


def test_a_workspace_is_not_made_off_the_gpu():
    sv.build()
    for make in (sv.CacheWorkspace, sv.cache_workspace):
        with pytest.raises(sv.SpecVerifyError, match="CUDA device"):
            make("cpu")
