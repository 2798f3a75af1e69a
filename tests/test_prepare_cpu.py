"""When an operator's kernels are prepared, without a GPU: the library's host
code linked with fakes of the CUDA calls and of the kernels' launches."""
from __future__ import annotations

import ctypes
import subprocess
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

import pytest

from split_bf16_gemm_swapped_gb300 import _build

OK, CUDA = 0, -5
P = 0x100000         # an aligned address: the fakes read no memory

KERNELS = r"""
#include <cuda.h>
#include <cuda_runtime.h>
#include <string.h>
#include "splitk_i8.cuh"
#include "splitk_internal.h"

// how often each was prepared or read, and whether it fails
extern "C" {
__attribute__((visibility("default"))) int prepared_i8, prepared_logprobs, read_i8, fail_i8, fail_logprobs, launches;
}

namespace splitk {
cudaError_t prepare_kernels(int) { return cudaSuccess; }
cudaError_t prepare_persistent(int) { return cudaSuccess; }
cudaError_t max_active_clusters_persistent(int, unsigned, size_t, int* n) { *n = 8; return cudaSuccess; }
cudaError_t launch_kernel(const LaunchArgs&, const CUtensorMap&, const KernelParams&, cudaStream_t) { ++launches; return cudaSuccess; }
cudaError_t launch_persistent(const LaunchArgs&, const CUtensorMap&, const KernelParams&, cudaStream_t) { ++launches; return cudaSuccess; }
cudaError_t launch_pdl_copy(const void*, void*, size_t, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_i8_stream(const I8Params&, int, cudaStream_t) { ++launches; return cudaSuccess; }
cudaError_t launch_i8_tile(const I8Params&, const I8Plan&, const I8Waits&, cudaStream_t) { ++launches; return cudaSuccess; }
cudaError_t read_and_clear_fault(int* w) { memset(w, 0, sizeof(int) * kFaultWords); return cudaSuccess; }
cudaError_t read_and_clear_fault_persistent(int* w) { memset(w, 0, sizeof(int) * kFaultWords); return cudaSuccess; }
cudaError_t read_and_clear_fault_i8(int* w) { ++read_i8; memset(w, 0, sizeof(int) * kFaultWords); return cudaSuccess; }
cudaError_t prepare_i8_tile(int, int (&clusters)[4]) {
  ++prepared_i8;
  if (fail_i8) return cudaErrorMemoryAllocation;
  clusters[0] = 76, clusters[1] = 36, clusters[2] = 22, clusters[3] = 16;
  return cudaSuccess;
}
cudaError_t prepare_logprobs(int (&clusters)[3]) {
  ++prepared_logprobs;
  if (fail_logprobs) return cudaErrorMemoryAllocation;
  clusters[0] = clusters[1] = clusters[2] = 16;
  return cudaSuccess;
}
}  // namespace splitk

// what splitk_logprobs() asks for
extern "C" __attribute__((visibility("default"))) int ask_logprobs() {
  splitk::DeviceSize d;
  return splitk::require_logprobs(&d);
}

"""

RUNTIME = r"""
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>

static CUresult encode(CUtensorMap* m, ...) { memset(m, 0, sizeof(*m)); return CUDA_SUCCESS; }

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3
     : a == cudaDevAttrMultiProcessorCount ? 152 : a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 232448 : 233472;
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
  *f = (void*)&encode;
  if (r) *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t n) { *p = malloc(n); return cudaSuccess; }
cudaError_t cudaMallocHost(void** p, size_t n) { *p = malloc(n); return cudaSuccess; }
cudaError_t cudaFree(void* p) { free(p); return cudaSuccess; }
cudaError_t cudaFreeHost(void* p) { free(p); return cudaSuccess; }
cudaError_t cudaMemcpy(void*, const void*, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaEventCreate(cudaEvent_t*) { return cudaSuccess; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventElapsedTime(float* ms, cudaEvent_t, cudaEvent_t) { *ms = 1.0f; return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void** p, const void*) { *p = (void*)0x1000; return cudaSuccess; }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void*) { memset(a, 0, sizeof(*a)); return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) { *s = cudaStreamCaptureStatusNone; return cudaSuccess; }
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
}
"""


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    where = tmp_path_factory.mktemp("fakes")
    (where / "kernels.cu").write_text(KERNELS)
    (where / "runtime.cpp").write_text(RUNTIME)
    nvcc = _build._nvcc()
    cuda = Path(nvcc).resolve().parent.parent / "include"
    common = [nvcc, *_build.ARCH_FLAGS, "-O1", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I", str(_build.INCLUDE), "-I", str(_build.CSRC), "-c"]
    jobs = [[*common, str(_build.CSRC / "splitk_host.cu"), "-o", str(where / "host.o")],
            [*common, str(_build.CSRC / "splitk_i8.cu"), "-o", str(where / "i8.o")],
            [*common, str(where / "kernels.cu"), "-o", str(where / "kernels.o")],
            ["g++", "-O1", "-std=c++17", "-fPIC", "-I", str(cuda), "-c", str(where / "runtime.cpp"), "-o",
             str(where / "runtime.o")]]
    with ThreadPoolExecutor() as pool:
        for res in pool.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs):
            assert res.returncode == 0, res.stderr[-3000:]
    # (its calls go to the fakes, whatever CUDA runtime the process holds)
    so = where / "libfake.so"
    res = subprocess.run(["g++", "-shared", "-o", str(so), *(str(where / f) for f in ("host.o", "i8.o", "kernels.o", "runtime.o")),
                          "-Wl,-z,defs,-Bsymbolic", "-lpthread"], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    return so


@pytest.fixture
def lib(library, tmp_path):
    """A copy of its own: nothing prepared yet."""
    import shutil
    so = shutil.copy(library, tmp_path / "fake.so")
    lib = ctypes.CDLL(str(so))
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.splitk_gemm_bf16.argtypes = [vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_gemm_i8.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_get_fault.argtypes = [vp]
    return lib


def count(lib, name):
    return ctypes.c_int.in_dll(lib, name)


def bf16(lib):
    return lib.splitk_gemm_bf16(P, P, P, 4, 256, 1024, 1, 0, None)


def i8(lib):
    return lib.splitk_gemm_i8(P, P, P, P, None, P, 0, 64, 1024, 1024, 1, None)


def test_the_bf16_product_prepares_its_own_kernels_alone(lib):
    assert bf16(lib) == OK and count(lib, "launches").value == 1
    assert lib.splitk_get_fault(None) == OK
    for name in ("prepared_i8", "prepared_logprobs", "read_i8"):
        assert count(lib, name).value == 0, name


def test_it_does_not_depend_on_the_other_operators(lib):
    count(lib, "fail_i8").value = count(lib, "fail_logprobs").value = 1
    assert bf16(lib) == OK
    assert i8(lib) == CUDA and lib.ask_logprobs() == CUDA
    assert bf16(lib) == OK
    # what failed is tried again
    count(lib, "fail_i8").value = count(lib, "fail_logprobs").value = 0
    assert i8(lib) == OK and lib.ask_logprobs() == OK


def test_operators_are_prepared_once_at_their_first_use(lib):
    for _ in range(3):
        assert i8(lib) == OK
    assert (count(lib, "prepared_i8").value, count(lib, "prepared_logprobs").value) == (1, 0)
    for _ in range(3):
        assert lib.ask_logprobs() == OK
    assert (count(lib, "prepared_i8").value, count(lib, "prepared_logprobs").value) == (1, 1)
    assert lib.splitk_get_fault(None) == OK and count(lib, "read_i8").value == 1
