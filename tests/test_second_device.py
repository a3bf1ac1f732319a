"""Kernels with more than 48 KB of dynamic shared memory need an attribute that
belongs to one device. Without a GPU: the library's CUDA runtime calls are
answered by a stand-in (loaded in front of the real runtime in a process of its
own) that refuses a launch whose attribute the current device has not been given,
as the runtime does. A second device of the same process has to get its own."""
import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest

from nvfp4_w4a4_moe_permute_gb300 import build as B

RUNTIME = r"""
#include <cuda.h>
#include <cuda_runtime.h>
#include <map>
#include <utility>
static int device = 0, launches = 0;
static std::map<std::pair<int, const void*>, size_t> allowed;
static CUresult encode(...) { return CUDA_SUCCESS; }
static cudaError_t launch(const void* kernel, size_t smem) {
  if (smem > 48 * 1024 && allowed[{device, kernel}] < smem) return cudaErrorInvalidValue;
  ++launches;
  return cudaSuccess;
}
extern "C" {
void standin_set_device(int d) { device = d; }
int standin_launches() { return launches; }
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int n) {
  allowed[{device, f}] = n;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  *n = 76;
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *f = reinterpret_cast<void*>(&encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  return launch(f, c->dynamicSmemBytes);
}
cudaError_t __cudaLaunchKernel(cudaKernel_t f, dim3, dim3, void**, size_t smem, cudaStream_t) {
  return launch(reinterpret_cast<const void*>(f), smem);
}
}
"""

P = 1 << 20   # an address that nothing reads


def steps(lib):
    """Calls whose kernels need the attribute, each on a device that is new to it."""
    from nvfp4_w4a4_moe_permute_gb300 import minite as M
    t = np.zeros(1, dtype=M.ADAMW_TENSOR)
    for k in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        t[k] = P
    t["n"] = 1000
    for dtype in (0, 1):
        yield "forward", lambda: lib.minite_grouped_gemm_bf16(P, 64, P, 0, P, 16, 64, 64, 4, P, 64, dtype, None, None)
        yield "activation gradient", lambda: lib.minite_grouped_gemm_bf16(P, 64, P, 1, P, 16, 64, 64, 4, P, 64, dtype, None, None)
        yield "weight gradient", lambda: lib.minite_grouped_wgrad_bf16(P, 64, P, 64, P, 16, 64, 64, 4, P, dtype, 0, None, None)
    for n in (1, 100):
        many = np.repeat(t, n)
        yield f"AdamW of {n}", lambda: lib.minite_adamw_step(many.ctypes.data, n, 1, 1, 8, 1e-3, 0.9, 0.95, 1e-8, 0.0, 1, None, None)
    for variant in (0, 1, 2):
        lib.minite_set_gemm_variant(variant)
        yield f"NVFP4 product {variant}", lambda: lib.minite_grouped_gemm_nvfp4(P, P, P, P, P, P, P, P, 256, 256, 256, 4, P, 0, None, None)
    lib.minite_set_gemm_variant(0)
    yield "both orientations", lambda: lib.minite_quantize_nvfp4_dual(P, 2, 256, 256, P, P, P, P, P, P, 1 << 20, None, None)


def child():
    from nvfp4_w4a4_moe_permute_gb300 import minite as M
    lib, runtime = M.load(), ctypes.CDLL(os.environ["LD_PRELOAD"])
    for what, call in steps(lib):
        for device in (0, 1, 0, 5):
            runtime.standin_set_device(device)
            before = runtime.standin_launches()
            rc = call()
            assert rc == 0 and runtime.standin_launches() > before, f"{what} on device {device}: status {rc}"
    print("every call went through")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_device_gets_its_shared_memory(tmp_path):
    B.build()
    src, lib = tmp_path / "runtime.cpp", tmp_path / "runtime.so"
    src.write_text(RUNTIME)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc_path()))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", include, str(src), "-o", str(lib)], check=True)
    env = {**os.environ, "LD_PRELOAD": str(lib), "PYTHONPATH": B.ROOT}
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, cwd=B.ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "every call went through" in r.stdout, r.stdout + r.stderr[-2000:]


if __name__ == "__main__":
    child()
