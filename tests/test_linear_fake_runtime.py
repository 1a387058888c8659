"""The entry points of mlp_linear over a fake CUDA runtime with two devices, on the CPU: every entry leaves the caller's current
device as it was, every runtime call's error comes back as a status, and none is left with the runtime."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mlp_latency_gb300", "csrc")

DRIVER = r"""
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <cuda.h>
#include <cuda_runtime_api.h>
#include "mlp_block.h"

static int current, fail_at, calls, set_to, launches;
static cudaError_t last;
static bool restoring;
static const int *caller;
static cudaError_t call(cudaError_t e = cudaErrorUnknown)
{
    if (calls++ != fail_at)
        return cudaSuccess;
    return last = e;
}
static CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                       const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill)
{
    return CUDA_SUCCESS;
}
extern "C" {
void **__cudaRegisterFatBinary(void *) { static void *p; return &p; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
char __cudaInitModule(void **) { return 0; }
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
cudaError_t __cudaGetKernel(cudaKernel_t *, const void *) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void **, size_t, cudaStream_t) { return call(); }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
cudaError_t cudaGetLastError(void) { cudaError_t e = last; last = cudaSuccess; return e; }
cudaError_t cudaGetDevice(int *d) { *d = current; return call(); }
cudaError_t cudaSetDevice(int d)
{
    const bool back = set_to && d == *caller;
    if (d > 1)
        return last = cudaErrorInvalidDevice;
    if (call() != cudaSuccess) {
        restoring |= back;
        return last;
    }
    current = d;
    set_to = 1;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 152; return call(); }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return call(); }
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *) { *n = 152; return call(); }
cudaError_t cudaMalloc(void **p, size_t) { *p = reinterpret_cast<void *>(1 << 20); return call(cudaErrorMemoryAllocation); }
cudaError_t cudaFree(void *) { return call(); }
cudaError_t cudaMemset(void *, int, size_t) { return call(); }
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return call(); }
cudaError_t cudaMemcpyAsync(void *d, const void *, size_t n, cudaMemcpyKind, cudaStream_t) { std::memset(d, 1, n); return call(); }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return call(); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *, void **) { ++launches; return call(); }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **p, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *q)
{
    *p = reinterpret_cast<void *>(&encode);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
}

static int bad;
// One entry, called with its n-th runtime call failing, for every n that it reaches.
template <typename F>
static void every_failure(const char *what, int device, bool reports, F entry)
{
    for (int n = -1;; ++n) {
        current = device;
        caller = &device;
        calls = set_to = launches = 0;
        restoring = false;
        last = cudaSuccess;
        fail_at = n;
        const int status = entry();
        const bool failed = n >= 0 && n < calls;
        if (last != cudaSuccess || (!restoring && current != device) || (reports && (status != 0) != (failed && !restoring))) {
            std::printf("%s, device %d, call %d of %d fails: status %d, error left %d, device %d\n", what, device, n, calls, status, last, current);
            ++bad;
        }
        if (n >= calls)
            return;
    }
}

int main()
{
    void *const P = reinterpret_cast<void *>(1 << 20);
    int32_t *const off = static_cast<int32_t *>(P);
    mlp_linear_t h;
    mlp_linear_desc d = {512, 520, 0, 0, MLP_ACT_GELU_TANH, MLP_DT_BF16, MLP_DT_BF16, 0, 0};
    current = 1;
    fail_at = -1;
    d.device = 2;
    if (mlp_linear_create(&d, &h) != MLP_ERR_CUDA || current != 1 || last != cudaSuccess)
        std::printf("a device that does not exist\n"), ++bad;
    for (int device = 0; device < 2; ++device)
        for (int experts = 0; experts <= 4; experts += 4) {
            d.device = 0;
            d.experts = experts;
            const int32_t *o = experts ? off : nullptr;
            every_failure("create", device, true, [&] {
                const int s = mlp_linear_create(&d, &h);
                if (s == 0)
                    std::printf(h ? "" : "no handle\n");
                return s;
            });
            fail_at = -1;
            mlp_linear_create(&d, &h);
            for (int64_t rows : {0, 40, 3000}) {
                every_failure("forward", device, true, [&] { return mlp_linear_forward(h, rows, P, 512, P, P, P, 520, o, P, 520, P, 520, nullptr); });
                for (int what = 1; what < 8; ++what)
                    every_failure("backward", device, true, [&] {
                        return mlp_linear_backward(h, rows, P, 520, P, 512, P, P, 520, o, what & 1 ? P : nullptr, 512, what & 2 ? P : nullptr,
                                                   what & 4 ? P : nullptr, P, nullptr);
                    });
            }
            every_failure("check", device, false, [&] { return mlp_linear_check(h, nullptr); });
            every_failure("destroy", device, false, [&] {
                mlp_linear_t g = nullptr;
                const int keep = fail_at, before = current;
                fail_at = -1;
                mlp_linear_create(&d, &g);
                current = before;
                calls = set_to = 0;
                fail_at = keep;
                return mlp_linear_destroy(g);
            });
        }
    std::printf("%d wrong\n", bad);
    return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="no nvcc")
def test_entries_over_a_fake_runtime(tmp_path):
    include = os.path.join(ROOT, "include")
    common = ["nvcc", "-std=c++17", "-Xcicc", "-O0", "-gencode", "arch=compute_103a,code=compute_103a", "-I", include]
    driver = tmp_path / "driver.cpp"
    driver.write_text(DRIVER)
    subprocess.run([*common, "-c", "-o", str(tmp_path / "linear.o"), os.path.join(CSRC, "linear.cu")], check=True)
    subprocess.run([*common, "-c", "-o", str(tmp_path / "driver.o"), str(driver)], check=True)
    exe = str(tmp_path / "driver")
    subprocess.run(["g++", "-o", exe, str(tmp_path / "driver.o"), str(tmp_path / "linear.o")], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip().endswith("0 wrong"), run.stdout[-3000:]
