"""What the library remembers per device, with a fake of the runtime (CPU only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "device_state.h"
#include <cstdio>
#include <thread>
static int device, calls, lookups, limit[100];
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int v) {
    ++calls;
    if (answer == cudaSuccess) limit[device] = v;
    return answer;
}
extern "C" cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int d) { ++lookups; *v = 100 + d; return cudaSuccess; }
static void kernel(int) {}
static void other(int) {}
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
    using sga::allow_smem;
    CHECK(allow_smem<kernel>(48 * 1024) == cudaSuccess && calls == 0);
    CHECK(allow_smem<kernel>(100000) == cudaSuccess && limit[0] == 100000);
    CHECK(allow_smem<kernel>(60000) == cudaSuccess && calls == 1 && limit[0] == 100000);
    device = 1;   // a limit is a device's own
    CHECK(allow_smem<kernel>(60000) == cudaSuccess && limit[1] == 60000);
    CHECK(allow_smem<kernel>(90000) == cudaSuccess && limit[1] == 90000 && calls == 3);
    CHECK(allow_smem<other>(60000) == cudaSuccess && calls == 4);   // and a kernel's
    device = 0;
    CHECK(allow_smem<kernel>(100000) == cudaSuccess && calls == 4);
    answer = cudaErrorInvalidValue;   // a refusal is not remembered
    CHECK(allow_smem<kernel>(300000) == cudaErrorInvalidValue && calls == 5);
    answer = cudaSuccess;
    CHECK(allow_smem<kernel>(200000) == cudaSuccess && calls == 6 && limit[0] == 200000);
    device = sga::kMaxDevices;   // past what is remembered: told every time
    CHECK(allow_smem<kernel>(60000) == cudaSuccess && allow_smem<kernel>(60000) == cudaSuccess && calls == 8);
    device = 0;
    CHECK(sga::device_sms() == 100 && sga::device_sms() == 100 && lookups == 1);
    device = 2;
    CHECK(sga::device_sms() == 102 && lookups == 2);
    return 0;
}
"""


def test_limits_and_sizes_belong_to_a_device(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if not os.path.exists(os.path.join(include, "cuda_runtime_api.h")) or not shutil.which("g++"):
        pytest.skip("no host compiler or CUDA headers")
    src, exe = tmp_path / "state.cpp", tmp_path / "state"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++20", "-O1", "-I", os.path.join(ROOT, "sparse_graph_attention_csr_gb300", "csrc"), "-isystem", include,
                    str(src), "-o", str(exe), "-pthread"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
