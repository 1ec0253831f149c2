"""A kernel's attributes are set once on every device it is launched on (csrc/ops.h), checked on the host with a current device of its
own."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = next((p for p in (os.environ.get("CUDA_HOME"), "/usr/local/cuda") if p and os.path.exists(os.path.join(p, "include"))), None)

SOURCE = r"""
#include <cstdio>
#include "ops.h"

static int current = 0;
static cudaError_t fails = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* device) {
    *device = current;
    return fails;
}

static int calls[moe::kMaxDevices];
static cudaError_t prepare(int* device) {
    return moe::once_per_device(device, [](int d) {
        ++calls[d];
        return d == 3 ? cudaErrorInvalidValue : cudaSuccess;
    });
}
static cudaError_t other(int* device) {
    return moe::once_per_device(device, [](int) { return cudaErrorUnknown; });
}

#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
    const int order[] = {0, 0, 1, 3, 0, 1, 3, 2};
    for (int d : order) {
        int device = -1;
        current = d;
        CHECK(prepare(&device) == (d == 3 ? cudaErrorInvalidValue : cudaSuccess));
        CHECK(device == d);
    }
    for (int d = 0; d < 4; ++d) CHECK(calls[d] == 1);
    int device = 0;
    current = 0;
    CHECK(other(&device) == cudaErrorUnknown);
    current = moe::kMaxDevices;
    CHECK(prepare(&device) == cudaErrorInvalidDevice);
    current = 0;
    fails = cudaErrorNoDevice;
    CHECK(prepare(&device) == cudaErrorNoDevice);
    return 0;
}
"""


def test_attributes_are_set_once_on_each_device(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or CUDA is None:
        pytest.skip("no C++ compiler or CUDA headers")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(SOURCE)
    cc = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-pthread", "-I", os.path.join(ROOT, "include"), "-I",
                         os.path.join(ROOT, "moe_expert_ffn_topk_gb300", "csrc"), "-I", os.path.join(CUDA, "include"), str(src), "-o",
                         str(exe)], capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout


@pytest.mark.parametrize("name", ["moe_layer.cuh", "fp8_matmul.cu"])
def test_kernels_of_moe_ops_use_it(name):
    src = open(os.path.join(ROOT, "moe_expert_ffn_topk_gb300", "csrc", name)).read()
    assert "once_per_device(" in src and "std::once_flag" not in src
