"""The shared-memory limit of a kernel is set on each device that launches it, once, and again after a failure: the host code
compiled against a stand-in for the CUDA runtime (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "smem_limit.h"
#include <cstdio>
static int device = 0, calls[64], failing = 0;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute a, int bytes) {
    if (a != cudaFuncAttributeMaxDynamicSharedMemorySize || bytes != 100000) return cudaErrorInvalidValue;
    ++calls[device];
    return failing ? cudaErrorInvalidValue : cudaSuccess;
}
#define EXPECT(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
    mm::SmemLimit a, b;
    static int kernel;
    failing = 1;
    EXPECT(a.allow(&kernel, 100000) != cudaSuccess && calls[0] == 1);
    failing = 0;
    for (int i = 0; i < 3; ++i) EXPECT(a.allow(&kernel, 100000) == cudaSuccess && calls[0] == 2);
    for (device = 1; device < 64; ++device)
        for (int i = 0; i < 2; ++i) EXPECT(a.allow(&kernel, 100000) == cudaSuccess && calls[device] == 1);
    device = 0;
    EXPECT(a.allow(&kernel, 100000) == cudaSuccess && calls[0] == 2);
    EXPECT(b.allow(&kernel, 100000) == cudaSuccess && calls[0] == 3);
    std::puts("ok");
    return 0;
}
"""


def include_dir():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    for d in (os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"), "/usr/local/cuda/include"):
        if os.path.exists(os.path.join(d, "cuda_runtime_api.h")):
            return d
    pytest.skip("no CUDA headers")


def test_once_on_each_device(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "dense_packed_bit_gb300", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-I", csrc, "-I", include_dir(), str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_the_serving_kernels_use_it():
    # a static in a function remembers one device's outcome for all of them
    for name in ("cache_attention_rows.cu", "cache_attention_tiles.cu", "sample.cu"):
        text = open(os.path.join(ROOT, "dense_packed_bit_gb300", "csrc", name)).read()
        assert "cudaFuncSetAttribute" not in text and "SmemLimit" in text, name
