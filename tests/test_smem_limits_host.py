"""Dynamic shared memory beyond the default is allowed per kernel and per device.
No GPU: the helper runs against a stand-in runtime with several devices."""
import glob
import os
import shutil
import subprocess

import pytest

from paged_kv_chunk_chunked_gb300 import build as pkv_build

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "internal.h"

static thread_local int device = 0;
static int calls = 0;
static int limit[2][100];                    // by kernel and device
static void kernel_a() {}
static void kernel_b() {}
static bool fail_next = false;

extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
    if (a != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaErrorInvalidValue;
    if (fail_next) { fail_next = false; return cudaErrorInvalidValue; }
    ++calls;
    limit[f == (const void*)kernel_b][device] = v;
    return cudaSuccess;
}

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
    static pkv::SmemGrant a, b;
    for (int turn = 0; turn < 3; ++turn)
        for (int d : {0, 1, 7, 99}) {        // 99: beyond the table, set each time
            device = d;
            CHECK(pkv::allow_smem(kernel_a, 100000, a) == cudaSuccess && limit[0][d] == 100000);
        }
    CHECK(calls == 3 + 3 && limit[1][0] == 0);
    device = 1;
    CHECK(pkv::allow_smem(kernel_b, 60000, b) == cudaSuccess && limit[1][1] == 60000 && limit[1][0] == 0);
    CHECK(pkv::allow_smem(kernel_b, 50000, b) == cudaSuccess && limit[1][1] == 60000);   // less is allowed already
    CHECK(pkv::allow_smem(kernel_b, 200000, b) == cudaSuccess && limit[1][1] == 200000);
    device = 2;
    fail_next = true;                        // a failure is not remembered as a success
    CHECK(pkv::allow_smem(kernel_b, 60000, b) == cudaErrorInvalidValue);
    CHECK(pkv::allow_smem(kernel_b, 60000, b) == cudaSuccess && limit[1][2] == 60000);
    std::vector<std::thread> ts;
    for (int i = 0; i < 16; ++i)             // the largest request holds, whatever the order
        ts.emplace_back([i] {
            device = 3;
            pkv::allow_smem(kernel_a, 1000 * (1 + i * 7 % 16), a);
        });
    for (auto& t : ts) t.join();
    CHECK(limit[0][3] == 16000);
    std::puts("ok");
    return 0;
}
"""


def test_one_limit_per_kernel_and_device(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(pkv_build.nvcc()))), "include")
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", pkv_build.CSRC, "-I", os.path.join(pkv_build.ROOT, "include"),
                    "-I", cuda, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_no_kernel_keeps_a_limit_of_its_own():
    """Every limit goes through the helper: a flag per process would leave out the second device."""
    for path in sorted(glob.glob(os.path.join(pkv_build.CSRC, "*"))):
        with open(path) as f:
            if os.path.basename(path) != "internal.h":
                assert "cudaFuncSetAttribute" not in f.read(), path
