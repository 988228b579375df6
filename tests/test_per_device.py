"""What the launchers keep per device (no GPU): the header against a stand-in for the runtime."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "engram_gram_conditional_gb300", "csrc")

SOURCE = r"""
#include <stdio.h>
#include <thread>
#include <vector>
#include "per_device.h"

static thread_local int g_device = 0;
static cudaError_t g_answer = cudaSuccess;
static int g_limit[70], g_set = 0;  // the limit of one kernel on each device
extern "C" cudaError_t cudaGetDevice(int* d) { *d = g_device; return g_answer; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int v) {
    g_limit[g_device] = v;
    ++g_set;
    return cudaSuccess;
}
static void kernel() {}
#define CHECK(x) if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; }

int main() {
    static engram::PerDevice allowed, known;
    for (int round = 0; round < 3; ++round)
        for (int d : {0, 1, 7, 63}) {
            g_device = d;
            CHECK(engram::allow_shared(allowed, (const void*)kernel, 1000) == cudaSuccess);
        }
    for (int d : {0, 1, 7, 63}) CHECK(g_limit[d] == 1000);
    CHECK(g_limit[2] == 0 && g_set == 4);  // once per device
    int made = 0, v = 0;
    auto make = [&](int* x) { ++made; *x = 10 + g_device; return cudaSuccess; };
    for (int d : {3, 4, 3, 4, 66, 66}) {  // (the last is beyond what is kept)
        g_device = d;
        CHECK(known.get(&v, make) == cudaSuccess && v == 10 + d);
    }
    CHECK(made == 4);
    // an error is returned and not kept
    g_device = 5;
    CHECK(known.get(&v, [](int*) { return cudaErrorInvalidValue; }) == cudaErrorInvalidValue);
    CHECK(known.get(&v, make) == cudaSuccess && v == 15 && made == 5);
    g_answer = cudaErrorNoDevice;
    CHECK(known.get(&v, make) == cudaErrorNoDevice && made == 5);
    g_answer = cudaSuccess;
    // many threads, each on a device of its own
    static engram::PerDevice many;
    std::vector<std::thread> threads;
    std::vector<int> got(32);
    for (int t = 0; t < 32; ++t)
        threads.emplace_back([&, t] {
            g_device = t % 8;
            for (int i = 0; i < 1000; ++i)
                many.get(&got[t], [](int* x) { *x = 100 + g_device; return cudaSuccess; });
        });
    for (auto& t : threads) t.join();
    for (int t = 0; t < 32; ++t) CHECK(got[t] == 100 + t % 8);
    printf("ok\n");
}
"""


def test_per_device(tmp_path):
    gxx = shutil.which("g++")
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not gxx or not os.path.exists(nvcc):
        pytest.skip("no compiler")
    src = tmp_path / "per_device.cpp"
    src.write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-I", CSRC, "-I", cuda, str(src), "-o",
                    str(tmp_path / "t"), "-lpthread"], check=True)
    assert subprocess.run([str(tmp_path / "t")], capture_output=True, text=True).stdout == "ok\n"


def test_limits_are_raised_per_device():
    """Kernels' shared-memory limits are raised through the header only."""
    for name in sorted(os.listdir(CSRC)):
        if name != "per_device.h":
            assert "cudaFuncSetAttribute" not in open(os.path.join(CSRC, name)).read(), name
