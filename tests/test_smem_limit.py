"""The launchers' shared-memory limits under first calls from several host
threads, on a stand-in for the CUDA runtime (no GPU): the limit is assigned, not
raised, so a smaller size that is set late must not undo a larger one."""
import os
import shutil
import subprocess

import pytest

from score_top_expert_gb300 import build as B

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <map>
#include <thread>

#include "router_smem.cuh"

using namespace moe_router;
using namespace std::chrono_literals;

static int device_of_calls = 0;
static std::atomic<int> limit{48 * 1024}, calls{0}, fail{0};

extern "C" cudaError_t cudaGetDevice(int* d) { *d = device_of_calls; return cudaSuccess; }

// sizes below 100 KB take long to arrive
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int value) {
  ++calls;
  if (value < 100 * 1024) std::this_thread::sleep_for(300ms);
  if (fail) return cudaErrorInvalidValue;
  limit = value;
  return cudaSuccess;
}

static void kernel() {}
static int bad = 0;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); bad = 1; } } while (0)

int main() {
  {  // a small size is on its way while a large one is set
    std::atomic<int> granted[kSmemDevs] = {};
    std::thread small([&] { CHECK(allow_smem(kernel, 80 * 1024, granted) == cudaSuccess); });
    std::this_thread::sleep_for(100ms);
    std::thread large([&] {
      CHECK(allow_smem(kernel, 200 * 1024, granted) == cudaSuccess);
    });
    small.join();
    large.join();
    // a launch of any size up to the recorded one has to find the limit set
    CHECK(allow_smem(kernel, 150 * 1024, granted) == cudaSuccess);
    CHECK(limit >= 200 * 1024);
  }
  {  // a smaller size sets nothing, a failure is not recorded
    std::atomic<int> granted[kSmemDevs] = {};
    CHECK(allow_smem(kernel, 120 * 1024, granted) == cudaSuccess);
    calls = 0;
    CHECK(allow_smem(kernel, 110 * 1024, granted) == cudaSuccess);
    CHECK(allow_smem(kernel, 16 * 1024, granted) == cudaSuccess);
    CHECK(calls == 0);
    fail = 1;
    CHECK(allow_smem(kernel, 140 * 1024, granted) != cudaSuccess);
    fail = 0;
    CHECK(allow_smem(kernel, 140 * 1024, granted) == cudaSuccess);
    CHECK(calls == 2 && limit == 140 * 1024);
  }
  {  // a device without a record is set at each call
    std::atomic<int> granted[kSmemDevs] = {};
    device_of_calls = kSmemDevs;
    calls = 0;
    CHECK(allow_smem(kernel, 130 * 1024, granted) == cudaSuccess);
    CHECK(allow_smem(kernel, 130 * 1024, granted) == cudaSuccess);
    CHECK(calls == 2);
  }
  return bad;
}
"""


def test_first_calls_of_two_sizes_from_two_threads(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc()))), "include")
    src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", f"-I{cuda}", f"-I{B.CSRC}", str(src),
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
