"""The record of a kernel's shared-memory limit, with the runtime's calls
replaced by ones that keep the limit in a variable: two host threads that ask
for different sizes at once never leave the limit below what is recorded."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

#include "internal.h"

static std::atomic<int> g_limit{0};        // what the driver holds
static std::atomic<bool> g_first_in{false}, g_second_done{false};

extern "C" cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes) {
  g_limit = bytes;
  if (bytes == 100000) {                   // the larger size's call takes its time
    g_first_in = true;
    for (int i = 0; i < 50 && !g_second_done; ++i)
      std::this_thread::sleep_for(std::chrono::milliseconds(10));
  }
  return cudaSuccess;
}

int main() {
  static sa::SmemLimit limit;
  std::thread a([] { limit.raise(nullptr, 100000); });
  std::thread b([] {
    while (!g_first_in) std::this_thread::yield();
    limit.raise(nullptr, 60000);
    g_second_done = true;
  });
  a.join();
  b.join();
  for (int bytes : {50000, 60000, 80000, 100000, 120000}) {
    if (limit.raise(nullptr, bytes) != cudaSuccess || g_limit < bytes) {
      std::printf("a launch of %d bytes meets a limit of %d\n", bytes, g_limit.load());
      return 1;
    }
  }
  return 0;
}
"""


def test_two_threads_raise_one_limit(tmp_path):
    gxx = shutil.which("g++")
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if gxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-pthread", "-I", cuda, "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "block_sparse_paged_csr_gb300", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
