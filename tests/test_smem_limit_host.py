"""The recorded shared-memory limit of a kernel under calls from two host
threads, against a fake of the CUDA calls (CPU)."""
from __future__ import annotations

import subprocess

from h2o_heavy_hitter_decode_gb300 import build as hbuild

# The fake keeps the limit that was set last, as CUDA does.  A setting of the larger limit does not return before the
# other thread has set its own, or half a second has passed.
PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "smem_limit.h"

static std::atomic<int> limit{0}, calls{0}, small_set{0}, large_began{0};
extern "C" cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int v) {
  ++calls;
  limit = v;
  if (v == 90000) {
    large_began = 1;
    for (int i = 0; i < 500 && !small_set; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
  } else {
    small_set = 1;
  }
  return cudaSuccess;
}
int main() {
  static h2o::blk::SmemLimit s;
  int failed = 0;
  auto launch = [&](int want) { if (s.raise(nullptr, want) != cudaSuccess || limit < want) ++failed; };
  std::thread large([&] { launch(90000); });
  std::thread small([&] {
    while (!large_began) std::this_thread::yield();
    launch(50000);
  });
  large.join();
  small.join();
  launch(90000);
  launch(60000);
  const int before = calls;
  launch(90000);
  launch(70000);
  std::printf("%d failed, limit %d, %d calls after the first\n", failed, limit.load(), calls - before);
  return failed || calls != before;
}
"""


def test_two_threads_keep_the_larger_limit(tmp_path):
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run([hbuild.nvcc(), "-std=c++17", "-cudart", "none", "-I", hbuild.CSRC, "-Xcompiler", "-pthread",
                    str(src), "-o", str(exe), "-lpthread"], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
