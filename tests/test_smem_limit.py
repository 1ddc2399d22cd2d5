"""The table of shared-memory limits (csrc/smem_limit.h) under two threads, compiled for the host alone: the
limits are a program's variables, set with a delay that lets the other thread pass."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "smem_limit.h"

static void nap(int ms) { std::this_thread::sleep_for(std::chrono::milliseconds(ms)); }

int main() {
  static lora::SmemLimits<4, 2> table;
  static int kernels[6];
  static size_t limit[6][2];
  static int sets[6];
  auto raise = [&](int k, int dev, size_t bytes, int ms) {
    return table.raise(&kernels[k], dev, bytes, [&, k, dev, bytes, ms] {
      nap(ms);
      ++sets[k];
      limit[k][dev] = bytes;
      return 0;
    });
  };
  // the smaller size starts first and is set last
  std::thread a([&] { raise(0, 0, 1000, 300); });
  std::thread b([&] { nap(100); raise(0, 0, 5000, 0); });
  a.join();
  b.join();
  std::printf("raced %zu\n", limit[0][0]);
  raise(0, 0, 5000, 0);
  std::printf("after %zu\n", limit[0][0]);
  const int before = sets[0];
  raise(0, 0, 4000, 0);
  std::printf("again %d\n", sets[0] - before);
  raise(0, 1, 700, 0);  // each device its own
  std::printf("device %zu %zu\n", limit[0][0], limit[0][1]);
  // a call that fails leaves nothing behind
  const int e = table.raise(&kernels[1], 0, 10, [] { return 7; });
  std::printf("failed %d\n", e);
  raise(1, 0, 10, 0);
  std::printf("retried %zu\n", limit[1][0]);
  for (int k = 2; k < 6; ++k) raise(k, 0, 10, 0);  // more kernels than slots: set at each call
  raise(5, 0, 10, 0);
  std::printf("full %d %d\n", sets[2], sets[5]);
  return 0;
}
"""


def test_two_threads_leave_the_larger_limit(tmp_path):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "limits.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "limits"
    subprocess.run([cc, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-pthread", "-I",
                    os.path.join(ROOT, "segmented_gather_gemm_lora_gb300", "csrc"), str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    out = dict(line.split(" ", 1) for line in subprocess.run([str(exe)], check=True, capture_output=True,
                                                             text=True, timeout=60).stdout.splitlines())
    assert out["raced"] == "5000" and out["after"] == "5000"
    assert out["again"] == "0"
    assert out["device"] == "5000 700"
    assert out["failed"] == "7" and out["retried"] == "10"
    assert out["full"] == "1 2"
