"""First calls from several threads: the lookup of the driver's tensor-map encoder (csrc/tensor_map.cuh), compiled for the
host with a runtime whose lookup takes its time."""
import subprocess

from weight_only_int4_route_gb300 import build as B

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "tensor_map.cuh"

static std::atomic<int> lookups{0};
extern "C" cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(const char *, void **ptr, unsigned int, unsigned long long,
                                                                  cudaDriverEntryPointQueryResult *result) {
  ++lookups;
  std::this_thread::sleep_for(std::chrono::milliseconds(200));
  *ptr = reinterpret_cast<void *>(0x1000);
  *result = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

int main() {
  std::atomic<int> without{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 4; ++i)
    threads.emplace_back([&, i] {
      std::this_thread::sleep_for(std::chrono::milliseconds(20 * i));
      if (moe::encode_fn() == nullptr) ++without;
    });
  for (auto &t : threads) t.join();
  std::printf("%d %d\n", without.load(), lookups.load());
}
"""


def test_no_thread_is_told_that_there_is_no_encoder(tmp_path):
    src, exe = tmp_path / "first.cpp", tmp_path / "first"
    src.write_text(PROGRAM)
    r = subprocess.run([B.nvcc(), "-std=c++17", "-cudart", "none", "-I", B.CSRC, "-I", B.INCLUDE, str(src), "-o", str(exe), "-Xcompiler",
                        "-pthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.split() == ["0", "1"]
