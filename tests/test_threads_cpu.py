"""Host code that several threads enter at once (no GPU: the CUDA call behind it is a slow stand-in)."""
import os
import subprocess

from linear_attention_recurrence_fwd_gb300 import build

FIRST_CALLS = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "tma_host.h"

extern "C" cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned int, unsigned long long,
                                                        cudaDriverEntryPointQueryResult* q) {
  std::this_thread::sleep_for(std::chrono::milliseconds(200));
  *p = reinterpret_cast<void*>(16);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

int main() {
  std::atomic<int> without{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 4; ++i)
    threads.emplace_back([&] { without += kda::tensor_map_encoder() == nullptr; });
  for (auto& t : threads) t.join();
  std::printf("%d", without.load());
}
"""


def test_first_calls_find_the_tensor_map_encoder(tmp_path):
    source, program = tmp_path / "first.cpp", tmp_path / "first"
    source.write_text(FIRST_CALLS)
    cuda = os.path.dirname(os.path.dirname(build.nvcc()))
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", build.CSRC, "-I", os.path.join(cuda, "include"), str(source), "-o",
                    str(program)], check=True)
    assert subprocess.run([str(program)], capture_output=True, text=True, timeout=60).stdout == "0"
