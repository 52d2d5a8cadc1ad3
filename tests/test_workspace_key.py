"""Whom a library workspace belongs to (csrc/stream_key.h): no two streams that can run at
the same time share one.  Compiled and run on the host; no GPU needed."""
import os
import shutil
import subprocess

import pytest

from gqa_attention_kv_split_gb300 import build_lib

PROGRAM = r"""
#include <cstdio>
#include <set>
#include <thread>

#include "stream_key.h"

#define CHECK(x) \
  do { \
    if (!(x)) { \
      std::printf("%s\n", #x); \
      return 1; \
    } \
  } while (0)

int main() {
  using gqa::StreamKey;
  using gqa::stream_key;
  const cudaStream_t own = reinterpret_cast<cudaStream_t>(0x7f0000001000);
  auto there = [](cudaStream_t s) {  // the key that a thread of its own sees
    StreamKey k;
    std::thread([&] { k = stream_key(0, s); }).join();
    return k;
  };
  for (cudaStream_t s : {own, cudaStream_t(nullptr), cudaStreamLegacy}) CHECK(stream_key(0, s) == there(s));
  CHECK(stream_key(0, cudaStreamPerThread) == stream_key(0, cudaStreamPerThread));
  CHECK(stream_key(0, cudaStreamPerThread) != stream_key(1, cudaStreamPerThread));
  CHECK(stream_key(0, own) != stream_key(0, nullptr));
  std::set<StreamKey> seen{stream_key(0, cudaStreamPerThread), stream_key(0, own), stream_key(0, nullptr)};
  for (int i = 0; i < 8; ++i) CHECK(seen.insert(there(cudaStreamPerThread)).second);  // not an ended thread's either
  return 0;
}
"""


def test_threads_do_not_share_the_per_thread_stream(tmp_path):
    nvcc = os.path.realpath(build_lib._nvcc())
    include = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    if not os.path.exists(os.path.join(include, "cuda_runtime_api.h")):
        pytest.skip("no CUDA headers")
    src, exe = tmp_path / "key.cpp", tmp_path / "key"
    src.write_text(PROGRAM)
    r = subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-Wall", "-Werror", "-pthread", "-I", build_lib.CSRC, "-I", include,
                        str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
