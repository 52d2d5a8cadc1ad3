// stream_key.h -- whom a library workspace belongs to: a device's stream.
#pragma once
#include <cuda_runtime_api.h>

#include <atomic>
#include <cstdint>
#include <tuple>

namespace gqa {

// This host thread's number; no other thread of the process ever has it.
inline uint64_t thread_number() {
  static std::atomic<uint64_t> last{0};
  thread_local const uint64_t mine = ++last;
  return mine;
}

// Device, stream handle, and the thread where the handle alone does not name a stream:
// cudaStreamPerThread is one handle for a stream of each thread.
using StreamKey = std::tuple<int, uintptr_t, uint64_t>;
inline StreamKey stream_key(int dev, cudaStream_t stream) {
  return {dev, reinterpret_cast<uintptr_t>(stream), stream == cudaStreamPerThread ? thread_number() : 0};
}

}  // namespace gqa
