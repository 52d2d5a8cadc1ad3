// api_util.h -- what the translation units of the C ABI (api.cpp, api_paged.cpp) share:
// error messages, device scoping, checks of pointers and descriptors, workspaces.
#pragma once
#include "../../include/gqa.h"

#include <cuda_runtime.h>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <initializer_list>
#include <cstdio>
#include <cstring>
#include <exception>
#include <map>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "stream_key.h"

namespace gqa {
namespace api {
inline thread_local std::string t_last_error;

inline gqa_status fail(gqa_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return st;
}

inline gqa_status cuda_fail(cudaError_t e, const char* what) {
  return fail(GQA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

#define GQA_CUDA_TRY(expr, what)                   \
  do {                                             \
    cudaError_t _e = (expr);                       \
    if (_e != cudaSuccess) return cuda_fail(_e, what); \
  } while (0)

// Switches to `dev` for the lifetime of the object; restores the previous
// current device afterwards.
class ScopedDevice {
 public:
  explicit ScopedDevice(int dev) {
    if (cudaGetDevice(&prev_) != cudaSuccess) prev_ = -1;
    if (prev_ != dev) ok_ = (cudaSetDevice(dev) == cudaSuccess);
    switched_ = (prev_ != dev) && ok_;
  }
  ~ScopedDevice() {
    if (switched_ && prev_ >= 0) cudaSetDevice(prev_);
  }
  bool ok() const { return ok_; }

 private:
  int prev_ = -1;
  bool ok_ = true;
  bool switched_ = false;
};

// Where a pointer lives.
struct Where {
  bool host;
  int device;
};

inline gqa_status classify(const void* p, const char* name, Where* w) {
  cudaPointerAttributes a;
  cudaError_t e = cudaPointerGetAttributes(&a, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_fail(e, "cudaPointerGetAttributes");
  }
  if (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged) {
    w->host = false;
    w->device = a.device;
  } else {
    w->host = true;
    w->device = -1;
  }
  (void)name;
  return GQA_OK;
}

struct Arg {
  const void* p;
  const char* name;
  size_t align;
};

constexpr int kAnyDevice = -1000;  // no expectation from a descriptor

// All pointers on one side: either the same device or all host; when
// `expect` is a descriptor's device field (-1 = host), the memory must be
// there.
inline gqa_status locate(const std::vector<Arg>& args, Where* out, int expect = kAnyDevice) {
  for (const Arg& a : args)
    if (a.p == nullptr) return fail(GQA_ERR_INVALID_ARG, "%s is a null pointer", a.name);
  Where first{};
  for (size_t i = 0; i < args.size(); ++i) {
    Where w;
    gqa_status st = classify(args[i].p, args[i].name, &w);
    if (st != GQA_OK) return st;
    if (i == 0) {
      first = w;
    } else if (w.host != first.host || w.device != first.device) {
      return fail(GQA_ERR_DEVICE_MISMATCH, "%s is on %s %d but %s is on %s %d", args[i].name,
                  w.host ? "host" : "device", w.device, args[0].name, first.host ? "host" : "device",
                  first.device);
    }
    if (!w.host && (reinterpret_cast<uintptr_t>(args[i].p) % args[i].align) != 0)
      return fail(GQA_ERR_INVALID_ARG, "%s is not %zu-byte aligned", args[i].name, args[i].align);
  }
  const int real = first.host ? -1 : first.device;
  if (expect != kAnyDevice && real != expect)
    return fail(GQA_ERR_DEVICE_MISMATCH, "the descriptors say device %d but the memory is on %s %d", expect,
                first.host ? "host" : "device", first.device);
  *out = first;
  return GQA_OK;
}

// Grow-only device scratch per (device, stream).
struct Workspace {
  void* ptr = nullptr;
  size_t bytes = 0;
};
inline std::mutex g_ws_mu;
using WorkspaceMap = std::map<gqa::StreamKey, Workspace>;
inline WorkspaceMap g_ws;
// Of gqa_paged_attn_t's calls without a workspace (a map of their own: growing one
// never moves the other, which a captured call may have been given).
inline WorkspaceMap g_paged_ws;
// Of gqa_paged_tree_attn_t's.
inline WorkspaceMap g_tree_ws;
inline std::mutex g_paged_launch_mu;

inline gqa_status workspace(int dev, cudaStream_t stream, size_t bytes, void** out, WorkspaceMap& map = g_ws) {
  *out = nullptr;
  if (bytes == 0) return GQA_OK;
  std::lock_guard<std::mutex> lk(g_ws_mu);
  Workspace& w = map[gqa::stream_key(dev, stream)];
  if (w.bytes < bytes) {
    if (w.ptr) {
      // Work queued on this stream may still use the old buffer.
      cudaError_t e = cudaStreamSynchronize(stream);
      if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
      cudaFree(w.ptr);
      w.ptr = nullptr;
      w.bytes = 0;
    }
    size_t grow = bytes + bytes / 8;
    cudaError_t e = cudaMalloc(&w.ptr, grow);
    if (e != cudaSuccess) {
      cudaGetLastError();
      w.ptr = nullptr;
      e = cudaMalloc(&w.ptr, bytes);
      if (e != cudaSuccess) {
        cudaGetLastError();
        w.ptr = nullptr;
        return fail(GQA_ERR_OOM, "workspace of %zu bytes: %s", bytes, cudaGetErrorString(e));
      }
      grow = bytes;
    }
    w.bytes = grow;
  }
  *out = w.ptr;
  return GQA_OK;
}

// Gives back a thread's g_paged_ws and g_tree_ws buffers when it ends: its per-thread stream ends with it.
// (g_ws's stay until gqa_release_workspace: a captured call may have been given one.)
struct ThreadEnd {
  uint64_t thread = 0;
  ~ThreadEnd() {
    if (!thread) return;
    std::lock_guard<std::mutex> lk(g_ws_mu);
    int prev = -1;
    cudaGetDevice(&prev);
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // (leaves a capture of another thread alone)
    cudaThreadExchangeStreamCaptureMode(&mode);
    for (WorkspaceMap* map : {&g_paged_ws, &g_tree_ws})
      for (auto it = map->begin(); it != map->end();) {
        if (std::get<2>(it->first) != thread) {
          ++it;
          continue;
        }
        cudaSetDevice(std::get<0>(it->first));
        cudaStreamSynchronize(cudaStreamPerThread);
        cudaFree(it->second.ptr);
        it = map->erase(it);
      }
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (prev >= 0) cudaSetDevice(prev);
  }
};

// Carves 256-byte aligned sub-buffers out of one allocation.
struct Carver {
  size_t off = 0;
  size_t take(size_t bytes) {
    size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  }
};

// ---- tensor descriptors (gqa_tensor) ---------------------------------------

inline const char* dtype_name(int32_t d) {
  switch (d) {
    case GQA_F16: return "f16";
    case GQA_E4M3: return "e4m3";
    case GQA_U8: return "u8";
    case GQA_I32: return "i32";
    case GQA_F32: return "f32";
    case GQA_BF16: return "bf16";
    default: return "unknown";
  }
}

// Structural check of one descriptor: non-null, an accepted dtype, the rank
// and shape asked for (-1 = any extent, returned in got[]), dense row-major
// strides (in elements; a dimension of extent 1 may carry any stride).  No
// CUDA call: it runs before anything touches the device.
inline gqa_status check_desc(const gqa_tensor* t, const char* name, std::initializer_list<int32_t> dtypes,
                      std::initializer_list<int64_t> shape, int64_t* got = nullptr) {
  if (!t) return fail(GQA_ERR_INVALID_ARG, "%s: null descriptor", name);
  if (!t->data) return fail(GQA_ERR_INVALID_ARG, "%s is a null pointer", name);
  bool dt_ok = false;
  for (int32_t d : dtypes) dt_ok |= (t->dtype == d);
  if (!dt_ok) {
    std::string want;
    for (int32_t d : dtypes) want += std::string(want.empty() ? "" : " or ") + dtype_name(d);
    return fail(GQA_ERR_INVALID_ARG, "%s has dtype %s; expected %s", name, dtype_name(t->dtype), want.c_str());
  }
  const int nd = (int)shape.size();
  if (t->ndim != nd) return fail(GQA_ERR_INVALID_ARG, "%s has %d dimensions; expected %d", name, t->ndim, nd);
  int i = 0;
  for (int64_t want : shape) {
    const int64_t have = t->shape[i];
    if (have < 0) return fail(GQA_ERR_INVALID_ARG, "%s: negative extent in dimension %d", name, i);
    if (want >= 0 && have != want)
      return fail(GQA_ERR_UNSUPPORTED_SHAPE, "%s has extent %lld in dimension %d; expected %lld", name,
                  (long long)have, i, (long long)want);
    if (got) got[i] = have;
    ++i;
  }
  int64_t expect = 1;
  for (int d = nd - 1; d >= 0; --d) {
    if (t->shape[d] != 1 && t->strides[d] != expect)
      return fail(GQA_ERR_INVALID_ARG, "%s is not dense row-major (stride %lld in dimension %d; expected %lld)", name,
                  (long long)t->strides[d], d, (long long)expect);
    expect *= t->shape[d];
  }
  return GQA_OK;
}

// Every descriptor names the same device (or all host memory, device -1).
// (Where the memory really is, is checked once per pointer by locate().)
inline gqa_status check_devices(std::initializer_list<std::pair<const gqa_tensor*, const char*>> ts) {
  const gqa_tensor* first = ts.begin()->first;
  for (const auto& t : ts)
    if (t.first->device != first->device)
      return fail(GQA_ERR_DEVICE_MISMATCH, "%s is on device %d but %s is on device %d", t.second, t.first->device,
                  ts.begin()->second, first->device);
  return GQA_OK;
}

#define GQA_TRY(expr)                  \
  do {                                 \
    gqa_status _s = (expr);            \
    if (_s != GQA_OK) return _s;       \
  } while (0)

// Runs an entry point's body; no exception (a failed allocation on the host) crosses the boundary.
template <typename F>
gqa_status guarded(F&& body) {
  try {
    return body();
  } catch (const std::exception& e) {
    return fail(GQA_ERR_OOM, "%s", e.what());
  } catch (...) {
    return fail(GQA_ERR_OOM, "an exception");
  }
}

}  // namespace api
}  // namespace gqa
