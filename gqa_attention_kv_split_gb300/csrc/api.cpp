// api.cpp -- the C ABI of libgqa (include/gqa.h): argument validation,
// device scoping, workspace ownership, host-buffer staging and launch.
//
// Launcher conventions follow "FlashInfer NVFP4 QKV GEMM 최적화: SM103a
// Epilogue 통합 및 CUDA 런처 개선", section 2: every tensor must sit on one
// device (checked per pointer), the call switches to that device and
// restores the caller's (no current-device check), and a launch grid must be
// positive.  Nothing here computes attention; every step of the path runs in
// the kernels of decode.cu and ctx_nvfp4.cu.
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

#include "kernels.h"
#include "paged.h"
#include "stream_key.h"

namespace {

thread_local std::string t_last_error;

gqa_status fail(gqa_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return st;
}

gqa_status cuda_fail(cudaError_t e, const char* what) {
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

gqa_status classify(const void* p, const char* name, Where* w) {
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
gqa_status locate(const std::vector<Arg>& args, Where* out, int expect = kAnyDevice) {
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
std::mutex g_ws_mu;
using WorkspaceMap = std::map<gqa::StreamKey, Workspace>;
WorkspaceMap g_ws;
// Of gqa_paged_attn_t's calls without a workspace (a map of their own: growing one
// never moves the other, which a captured call may have been given).
WorkspaceMap g_paged_ws;
std::mutex g_paged_launch_mu;

gqa_status workspace(int dev, cudaStream_t stream, size_t bytes, void** out, WorkspaceMap& map = g_ws) {
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

// Gives back a thread's g_paged_ws buffers when it ends: its per-thread stream ends with it.
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
    for (auto it = g_paged_ws.begin(); it != g_paged_ws.end();) {
      if (std::get<2>(it->first) != thread) {
        ++it;
        continue;
      }
      cudaSetDevice(std::get<0>(it->first));
      cudaStreamSynchronize(cudaStreamPerThread);
      cudaFree(it->second.ptr);
      it = g_paged_ws.erase(it);
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

const char* dtype_name(int32_t d) {
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
gqa_status check_desc(const gqa_tensor* t, const char* name, std::initializer_list<int32_t> dtypes,
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
gqa_status check_devices(std::initializer_list<std::pair<const gqa_tensor*, const char*>> ts) {
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

std::atomic<int> g_starve{0};
std::atomic<int> g_ctx_stages{0}, g_ctx_slots{0}, g_decode_stages{0}, g_ctx_grid{0};

}  // namespace

namespace gqa {
int starve_producers() { return g_starve.load(std::memory_order_relaxed); }
int schedule_ctx_stages() { return g_ctx_stages.load(std::memory_order_relaxed); }
int schedule_ctx_slots() { return g_ctx_slots.load(std::memory_order_relaxed); }
int schedule_decode_stages() { return g_decode_stages.load(std::memory_order_relaxed); }
int schedule_ctx_grid() { return g_ctx_grid.load(std::memory_order_relaxed); }
}  // namespace gqa

extern "C" {

const char* gqa_last_error(void) { return t_last_error.c_str(); }

int gqa_version(void) { return 401; }  // 0.4.1: caps of any size, workspaces of per-thread streams, every offset checked

namespace {
gqa_status decode_impl(const void* q, const void* kv, const int32_t* seq_lens, void* out, int64_t batch,
                       int64_t capacity, float q_scale, gqa_stream_t stream_, int expect) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (batch < 1 || batch > 65535) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 65535]", (long long)batch);
  if (capacity < 1 || capacity > 2147483647LL)
    return fail(GQA_ERR_UNSUPPORTED, "capacity %lld outside [1, 2^31-1]", (long long)capacity);
  if (!std::isfinite(q_scale)) return fail(GQA_ERR_INVALID_ARG, "q_scale is not finite");
  Where where;
  gqa_status st =
      locate({{q, "q", 16}, {kv, "kv", 16}, {seq_lens, "seq_lens", 4}, {out, "out", 16}}, &where, expect);
  if (st != GQA_OK) return st;

  const gqa::DecodePlan plan = gqa::plan_decode(batch, capacity);
  if (plan.n_splits < 1) return fail(GQA_ERR_INVALID_ARG, "launch grid must be positive");
  const size_t part_bytes = gqa::decode_workspace_bytes(batch, plan);

  if (!where.host) {
    ScopedDevice sd(where.device);
    if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
    void* ws = nullptr;
    if ((st = workspace(where.device, stream, part_bytes, &ws)) != GQA_OK) return st;
    GQA_CUDA_TRY(gqa::launch_decode(q, kv, seq_lens, out, batch, capacity, q_scale, plan, ws, stream),
                 "decode launch");
    return GQA_OK;
  }

  // Host buffers: stage the bytes the kernels read, run, copy the result back.
  int dev = 0;
  GQA_CUDA_TRY(cudaGetDevice(&dev), "cudaGetDevice");
  const size_t q_bytes = (size_t)batch * 32 * 128 * 2;
  const size_t slab = (size_t)capacity * 128 * 2;  // one (b, K|V, g) slab
  const size_t kv_bytes = (size_t)batch * 2 * 8 * slab;
  Carver c;
  const size_t o_q = c.take(q_bytes), o_kv = c.take(kv_bytes), o_len = c.take((size_t)batch * 4),
               o_out = c.take(q_bytes), o_part = c.take(part_bytes);
  void* ws = nullptr;
  if ((st = workspace(dev, stream, c.off, &ws)) != GQA_OK) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  GQA_CUDA_TRY(cudaMemcpyAsync(base + o_q, q, q_bytes, cudaMemcpyHostToDevice, stream), "copy q");
  GQA_CUDA_TRY(cudaMemcpyAsync(base + o_len, seq_lens, (size_t)batch * 4, cudaMemcpyHostToDevice, stream),
               "copy seq_lens");
  for (int64_t b = 0; b < batch; ++b) {
    int64_t len = seq_lens[b];
    len = len < 0 ? 0 : (len > capacity ? capacity : len);
    if (len == 0) continue;
    // 16 slabs (K and V of 8 heads), each with its first len tokens.
    const uint8_t* src = static_cast<const uint8_t*>(kv) + (size_t)b * 16 * slab;
    GQA_CUDA_TRY(cudaMemcpy2DAsync(base + o_kv + (size_t)b * 16 * slab, slab, src, slab, (size_t)len * 256, 16,
                                   cudaMemcpyHostToDevice, stream),
                 "copy kv");
  }
  GQA_CUDA_TRY(gqa::launch_decode(base + o_q, base + o_kv, reinterpret_cast<const int32_t*>(base + o_len),
                                  base + o_out, batch, capacity, q_scale, plan,
                                  part_bytes ? base + o_part : nullptr, stream),
               "decode launch");
  GQA_CUDA_TRY(cudaMemcpyAsync(out, base + o_out, q_bytes, cudaMemcpyDeviceToHost, stream), "copy out");
  GQA_CUDA_TRY(cudaStreamSynchronize(stream), "cudaStreamSynchronize");
  return GQA_OK;
}

gqa_status decode_paged_impl(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                             const int32_t* seq_lens, void* out, int64_t batch, int64_t num_pages,
                             int64_t max_pages_per_seq, float q_scale, gqa_stream_t stream_, int expect) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (batch < 1 || batch > 65535) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 65535]", (long long)batch);
  if (num_pages < 1 || num_pages > 2147483647LL)
    return fail(GQA_ERR_INVALID_ARG, "num_pages %lld out of range", (long long)num_pages);
  if (max_pages_per_seq < 1 || max_pages_per_seq > (2147483647LL / 64))
    return fail(GQA_ERR_INVALID_ARG, "max_pages_per_seq %lld out of range", (long long)max_pages_per_seq);
  if (!std::isfinite(q_scale)) return fail(GQA_ERR_INVALID_ARG, "q_scale is not finite");
  Where where;
  gqa_status st = locate({{q, "q", 16},
                          {k_pages, "k_pages", 16},
                          {v_pages, "v_pages", 16},
                          {block_table, "block_table", 4},
                          {seq_lens, "seq_lens", 4},
                          {out, "out", 16}},
                         &where, expect);
  if (st != GQA_OK) return st;
  const int64_t capacity = max_pages_per_seq * 64;
  const gqa::DecodePlan plan = gqa::plan_decode(batch, capacity);
  if (plan.n_splits < 1) return fail(GQA_ERR_INVALID_ARG, "launch grid must be positive");
  const size_t part_bytes = gqa::decode_workspace_bytes(batch, plan);
  gqa::DecodePages pg;
  pg.num_pages = num_pages;
  pg.max_pages_per_seq = max_pages_per_seq;

  if (!where.host) {
    ScopedDevice sd(where.device);
    if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
    void* ws = nullptr;
    if ((st = workspace(where.device, stream, part_bytes, &ws)) != GQA_OK) return st;
    pg.k_pages = k_pages;
    pg.v_pages = v_pages;
    pg.block_table = block_table;
    GQA_CUDA_TRY(gqa::launch_decode_paged(q, pg, seq_lens, out, batch, q_scale, plan, ws, stream),
                 "paged decode launch");
    return GQA_OK;
  }

  // Host buffers: the host can read the lengths and the table, so check the
  // pages a sequence uses, then stage everything and run.
  for (int64_t b = 0; b < batch; ++b) {
    int64_t len = seq_lens[b];
    len = len < 0 ? 0 : (len > capacity ? capacity : len);
    for (int64_t p = 0; p < (len + 63) / 64; ++p) {
      const int32_t pgid = block_table[b * max_pages_per_seq + p];
      if (pgid < 0 || pgid >= num_pages)
        return fail(GQA_ERR_INVALID_ARG, "block_table[%lld][%lld] = %d outside [0, num_pages)", (long long)b,
                    (long long)p, pgid);
    }
  }
  int dev = 0;
  GQA_CUDA_TRY(cudaGetDevice(&dev), "cudaGetDevice");
  const size_t q_bytes = (size_t)batch * 32 * 128 * 2;
  const size_t page_bytes = (size_t)num_pages * 8 * 64 * 128 * 2;
  const size_t bt_bytes = (size_t)batch * max_pages_per_seq * 4;
  Carver c;
  const size_t o_q = c.take(q_bytes), o_k = c.take(page_bytes), o_v = c.take(page_bytes), o_bt = c.take(bt_bytes),
               o_len = c.take((size_t)batch * 4), o_out = c.take(q_bytes), o_part = c.take(part_bytes);
  void* ws = nullptr;
  if ((st = workspace(dev, stream, c.off, &ws)) != GQA_OK) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  const std::pair<size_t, std::pair<const void*, size_t>> copies[] = {
      {o_q, {q, q_bytes}},       {o_k, {k_pages, page_bytes}},        {o_v, {v_pages, page_bytes}},
      {o_bt, {block_table, bt_bytes}}, {o_len, {seq_lens, (size_t)batch * 4}}};
  for (const auto& cp : copies)
    GQA_CUDA_TRY(cudaMemcpyAsync(base + cp.first, cp.second.first, cp.second.second, cudaMemcpyHostToDevice, stream),
                 "stage input");
  pg.k_pages = base + o_k;
  pg.v_pages = base + o_v;
  pg.block_table = reinterpret_cast<const int32_t*>(base + o_bt);
  GQA_CUDA_TRY(gqa::launch_decode_paged(base + o_q, pg, reinterpret_cast<const int32_t*>(base + o_len), base + o_out,
                                        batch, q_scale, plan, part_bytes ? base + o_part : nullptr, stream),
               "paged decode launch");
  GQA_CUDA_TRY(cudaMemcpyAsync(out, base + o_out, q_bytes, cudaMemcpyDeviceToHost, stream), "copy out");
  GQA_CUDA_TRY(cudaStreamSynchronize(stream), "cudaStreamSynchronize");
  return GQA_OK;
}
}  // namespace

gqa_status gqa_decode(const void* q, const void* kv, const int32_t* seq_lens, void* out, int64_t batch,
                      int64_t capacity, float q_scale, gqa_stream_t stream) {
  return decode_impl(q, kv, seq_lens, out, batch, capacity, q_scale, stream, kAnyDevice);
}

gqa_status gqa_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                            const int32_t* seq_lens, void* out, int64_t batch, int64_t num_pages,
                            int64_t max_pages_per_seq, float q_scale, gqa_stream_t stream) {
  return decode_paged_impl(q, k_pages, v_pages, block_table, seq_lens, out, batch, num_pages, max_pages_per_seq,
                           q_scale, stream, kAnyDevice);
}

gqa_status gqa_decode_noalloc(const void* q, const void* kv, const int32_t* seq_lens, void* out, int64_t batch,
                              int64_t capacity, float q_scale, gqa_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (batch < 1 || batch > 65535) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 65535]", (long long)batch);
  if (capacity < 1 || capacity > 2147483647LL)
    return fail(GQA_ERR_UNSUPPORTED, "capacity %lld outside [1, 2^31-1]", (long long)capacity);
  if (!std::isfinite(q_scale)) return fail(GQA_ERR_INVALID_ARG, "q_scale is not finite");
  Where where;
  gqa_status st = locate({{q, "q", 16}, {kv, "kv", 16}, {seq_lens, "seq_lens", 4}, {out, "out", 16}}, &where);
  if (st != GQA_OK) return st;
  if (where.host)
    return fail(GQA_ERR_UNSUPPORTED,
                "gqa_decode_noalloc takes device pointers only (host buffers would need staging memory)");
  const gqa::DecodePlan plan = gqa::plan_decode(batch, capacity);
  const size_t need = gqa::decode_workspace_bytes(batch, plan);
  if (need > gqa::kDecodeStaticScratchBytes)
    return fail(GQA_ERR_UNSUPPORTED,
                "batch %lld x capacity %lld needs %zu bytes of split partials; the static scratch holds %zu "
                "(use gqa_decode)",
                (long long)batch, (long long)capacity, need, gqa::kDecodeStaticScratchBytes);
  ScopedDevice sd(where.device);
  if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
  GQA_CUDA_TRY(gqa::launch_decode_static_scratch(q, kv, seq_lens, out, batch, capacity, q_scale, plan, stream),
               "decode launch (static scratch)");
  return GQA_OK;
}

gqa_status gqa_decode_plan(int64_t batch, int64_t capacity, int32_t* tokens_per_split, int32_t* num_splits,
                           int32_t* num_launches) {
  if (batch < 1 || batch > 65535) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 65535]", (long long)batch);
  if (capacity < 1 || capacity > 2147483647LL)
    return fail(GQA_ERR_UNSUPPORTED, "capacity %lld outside [1, 2^31-1]", (long long)capacity);
  const gqa::DecodePlan plan = gqa::plan_decode(batch, capacity);
  if (tokens_per_split) *tokens_per_split = plan.chunk;
  if (num_splits) *num_splits = plan.n_splits;
  if (num_launches) *num_launches = plan.n_splits > 1 ? 2 : 1;
  return GQA_OK;
}

gqa_status gqa_ctx_plan(int64_t batch, int64_t total_q, int64_t max_pages_per_seq, int32_t* tiles_per_split,
                        int32_t* num_splits, int32_t* num_launches, int32_t* persistent, int32_t* decode_shaped) {
  if (batch < 1 || batch > (1 << 20)) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 2^20]", (long long)batch);
  if (total_q < 0 || total_q > 2147483647LL) return fail(GQA_ERR_INVALID_ARG, "total_q %lld out of range", (long long)total_q);
  if (max_pages_per_seq < 1 || max_pages_per_seq > (2147483647LL / 64))
    return fail(GQA_ERR_INVALID_ARG, "max_pages_per_seq %lld out of range", (long long)max_pages_per_seq);
  const gqa::CtxPlan plan = gqa::plan_ctx(batch, total_q, max_pages_per_seq);
  if (tiles_per_split) *tiles_per_split = plan.tiles_per_split;
  if (num_splits) *num_splits = plan.n_splits;
  if (num_launches) *num_launches = total_q == 0 ? 0 : (plan.n_splits > 1 || plan.decode_rows ? 2 : 1);
  if (persistent) *persistent = total_q > 0 && plan.n_splits == 1 && plan.persistent && !plan.decode_rows ? 1 : 0;
  if (decode_shaped) *decode_shaped = total_q > 0 && plan.decode_rows ? 1 : 0;
  return GQA_OK;
}

namespace {
gqa_status ctx_impl(const void* q_fp8, float q_scale, const void* k_fp4, const void* k_sf, const void* v_fp4,
                    const void* v_sf, const int32_t* block_table, const int32_t* qo_indptr, const int32_t* kv_lens,
                    void* out_fp8, float out_scale, int64_t batch, int64_t total_q, int64_t num_pages,
                    int64_t max_pages_per_seq, gqa_stream_t stream_, int expect) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (batch < 1 || batch > (1 << 20))
    return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 2^20]", (long long)batch);
  if (total_q < 0 || total_q > 2147483647LL) return fail(GQA_ERR_INVALID_ARG, "total_q %lld out of range", (long long)total_q);
  if (num_pages < 1 || num_pages > 2147483647LL) return fail(GQA_ERR_INVALID_ARG, "num_pages %lld out of range", (long long)num_pages);
  if (max_pages_per_seq < 1 || max_pages_per_seq > (2147483647LL / 64))
    return fail(GQA_ERR_INVALID_ARG, "max_pages_per_seq %lld out of range", (long long)max_pages_per_seq);
  if (!std::isfinite(q_scale)) return fail(GQA_ERR_INVALID_ARG, "q_scale is not finite");
  if (!std::isfinite(out_scale) || !(out_scale > 0.f)) return fail(GQA_ERR_INVALID_ARG, "out_scale must be finite and > 0");
  Where where;
  gqa_status st = locate({{q_fp8, "q_fp8", 16},
                          {k_fp4, "k_fp4", 16},
                          {k_sf, "k_sf", 16},
                          {v_fp4, "v_fp4", 16},
                          {v_sf, "v_sf", 16},
                          {block_table, "block_table", 4},
                          {qo_indptr, "qo_indptr", 4},
                          {kv_lens, "kv_lens", 4},
                          {out_fp8, "out_fp8", 16}},
                         &where, expect);
  if (st != GQA_OK) return st;

  gqa::CtxArgs a;
  a.starve = gqa::starve_producers();
  a.q_scale = q_scale;
  a.out_scale = out_scale;
  a.batch = batch;
  a.total_q = total_q;
  a.num_pages = num_pages;
  a.max_pages_per_seq = max_pages_per_seq;
  const gqa::CtxPlan plan = gqa::plan_ctx(batch, total_q, max_pages_per_seq);
  const size_t part_bytes = gqa::ctx_workspace_bytes(total_q, plan);

  if (!where.host) {
    if (total_q == 0) return GQA_OK;
    ScopedDevice sd(where.device);
    if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
    void* part = nullptr;
    if (part_bytes && (st = workspace(where.device, stream, part_bytes, &part)) != GQA_OK) return st;
    a.q = static_cast<const uint8_t*>(q_fp8);
    a.k_fp4 = static_cast<const uint8_t*>(k_fp4);
    a.k_sf = static_cast<const uint8_t*>(k_sf);
    a.v_fp4 = static_cast<const uint8_t*>(v_fp4);
    a.v_sf = static_cast<const uint8_t*>(v_sf);
    a.block_table = block_table;
    a.qo_indptr = qo_indptr;
    a.kv_lens = kv_lens;
    a.out = static_cast<uint8_t*>(out_fp8);
    cudaError_t e = gqa::launch_ctx(a, plan, part, stream);
    if (e == cudaErrorNotSupported) return fail(GQA_ERR_UNSUPPORTED, "context kernel not available in this build");
    GQA_CUDA_TRY(e, "ctx launch");
    return GQA_OK;
  }

  // Host buffers: the host can read the metadata, so check it fully.
  if (qo_indptr[0] != 0 || qo_indptr[batch] != total_q)
    return fail(GQA_ERR_INVALID_ARG, "qo_indptr must start at 0 and end at total_q");
  for (int64_t b = 0; b < batch; ++b) {
    if (qo_indptr[b + 1] < qo_indptr[b]) return fail(GQA_ERR_INVALID_ARG, "qo_indptr decreases at %lld", (long long)b);
    if (kv_lens[b] < 0 || (int64_t)kv_lens[b] > 64 * max_pages_per_seq)
      return fail(GQA_ERR_INVALID_ARG, "kv_lens[%lld] = %d out of range", (long long)b, kv_lens[b]);
    const int64_t np = ((int64_t)kv_lens[b] + 63) / 64;
    for (int64_t p = 0; p < np; ++p) {
      const int32_t pg = block_table[b * max_pages_per_seq + p];
      if (pg < 0 || pg >= num_pages)
        return fail(GQA_ERR_INVALID_ARG, "block_table[%lld][%lld] = %d outside [0, num_pages)", (long long)b,
                    (long long)p, pg);
    }
  }
  if (total_q == 0) return GQA_OK;
  int dev = 0;
  GQA_CUDA_TRY(cudaGetDevice(&dev), "cudaGetDevice");
  const size_t q_bytes = (size_t)total_q * 32 * 128;
  const size_t fp4_bytes = (size_t)num_pages * 8 * 64 * 64;
  const size_t sf_bytes = (size_t)num_pages * 8 * 64 * 8;
  const size_t bt_bytes = (size_t)batch * max_pages_per_seq * 4;
  Carver c;
  const size_t o_q = c.take(q_bytes), o_kf = c.take(fp4_bytes), o_ks = c.take(sf_bytes), o_vf = c.take(fp4_bytes),
               o_vs = c.take(sf_bytes), o_bt = c.take(bt_bytes), o_qi = c.take((size_t)(batch + 1) * 4),
               o_kl = c.take((size_t)batch * 4), o_out = c.take(q_bytes), o_part = c.take(part_bytes);
  void* ws = nullptr;
  if ((st = workspace(dev, stream, c.off, &ws)) != GQA_OK) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  const std::pair<size_t, std::pair<const void*, size_t>> copies[] = {
      {o_q, {q_fp8, q_bytes}},  {o_kf, {k_fp4, fp4_bytes}}, {o_ks, {k_sf, sf_bytes}},
      {o_vf, {v_fp4, fp4_bytes}}, {o_vs, {v_sf, sf_bytes}},   {o_bt, {block_table, bt_bytes}},
      {o_qi, {qo_indptr, (size_t)(batch + 1) * 4}}, {o_kl, {kv_lens, (size_t)batch * 4}}};
  for (const auto& cp : copies)
    GQA_CUDA_TRY(cudaMemcpyAsync(base + cp.first, cp.second.first, cp.second.second, cudaMemcpyHostToDevice, stream),
                 "stage input");
  a.q = base + o_q;
  a.k_fp4 = base + o_kf;
  a.k_sf = base + o_ks;
  a.v_fp4 = base + o_vf;
  a.v_sf = base + o_vs;
  a.block_table = reinterpret_cast<const int32_t*>(base + o_bt);
  a.qo_indptr = reinterpret_cast<const int32_t*>(base + o_qi);
  a.kv_lens = reinterpret_cast<const int32_t*>(base + o_kl);
  a.out = base + o_out;
  cudaError_t e = gqa::launch_ctx(a, plan, part_bytes ? base + o_part : nullptr, stream);
  if (e == cudaErrorNotSupported) return fail(GQA_ERR_UNSUPPORTED, "context kernel not available in this build");
  GQA_CUDA_TRY(e, "ctx launch");
  GQA_CUDA_TRY(cudaMemcpyAsync(out_fp8, base + o_out, q_bytes, cudaMemcpyDeviceToHost, stream), "copy out");
  GQA_CUDA_TRY(cudaStreamSynchronize(stream), "cudaStreamSynchronize");
  return GQA_OK;
}
}  // namespace

gqa_status nvfp4_paged_ctx_attn(const void* q_fp8, float q_scale, const void* k_fp4, const void* k_sf,
                                const void* v_fp4, const void* v_sf, const int32_t* block_table,
                                const int32_t* qo_indptr, const int32_t* kv_lens, void* out_fp8, float out_scale,
                                int64_t batch, int64_t total_q, int64_t num_pages, int64_t max_pages_per_seq,
                                gqa_stream_t stream) {
  return ctx_impl(q_fp8, q_scale, k_fp4, k_sf, v_fp4, v_sf, block_table, qo_indptr, kv_lens, out_fp8, out_scale,
                  batch, total_q, num_pages, max_pages_per_seq, stream, kAnyDevice);
}

gqa_status gqa_debug_dequant_pages(const void* fp4, const void* sf, const int32_t* block_table,
                                   const int32_t* kv_lens, void* out_e4m3, int64_t batch, int64_t num_pages,
                                   int64_t max_pages_per_seq, int64_t max_kv, gqa_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (batch < 1 || batch > 65535) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 65535]", (long long)batch);
  if (num_pages < 1 || max_pages_per_seq < 1 || max_kv < 1 || max_kv > 64 * max_pages_per_seq)
    return fail(GQA_ERR_INVALID_ARG, "bad num_pages / max_pages_per_seq / max_kv");
  Where where;
  gqa_status st = locate({{fp4, "fp4", 16}, {sf, "sf", 16}, {block_table, "block_table", 4},
                          {kv_lens, "kv_lens", 4}, {out_e4m3, "out_e4m3", 16}},
                         &where);
  if (st != GQA_OK) return st;
  if (where.host) return fail(GQA_ERR_UNSUPPORTED, "gqa_debug_dequant_pages takes device pointers only");
  ScopedDevice sd(where.device);
  if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
  GQA_CUDA_TRY(gqa::launch_dequant_pages(static_cast<const uint8_t*>(fp4), static_cast<const uint8_t*>(sf),
                                         block_table, kv_lens, static_cast<uint8_t*>(out_e4m3), batch, num_pages,
                                         max_pages_per_seq, max_kv, stream),
               "dequant launch");
  return GQA_OK;
}

gqa_status gqa_debug_wait_expiry(int device, gqa_stream_t stream) {
  ScopedDevice sd(device);
  if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", device);
  GQA_CUDA_TRY(gqa::launch_wait_expiry(reinterpret_cast<cudaStream_t>(stream)), "wait-expiry launch");
  return GQA_OK;
}

gqa_status gqa_set_schedule(int ctx_packed_stages, int ctx_kv_slots, int decode_stages) {
  if (!gqa::ctx_schedule_supported(ctx_packed_stages, ctx_kv_slots))
    return fail(GQA_ERR_UNSUPPORTED,
                "context ring depths (%d packed stages, %d K/V slots) are not instantiated; see gqa.h", ctx_packed_stages,
                ctx_kv_slots);
  if (!gqa::decode_schedule_supported(decode_stages))
    return fail(GQA_ERR_UNSUPPORTED, "decode ring depth %d is not instantiated (0, 4, 8, 12 or 16)", decode_stages);
  g_ctx_stages.store(ctx_packed_stages, std::memory_order_relaxed);
  g_ctx_slots.store(ctx_kv_slots, std::memory_order_relaxed);
  g_decode_stages.store(decode_stages, std::memory_order_relaxed);
  return GQA_OK;
}

gqa_status gqa_set_ctx_grid(int mode) {
  if (mode < GQA_CTX_GRID_PLANNED || mode > GQA_CTX_GRID_DECODE_SHAPED)
    return fail(GQA_ERR_INVALID_ARG, "context grid mode %d is not 0, 1, 2 or 3", mode);
  g_ctx_grid.store(mode, std::memory_order_relaxed);
  return GQA_OK;
}

gqa_status gqa_debug_starve_producers(int enable) {
  g_starve.store(enable ? 1 : 0, std::memory_order_relaxed);
  return GQA_OK;
}

gqa_status gqa_check_device_errors(int device, uint32_t* word) {
  if (!word) return fail(GQA_ERR_INVALID_ARG, "word is a null pointer");
  *word = 0;
  ScopedDevice sd(device);
  if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", device);
  uint32_t a = 0, b = 0, c = 0, d = 0, f = 0;
  GQA_CUDA_TRY(gqa::decode_read_errors(&a), "read decode error word");
  GQA_CUDA_TRY(gqa::ctx_read_errors(&b), "read ctx error word");
  GQA_CUDA_TRY(gqa::ctx_study_read_errors(&c), "read ctx study error word");
  GQA_CUDA_TRY(gqa::append_read_errors(&d), "read append error word");
  GQA_CUDA_TRY(gqa::paged_attn_read_errors(&f), "read paged attention error word");
  *word = a | b | c | d | f;
  if (*word & 1u) return fail(GQA_ERR_TIMEOUT, "a kernel's bounded wait expired (error word 0x%x)", *word);
  if (*word)
    return fail(GQA_ERR_INVALID_ARG,
                "a kernel met invalid metadata: bit 1 = out-of-range page index skipped, bit 2 = qo_indptr not "
                "non-decreasing from 0 to total_q, bit 3 = dequantisation self-check (error word 0x%x)",
                *word);
  return GQA_OK;
}

// ---- descriptor forms of the three operations --------------------------------

gqa_status gqa_decode_t(const gqa_tensor* q, const gqa_tensor* kv, const gqa_tensor* seq_lens, gqa_tensor* out,
                        float q_scale, gqa_stream_t stream) {
  int64_t qs[3], ks[5];
  GQA_TRY(check_desc(q, "q", {GQA_F16}, {-1, 32, 128}, qs));
  GQA_TRY(check_desc(kv, "kv", {GQA_F16}, {qs[0], 2, 8, -1, 128}, ks));
  GQA_TRY(check_desc(seq_lens, "seq_lens", {GQA_I32}, {qs[0]}));
  GQA_TRY(check_desc(out, "out", {GQA_F16}, {qs[0], 32, 128}));
  GQA_TRY(check_devices({{q, "q"}, {kv, "kv"}, {seq_lens, "seq_lens"}, {out, "out"}}));
  return decode_impl(q->data, kv->data, static_cast<const int32_t*>(seq_lens->data), out->data, qs[0], ks[3], q_scale,
                     stream, q->device);
}

gqa_status gqa_decode_paged_t(const gqa_tensor* q, const gqa_tensor* k_pages, const gqa_tensor* v_pages,
                              const gqa_tensor* block_table, const gqa_tensor* seq_lens, gqa_tensor* out,
                              float q_scale, gqa_stream_t stream) {
  int64_t qs[3], ps[4], bs[2];
  GQA_TRY(check_desc(q, "q", {GQA_F16}, {-1, 32, 128}, qs));
  GQA_TRY(check_desc(k_pages, "k_pages", {GQA_F16}, {-1, 8, 64, 128}, ps));
  GQA_TRY(check_desc(v_pages, "v_pages", {GQA_F16}, {ps[0], 8, 64, 128}));
  GQA_TRY(check_desc(block_table, "block_table", {GQA_I32}, {qs[0], -1}, bs));
  GQA_TRY(check_desc(seq_lens, "seq_lens", {GQA_I32}, {qs[0]}));
  GQA_TRY(check_desc(out, "out", {GQA_F16}, {qs[0], 32, 128}));
  GQA_TRY(check_devices({{q, "q"}, {k_pages, "k_pages"}, {v_pages, "v_pages"}, {block_table, "block_table"},
                         {seq_lens, "seq_lens"}, {out, "out"}}));
  return decode_paged_impl(q->data, k_pages->data, v_pages->data, static_cast<const int32_t*>(block_table->data),
                           static_cast<const int32_t*>(seq_lens->data), out->data, qs[0], ps[0], bs[1], q_scale, stream,
                           q->device);
}

gqa_status nvfp4_paged_ctx_attn_t(const gqa_tensor* q_fp8, float q_scale, const gqa_tensor* k_fp4,
                                  const gqa_tensor* k_sf, const gqa_tensor* v_fp4, const gqa_tensor* v_sf,
                                  const gqa_tensor* block_table, const gqa_tensor* qo_indptr,
                                  const gqa_tensor* kv_lens, gqa_tensor* out_fp8, float out_scale,
                                  gqa_stream_t stream) {
  int64_t qs[3], ps[4], ls[1], bs[2];
  GQA_TRY(check_desc(q_fp8, "q_fp8", {GQA_E4M3, GQA_U8}, {-1, 32, 128}, qs));
  GQA_TRY(check_desc(k_fp4, "k_fp4", {GQA_U8}, {-1, 8, 64, 64}, ps));
  GQA_TRY(check_desc(k_sf, "k_sf", {GQA_E4M3, GQA_U8}, {ps[0], 8, 64, 8}));
  GQA_TRY(check_desc(v_fp4, "v_fp4", {GQA_U8}, {ps[0], 8, 64, 64}));
  GQA_TRY(check_desc(v_sf, "v_sf", {GQA_E4M3, GQA_U8}, {ps[0], 8, 64, 8}));
  GQA_TRY(check_desc(kv_lens, "kv_lens", {GQA_I32}, {-1}, ls));
  GQA_TRY(check_desc(qo_indptr, "qo_indptr", {GQA_I32}, {ls[0] + 1}));
  GQA_TRY(check_desc(block_table, "block_table", {GQA_I32}, {ls[0], -1}, bs));
  GQA_TRY(check_desc(out_fp8, "out_fp8", {GQA_E4M3, GQA_U8}, {qs[0], 32, 128}));
  GQA_TRY(check_devices({{q_fp8, "q_fp8"}, {k_fp4, "k_fp4"}, {k_sf, "k_sf"}, {v_fp4, "v_fp4"}, {v_sf, "v_sf"},
                         {block_table, "block_table"}, {qo_indptr, "qo_indptr"}, {kv_lens, "kv_lens"},
                         {out_fp8, "out_fp8"}}));
  return ctx_impl(q_fp8->data, q_scale, k_fp4->data, k_sf->data, v_fp4->data, v_sf->data,
                  static_cast<const int32_t*>(block_table->data), static_cast<const int32_t*>(qo_indptr->data),
                  static_cast<const int32_t*>(kv_lens->data), out_fp8->data, out_scale, ls[0], qs[0], ps[0], bs[1],
                  stream, q_fp8->device);
}

// ---- paged cache of any layout: append, one-token attention -------------------

namespace {

int64_t dtype_bytes(int32_t d) {
  return d == GQA_F16 || d == GQA_BF16 ? 2 : d == GQA_E4M3 || d == GQA_U8 ? 1 : 4;
}

// Structural check of a tensor that may be strided: as check_desc, but the last
// dimension alone has to be dense and the other strides are multiples of 16 bytes;
// one that is written must not overlap itself.  An empty tensor may have no data.
gqa_status check_strided(const gqa_tensor* t, const char* name, std::initializer_list<int32_t> dtypes,
                         std::initializer_list<int64_t> shape, bool written, int64_t* got = nullptr) {
  if (!t) return fail(GQA_ERR_INVALID_ARG, "%s: null descriptor", name);
  gqa_tensor dense = *t;  // the checks that do not depend on the strides
  int64_t n = 1;
  if (t->ndim >= 0 && t->ndim <= 6)
    for (int d = t->ndim - 1; d >= 0; --d) {
      dense.strides[d] = n;
      if (t->shape[d] >= 0 && t->shape[d] <= (int64_t(1) << 40) && n <= (int64_t(1) << 40)) n *= t->shape[d];
    }
  if (!dense.data && n == 0) dense.data = &dense;
  GQA_TRY(check_desc(&dense, name, dtypes, shape, got));
  const int64_t esz = dtype_bytes(t->dtype);
  const int nd = t->ndim;
  if (t->shape[nd - 1] > 1 && t->strides[nd - 1] != 1)
    return fail(GQA_ERR_INVALID_ARG, "%s: the last dimension is not dense (stride %lld)", name, (long long)t->strides[nd - 1]);
  for (int d = 0; d < nd - 1; ++d) {
    if (t->shape[d] <= 1) continue;
    if (t->strides[d] < 0 || t->strides[d] > (int64_t(1) << 38) || t->strides[d] * esz % 16 != 0)
      return fail(GQA_ERR_INVALID_ARG, "%s: stride %lld in dimension %d is not a multiple of 16 bytes in [0, 2^38]", name,
                  (long long)t->strides[d], d);
  }
  if (!written) return GQA_OK;
  // Dimensions from the smallest stride up: each steps over all that the smaller ones cover.
  __int128 covered = t->shape[nd - 1];
  bool used[6] = {};
  for (int k = 0; k < nd - 1; ++k) {
    int at = -1;
    for (int d = 0; d < nd - 1; ++d)
      if (!used[d] && t->shape[d] > 1 && (at < 0 || t->strides[d] < t->strides[at])) at = d;
    if (at < 0) break;
    used[at] = true;
    if (t->strides[at] < covered)
      return fail(GQA_ERR_INVALID_ARG, "%s overlaps itself (stride %lld in dimension %d)", name, (long long)t->strides[at], at);
    covered += (__int128)t->strides[at] * (t->shape[at] - 1);
  }
  return GQA_OK;
}

// Stride of a dimension; 0 where its extent is 1 (nothing is ever added for it).
int64_t stride_of(const gqa_tensor* t, int d) { return t->shape[d] > 1 ? t->strides[d] : 0; }

gqa_status check_scale(float s, const char* name) {
  if (!std::isfinite(s) || !(s > 0.f) || !std::isfinite(1.f / s))
    return fail(GQA_ERR_INVALID_ARG, "%s must be finite and > 0", name);
  return GQA_OK;
}

using Named = std::pair<const gqa_tensor*, const char*>;

// What the two appends share: q, k, v, q_out, the metadata and the rope table; fills
// in everything but the pages.  Null q, q_out, indptr and rope are left out.
gqa_status append_common(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, const gqa_tensor* block_table,
                         const gqa_tensor* kv_lens, const gqa_tensor* indptr, const gqa_tensor* rope, const gqa_tensor* q_out,
                         std::initializer_list<int32_t> out_dtypes, int64_t hq, int64_t hkv, int64_t dim, int rot_step,
                         int interleaved, gqa::AppendArgs* a, std::vector<Named>* ts) {
  int64_t ks[3], qs[3], ls[1], bs[2], rs[2];
  GQA_TRY(check_strided(k, "k", {GQA_F16, GQA_BF16}, {-1, hkv, dim}, false, ks));
  GQA_TRY(check_strided(v, "v", {k->dtype}, {ks[0], ks[1], ks[2]}, false));
  if (ks[2] != 64 && ks[2] != 128 && ks[2] != 256)
    return fail(GQA_ERR_UNSUPPORTED_SHAPE, "head dim %lld is not 64, 128 or 256", (long long)ks[2]);
  if (ks[1] < 1 || ks[1] > 1024) return fail(GQA_ERR_UNSUPPORTED_SHAPE, "%lld KV heads: 1 to 1024 are taken", (long long)ks[1]);
  if (ks[0] > 2147483647LL) return fail(GQA_ERR_INVALID_ARG, "total %lld out of range", (long long)ks[0]);
  if ((q == nullptr) != (q_out == nullptr)) return fail(GQA_ERR_INVALID_ARG, "q and q_out go together: one of them is NULL");
  *ts = {{k, "k"}, {v, "v"}, {block_table, "block_table"}, {kv_lens, "kv_lens"}};
  if (q) {
    GQA_TRY(check_strided(q, "q", {k->dtype}, {ks[0], hq, ks[2]}, false, qs));
    if (qs[1] < 1 || qs[1] > 1024) return fail(GQA_ERR_UNSUPPORTED_SHAPE, "%lld query heads: 1 to 1024 are taken", (long long)qs[1]);
    GQA_TRY(check_strided(q_out, "q_out", out_dtypes, {ks[0], qs[1], ks[2]}, true));
    if (q_out->data && q_out->data == q->data)
      for (int d = 0; d < 2; ++d)
        if (q_out->dtype != q->dtype || stride_of(q, d) != stride_of(q_out, d))
          return fail(GQA_ERR_INVALID_ARG, "q_out may be q itself, with q's type and strides");
    ts->push_back({q, "q"});
    ts->push_back({q_out, "q_out"});
  }
  GQA_TRY(check_desc(kv_lens, "kv_lens", {GQA_I32}, {-1}, ls));
  if (ls[0] < 1 || ls[0] > (1 << 20)) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 2^20]", (long long)ls[0]);
  GQA_TRY(check_desc(block_table, "block_table", {GQA_I32}, {ls[0], -1}, bs));
  if (indptr) {
    GQA_TRY(check_desc(indptr, "qo_indptr", {GQA_I32}, {ls[0] + 1}));
    ts->push_back({indptr, "qo_indptr"});
  } else if (ks[0] != ls[0]) {
    return fail(GQA_ERR_INVALID_ARG, "without qo_indptr there is one token per sequence: %lld tokens, %lld sequences",
                (long long)ks[0], (long long)ls[0]);
  }
  *a = gqa::AppendArgs{};
  if (rope) {
    GQA_TRY(check_desc(rope, "rope", {GQA_F32}, {-1, -1}, rs));
    if (rs[1] < rot_step || rs[1] > ks[2] || rs[1] % rot_step != 0)
      return fail(GQA_ERR_UNSUPPORTED_SHAPE, "rope has %lld columns; a multiple of %d up to the head dim is wanted",
                  (long long)rs[1], rot_step);
    a->rope = static_cast<const float*>(rope->data);
    a->rope_len = rs[0];
    a->rot = (int)rs[1];
    ts->push_back({rope, "rope"});
  }
  a->interleaved = interleaved ? 1 : 0;
  a->k = k->data;
  a->v = v->data;
  a->block_table = static_cast<const int32_t*>(block_table->data);
  a->kv_lens = static_cast<const int32_t*>(kv_lens->data);
  a->indptr = indptr ? static_cast<const int32_t*>(indptr->data) : nullptr;
  a->k_tok = stride_of(k, 0);
  a->k_head = stride_of(k, 1);
  a->v_tok = stride_of(v, 0);
  a->v_head = stride_of(v, 1);
  if (q) {
    a->q = q->data;
    a->q_out = q_out->data;
    a->q_tok = stride_of(q, 0);
    a->q_head = stride_of(q, 1);
    a->qo_tok = stride_of(q_out, 0);
    a->qo_head = stride_of(q_out, 1);
    a->hq = (int)qs[1];
  }
  a->hkv = (int)ks[1];
  a->d = (int)ks[2];
  a->total = ks[0];
  a->batch = ls[0];
  a->max_pages_per_seq = bs[1];
  a->bf16 = k->dtype == GQA_BF16;
  a->inv_k = a->inv_v = a->inv_q = 1.f;
  return GQA_OK;
}

// All tensors on one device, where their descriptors say, 16-byte aligned (int32 ones
// 4-byte); host memory is refused.
gqa_status locate_tensors(const std::vector<Named>& ts, const char* op, Where* where) {
  std::vector<Arg> args;
  for (const Named& t : ts) {
    if (t.first->device != ts[0].first->device)
      return fail(GQA_ERR_DEVICE_MISMATCH, "%s is on device %d but %s is on device %d", t.second, t.first->device, ts[0].second,
                  ts[0].first->device);
    args.push_back({t.first->data, t.second, t.first->dtype == GQA_I32 ? size_t(4) : size_t(16)});
  }
  if (ts[0].first->device < 0) return fail(GQA_ERR_UNSUPPORTED, "%s takes device tensors only", op);
  GQA_TRY(locate(args, where, ts[0].first->device));
  return GQA_OK;
}

gqa_status run_append(const gqa::AppendArgs& a, const std::vector<Named>& ts, const char* op, gqa_stream_t stream) {
  if (a.total == 0) return GQA_OK;
  if (a.num_pages < 1 || a.num_pages > 2147483647LL) return fail(GQA_ERR_INVALID_ARG, "num_pages %lld out of range", (long long)a.num_pages);
  if (a.max_pages_per_seq < 1) return fail(GQA_ERR_INVALID_ARG, "block_table has no column");
  if (a.rope && a.rope_len < 1) return fail(GQA_ERR_INVALID_ARG, "rope has no row");
  Where where;
  GQA_TRY(locate_tensors(ts, op, &where));
  ScopedDevice sd(where.device);
  if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
  GQA_CUDA_TRY(gqa::launch_append(a, reinterpret_cast<cudaStream_t>(stream)), "append launch");
  return GQA_OK;
}

}  // namespace

gqa_status gqa_paged_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_pages,
                              gqa_tensor* v_pages, const gqa_tensor* block_table, const gqa_tensor* kv_lens,
                              const gqa_tensor* qo_indptr, const gqa_tensor* rope, gqa_tensor* q_out, int interleaved,
                              float k_scale, float v_scale, gqa_stream_t stream) {
  return guarded([&]() -> gqa_status {
    gqa::AppendArgs a;
    std::vector<Named> ts;
    if (!k) return fail(GQA_ERR_INVALID_ARG, "k: null descriptor");
    GQA_TRY(append_common(q, k, v, block_table, kv_lens, qo_indptr, rope, q_out, {k->dtype}, -1, -1, -1, 16, interleaved, &a, &ts));
    int64_t ps[4];
    GQA_TRY(check_strided(k_pages, "k_pages", {k->dtype, GQA_E4M3, GQA_U8}, {-1, a.hkv, -1, a.d}, true, ps));
    const bool e4m3 = k_pages->dtype != k->dtype;
    GQA_TRY(e4m3 ? check_strided(v_pages, "v_pages", {GQA_E4M3, GQA_U8}, {ps[0], a.hkv, ps[2], a.d}, true)
                 : check_strided(v_pages, "v_pages", {k->dtype}, {ps[0], a.hkv, ps[2], a.d}, true));
    if (a.total > 0 && (ps[2] < 1 || ps[2] > (1 << 20)))
      return fail(GQA_ERR_UNSUPPORTED_SHAPE, "page size %lld outside [1, 2^20]", (long long)ps[2]);
    GQA_TRY(check_scale(k_scale, "k_scale"));
    GQA_TRY(check_scale(v_scale, "v_scale"));
    if (!e4m3 && (k_scale != 1.f || v_scale != 1.f))
      return fail(GQA_ERR_INVALID_ARG, "k_scale and v_scale belong to E4M3 pages: 1 is wanted");
    a.mode = e4m3 ? gqa::kAppendE4m3 : gqa::kAppendSame;
    a.inv_k = 1.f / k_scale;
    a.inv_v = 1.f / v_scale;
    a.k_pages = k_pages->data;
    a.v_pages = v_pages->data;
    a.kp_page = stride_of(k_pages, 0);
    a.kp_head = stride_of(k_pages, 1);
    a.kp_slot = stride_of(k_pages, 2);
    a.vp_page = stride_of(v_pages, 0);
    a.vp_head = stride_of(v_pages, 1);
    a.vp_slot = stride_of(v_pages, 2);
    a.num_pages = ps[0];
    a.page_size = (int)ps[2];
    ts.push_back({k_pages, "k_pages"});
    ts.push_back({v_pages, "v_pages"});
    return run_append(a, ts, "gqa_paged_append", stream);
  });
}

gqa_status nvfp4_paged_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_fp4,
                                gqa_tensor* k_sf, gqa_tensor* v_fp4, gqa_tensor* v_sf, const gqa_tensor* block_table,
                                const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, const gqa_tensor* rope,
                                gqa_tensor* q_out, int interleaved, float q_scale, gqa_stream_t stream) {
  return guarded([&]() -> gqa_status {
    gqa::AppendArgs a;
    std::vector<Named> ts;
    if (!k) return fail(GQA_ERR_INVALID_ARG, "k: null descriptor");
    GQA_TRY(append_common(q, k, v, block_table, kv_lens, qo_indptr, rope, q_out, {GQA_E4M3, GQA_U8}, 32, 8, 128, 32, interleaved, &a,
                          &ts));
    int64_t ps[4];
    GQA_TRY(check_desc(k_fp4, "k_fp4", {GQA_U8}, {-1, 8, 64, 64}, ps));
    GQA_TRY(check_desc(k_sf, "k_sf", {GQA_E4M3, GQA_U8}, {ps[0], 8, 64, 8}));
    GQA_TRY(check_desc(v_fp4, "v_fp4", {GQA_U8}, {ps[0], 8, 64, 64}));
    GQA_TRY(check_desc(v_sf, "v_sf", {GQA_E4M3, GQA_U8}, {ps[0], 8, 64, 8}));
    GQA_TRY(check_scale(q_scale, "q_scale"));
    a.mode = gqa::kAppendNvfp4;
    a.inv_q = 1.f / q_scale;
    a.k_pages = k_fp4->data;
    a.v_pages = v_fp4->data;
    a.k_sf = static_cast<uint8_t*>(k_sf->data);
    a.v_sf = static_cast<uint8_t*>(v_sf->data);
    a.num_pages = ps[0];
    a.page_size = 64;
    for (const Named& t : {Named{k_fp4, "k_fp4"}, Named{k_sf, "k_sf"}, Named{v_fp4, "v_fp4"}, Named{v_sf, "v_sf"}}) ts.push_back(t);
    return run_append(a, ts, "nvfp4_paged_append", stream);
  });
}

int64_t gqa_paged_attn_workspace(int64_t q_heads, int64_t kv_heads, int64_t d) {
  if (kv_heads < 1 || q_heads < 1 || q_heads > 1024 || q_heads % kv_heads != 0 || (d != 64 && d != 128 && d != 256)) return 0;
  return (int64_t)gqa::paged_attn_workspace_bytes((int)q_heads, (int)kv_heads, (int)d);
}

gqa_status gqa_paged_attn_t(const gqa_tensor* q, const gqa_tensor* k_pages, const gqa_tensor* v_pages,
                            const gqa_tensor* block_table, const gqa_tensor* seq_lens, gqa_tensor* out, gqa_tensor* lse,
                            float q_scale, float k_scale, float v_scale, int window, float softcap, void* workspace_,
                            int64_t workspace_bytes, gqa_stream_t stream) {
  return guarded([&]() -> gqa_status {
    int64_t qs[3], ps[4], bs[2];
    GQA_TRY(check_strided(q, "q", {GQA_F16, GQA_BF16}, {-1, -1, -1}, false, qs));
    GQA_TRY(check_strided(k_pages, "k_pages", {q->dtype, GQA_E4M3, GQA_U8}, {-1, -1, -1, qs[2]}, true, ps));
    const bool e4m3 = k_pages->dtype != q->dtype;
    GQA_TRY(e4m3 ? check_strided(v_pages, "v_pages", {GQA_E4M3, GQA_U8}, {ps[0], ps[1], ps[2], qs[2]}, true)
                 : check_strided(v_pages, "v_pages", {q->dtype}, {ps[0], ps[1], ps[2], qs[2]}, true));
    GQA_TRY(check_desc(seq_lens, "seq_lens", {GQA_I32}, {qs[0]}));
    GQA_TRY(check_desc(block_table, "block_table", {GQA_I32}, {qs[0], -1}, bs));
    GQA_TRY(check_desc(out, "out", {q->dtype}, {qs[0], qs[1], qs[2]}));
    if (lse) GQA_TRY(check_desc(lse, "lse", {GQA_F32}, {qs[0], qs[1]}));
    if (qs[0] < 1 || qs[0] > 65535) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 65535]", (long long)qs[0]);
    if (qs[2] != 64 && qs[2] != 128 && qs[2] != 256)
      return fail(GQA_ERR_UNSUPPORTED_SHAPE, "head dim %lld is not 64, 128 or 256", (long long)qs[2]);
    if (ps[1] < 1 || qs[1] < 1 || qs[1] > 1024 || qs[1] % ps[1] != 0)
      return fail(GQA_ERR_UNSUPPORTED_SHAPE, "%lld query heads over %lld KV heads: 1 to 1024, a multiple, are taken",
                  (long long)qs[1], (long long)ps[1]);
    if (ps[2] != 16 && ps[2] != 32 && ps[2] != 64 && ps[2] != 128 && ps[2] != 256)
      return fail(GQA_ERR_UNSUPPORTED_SHAPE, "page size %lld is not 16, 32, 64, 128 or 256", (long long)ps[2]);
    if (ps[0] < 1 || ps[0] > 2147483647LL) return fail(GQA_ERR_INVALID_ARG, "num_pages %lld out of range", (long long)ps[0]);
    if (bs[1] < 1 || bs[1] > (int64_t(1) << 30) / ps[2])
      return fail(GQA_ERR_INVALID_ARG, "max_pages_per_seq %lld out of range", (long long)bs[1]);
    // (a block of the kernel counts the work of its share, in tiles of 32 tokens at least, in 31 bits)
    if (qs[0] * ps[1] * ((qs[1] / ps[1] + 7) / 8) > (int64_t(1) << 38) / (bs[1] * ps[2] / 32 + 16))
      return fail(GQA_ERR_UNSUPPORTED, "batch %lld x %lld KV heads x %lld tokens of capacity are too many", (long long)qs[0],
                  (long long)ps[1], (long long)(bs[1] * ps[2]));
    if (!std::isfinite(q_scale)) return fail(GQA_ERR_INVALID_ARG, "q_scale is not finite");
    GQA_TRY(check_scale(k_scale, "k_scale"));
    GQA_TRY(check_scale(v_scale, "v_scale"));
    if (window < 0) return fail(GQA_ERR_INVALID_ARG, "window %d is negative", window);
    if (!std::isfinite(softcap) || softcap < 0.f) return fail(GQA_ERR_INVALID_ARG, "softcap must be finite and >= 0");
    const int64_t need = gqa_paged_attn_workspace(qs[1], ps[1], qs[2]);
    if (workspace_ && workspace_bytes < need)
      return fail(GQA_ERR_INVALID_ARG, "workspace of %lld bytes; %lld are needed", (long long)workspace_bytes, (long long)need);
    gqa_tensor ws = *q;  // the workspace's place is checked with the tensors'
    ws.data = workspace_;
    std::vector<Named> ts = {{q, "q"}, {k_pages, "k_pages"}, {v_pages, "v_pages"}, {block_table, "block_table"},
                             {seq_lens, "seq_lens"}, {out, "out"}};
    if (workspace_) ts.push_back({&ws, "workspace"});
    gqa_tensor l;
    if (lse) {
      l = *lse;
      l.dtype = GQA_I32;  // (4-byte alignment)
      ts.push_back({&l, "lse"});
    }
    Where where;
    GQA_TRY(locate_tensors(ts, "gqa_paged_attn", &where));
    gqa::PagedAttnArgs a{};
    a.q = q->data;
    a.out = out->data;
    a.lse = lse ? static_cast<float*>(lse->data) : nullptr;
    a.k_pages = k_pages->data;
    a.v_pages = v_pages->data;
    a.block_table = static_cast<const int32_t*>(block_table->data);
    a.seq_lens = static_cast<const int32_t*>(seq_lens->data);
    a.q_seq = stride_of(q, 0);
    a.q_head = stride_of(q, 1);
    a.kp_page = k_pages->strides[0];
    a.kp_head = k_pages->strides[1];
    a.kp_slot = k_pages->strides[2];
    a.vp_page = v_pages->strides[0];
    a.vp_head = v_pages->strides[1];
    a.vp_slot = v_pages->strides[2];
    a.batch = qs[0];
    a.num_pages = ps[0];
    a.max_pages_per_seq = bs[1];
    a.hq = (int)qs[1];
    a.hkv = (int)ps[1];
    a.d = (int)qs[2];
    a.page_size = (int)ps[2];
    const bool bf16 = q->dtype == GQA_BF16;
    a.cache = e4m3 ? (bf16 ? gqa::kCacheE4m3 : gqa::kCacheE4m3F16) : bf16 ? gqa::kCacheBf16 : gqa::kCacheF16;
    a.scale = (float)((double)q_scale * k_scale / std::sqrt((double)qs[2]));
    a.v_scale = v_scale;
    a.softcap = softcap;
    a.window = window;
    a.starve = gqa::starve_producers();
    if (!std::isfinite(a.scale) || (softcap > 0.f && !std::isfinite((float)(4.0 * a.scale / softcap))))
      return fail(GQA_ERR_INVALID_ARG, "q_scale * k_scale (over softcap) is out of range");
    ScopedDevice sd(where.device);
    if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // A call's two kernels follow each other on the stream: another thread's call on the
    // same stream, and so with the same workspace, must not come between them.
    std::lock_guard<std::mutex> lk(g_paged_launch_mu);
    if (!workspace_) {
      cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
      GQA_CUDA_TRY(cudaStreamIsCapturing(s, &capture), "cudaStreamIsCapturing");
      if (capture != cudaStreamCaptureStatusNone)
        return fail(GQA_ERR_WORKSPACE, "a captured call needs a workspace of its own (%lld bytes)", (long long)need);
      if (s == cudaStreamPerThread) {
        static thread_local ThreadEnd end;
        end.thread = gqa::thread_number();
      }
      // As much as the largest head layout needs, so that it never moves; and allocated
      // without disturbing a capture of another thread.
      cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
      GQA_CUDA_TRY(cudaThreadExchangeStreamCaptureMode(&mode), "cudaThreadExchangeStreamCaptureMode");
      const gqa_status st = workspace(where.device, s, gqa::paged_attn_workspace_bytes(1024, 1, 256), &workspace_, g_paged_ws);
      cudaThreadExchangeStreamCaptureMode(&mode);
      GQA_TRY(st);
    }
    GQA_CUDA_TRY(gqa::launch_paged_attn(a, workspace_, s), "paged attention launch");
    return GQA_OK;
  });
}

gqa_status gqa_release_workspace(void) {
  std::lock_guard<std::mutex> lk(g_ws_mu);
  int prev = -1;
  cudaGetDevice(&prev);
  for (WorkspaceMap* map : {&g_ws, &g_paged_ws}) {
    for (auto& kv : *map) {
      if (kv.second.ptr) {
        cudaSetDevice(std::get<0>(kv.first));
        cudaFree(kv.second.ptr);
      }
    }
    map->clear();
  }
  if (prev >= 0) cudaSetDevice(prev);
  return GQA_OK;
}

}  // extern "C"
