// api_paged.cpp -- the C ABI of the paged caches of any layout (include/gqa.h): checks of
// the descriptors, workspaces and launches of the appends, the attentions and what drafted tokens need.
#include "api_util.h"
#include "kernels.h"
#include "paged.h"

using namespace gqa::api;
namespace {

int64_t dtype_bytes(int32_t d) {
  return d == GQA_F16 || d == GQA_BF16 ? 2 : d == GQA_E4M3 || d == GQA_U8 ? 1 : 4;
}

// Structural check of a tensor that may be strided: as check_desc, but the last
// dimension alone has to be dense and the other strides are multiples of `step` bytes;
// one that is written must not overlap itself.  An empty tensor may have no data.
gqa_status check_strided(const gqa_tensor* t, const char* name, std::initializer_list<int32_t> dtypes,
                         std::initializer_list<int64_t> shape, bool written, int64_t* got = nullptr, int step = 16) {
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
    if (t->strides[d] < 0 || t->strides[d] > (int64_t(1) << 38) || t->strides[d] * esz % step != 0)
      return fail(GQA_ERR_INVALID_ARG, "%s: stride %lld in dimension %d is not a multiple of %d bytes in [0, 2^38]", name,
                  (long long)t->strides[d], d, step);
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

// Do two dense tensors share a byte?
bool overlap(const gqa_tensor* a, const gqa_tensor* b) {
  auto bytes = [](const gqa_tensor* t) {
    uint64_t n = (uint64_t)dtype_bytes(t->dtype);
    for (int d = 0; d < t->ndim; ++d) n *= (uint64_t)t->shape[d];
    return n;
  };
  const uint64_t x = reinterpret_cast<uintptr_t>(a->data), y = reinterpret_cast<uintptr_t>(b->data), m = bytes(a), n = bytes(b);
  return m > 0 && n > 0 && (x < y ? y - x < m : x - y < n);
}

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

// What the appends with norms and positions add; null ones are left out.
struct AppendExtra {
  const gqa_tensor *positions, *q_norm, *k_norm;
  float eps;
};

gqa_status add_extra(const AppendExtra& x, bool has_q, int32_t dtype, gqa::AppendArgs* a, std::vector<Named>* ts) {
  if (x.positions) {
    gqa_tensor p = *x.positions;
    if (!p.data && a->total == 0) p.data = &p;  // (an empty tensor may have no data)
    GQA_TRY(check_desc(&p, "positions", {GQA_I32}, {a->total}));
    if (!a->rope) return fail(GQA_ERR_INVALID_ARG, "positions are rows of the rope table: there is none");
    a->positions = static_cast<const int32_t*>(x.positions->data);
    ts->push_back({x.positions, "positions"});
  }
  if (x.q_norm && !has_q) return fail(GQA_ERR_INVALID_ARG, "q_norm without q");
  const gqa_tensor* first = nullptr;
  for (const Named& w : {Named{x.q_norm, "q_norm"}, Named{x.k_norm, "k_norm"}}) {
    if (!w.first) continue;
    GQA_TRY(first ? check_desc(w.first, w.second, {first->dtype}, {a->d}) : check_desc(w.first, w.second, {dtype, GQA_F32}, {a->d}));
    first = w.first;
    ts->push_back(w);
  }
  if (first) {
    if (!std::isfinite(x.eps) || x.eps < 0.f) return fail(GQA_ERR_INVALID_ARG, "norm_eps must be finite and >= 0");
    a->q_norm = x.q_norm ? x.q_norm->data : nullptr;
    a->k_norm = x.k_norm ? x.k_norm->data : nullptr;
    a->norm_f32 = first->dtype == GQA_F32;
    a->norm_eps = x.eps;
  }
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

gqa_status append_impl(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_pages,
                       gqa_tensor* v_pages, const gqa_tensor* block_table, const gqa_tensor* kv_lens,
                       const gqa_tensor* qo_indptr, const gqa_tensor* rope, gqa_tensor* q_out, int interleaved,
                       float k_scale, float v_scale, const AppendExtra& extra, gqa_stream_t stream) {
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
  GQA_TRY(add_extra(extra, q != nullptr, k->dtype, &a, &ts));
  return run_append(a, ts, "gqa_paged_append", stream);
}

gqa_status nvfp4_append_impl(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_fp4,
                             gqa_tensor* k_sf, gqa_tensor* v_fp4, gqa_tensor* v_sf, const gqa_tensor* block_table,
                             const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, const gqa_tensor* rope,
                             gqa_tensor* q_out, int interleaved, float q_scale, const AppendExtra& extra, gqa_stream_t stream) {
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
  GQA_TRY(add_extra(extra, q != nullptr, k->dtype, &a, &ts));
  return run_append(a, ts, "nvfp4_paged_append", stream);
}

// The library's workspace of an attention for a stream, of the most that any call needs (so
// that it never moves); refused for a call that is being captured, which needs `need`.
gqa_status own_workspace(int device, cudaStream_t s, size_t most, int64_t need, WorkspaceMap& map, void** out) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  GQA_CUDA_TRY(cudaStreamIsCapturing(s, &capture), "cudaStreamIsCapturing");
  if (capture != cudaStreamCaptureStatusNone)
    return fail(GQA_ERR_WORKSPACE, "a captured call needs a workspace of its own (%lld bytes)", (long long)need);
  if (s == cudaStreamPerThread) {
    static thread_local ThreadEnd end;
    end.thread = gqa::thread_number();
  }
  // (allocated without disturbing a capture of another thread)
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  GQA_CUDA_TRY(cudaThreadExchangeStreamCaptureMode(&mode), "cudaThreadExchangeStreamCaptureMode");
  const gqa_status st = workspace(device, s, most, out, map);
  cudaThreadExchangeStreamCaptureMode(&mode);
  return st;
}

// What the two attentions share: queries [rows, hq, d] over pages, the table of `batch` sequences.
struct AttnSizes {
  int64_t rows, hq, d, num_pages, hkv, page_size, max_pages;
  bool e4m3;
};
gqa_status check_attn(const gqa_tensor* q, const gqa_tensor* k_pages, const gqa_tensor* v_pages, const gqa_tensor* block_table,
                      int64_t batch, const gqa_tensor* out, const gqa_tensor* lse, AttnSizes* z) {
  int64_t qs[3], ps[4], bs[2];
  GQA_TRY(check_strided(q, "q", {GQA_F16, GQA_BF16}, {-1, -1, -1}, false, qs));
  GQA_TRY(check_strided(k_pages, "k_pages", {q->dtype, GQA_E4M3, GQA_U8}, {-1, -1, -1, qs[2]}, true, ps));
  const bool e4m3 = k_pages->dtype != q->dtype;
  GQA_TRY(e4m3 ? check_strided(v_pages, "v_pages", {GQA_E4M3, GQA_U8}, {ps[0], ps[1], ps[2], qs[2]}, true)
               : check_strided(v_pages, "v_pages", {q->dtype}, {ps[0], ps[1], ps[2], qs[2]}, true));
  GQA_TRY(check_desc(block_table, "block_table", {GQA_I32}, {batch < 0 ? qs[0] : batch, -1}, bs));
  gqa_tensor o = *out, l;
  if (!o.data && qs[0] == 0) o.data = &o;  // (an empty tensor may have no data)
  GQA_TRY(check_desc(&o, "out", {q->dtype}, {qs[0], qs[1], qs[2]}));
  if (lse) {
    l = *lse;
    if (!l.data && qs[0] == 0) l.data = &l;
    GQA_TRY(check_desc(&l, "lse", {GQA_F32}, {qs[0], qs[1]}));
  }
  *z = {qs[0], qs[1], qs[2], ps[0], ps[1], ps[2], bs[1], e4m3};
  return GQA_OK;
}
gqa_status check_layout(const AttnSizes& z) {
  if (z.d != 64 && z.d != 128 && z.d != 256)
    return fail(GQA_ERR_UNSUPPORTED_SHAPE, "head dim %lld is not 64, 128 or 256", (long long)z.d);
  if (z.hkv < 1 || z.hq < 1 || z.hq > 1024 || z.hq % z.hkv != 0)
    return fail(GQA_ERR_UNSUPPORTED_SHAPE, "%lld query heads over %lld KV heads: 1 to 1024, a multiple, are taken",
                (long long)z.hq, (long long)z.hkv);
  if (z.page_size != 16 && z.page_size != 32 && z.page_size != 64 && z.page_size != 128 && z.page_size != 256)
    return fail(GQA_ERR_UNSUPPORTED_SHAPE, "page size %lld is not 16, 32, 64, 128 or 256", (long long)z.page_size);
  if (z.num_pages < 1 || z.num_pages > 2147483647LL)
    return fail(GQA_ERR_INVALID_ARG, "num_pages %lld out of range", (long long)z.num_pages);
  if (z.max_pages < 1 || z.max_pages > (int64_t(1) << 30) / z.page_size)
    return fail(GQA_ERR_INVALID_ARG, "max_pages_per_seq %lld out of range", (long long)z.max_pages);
  return GQA_OK;
}
gqa_status check_numbers(float q_scale, float k_scale, float v_scale, int window, int sinks, float softcap) {
  if (!std::isfinite(q_scale)) return fail(GQA_ERR_INVALID_ARG, "q_scale is not finite");
  GQA_TRY(check_scale(k_scale, "k_scale"));
  GQA_TRY(check_scale(v_scale, "v_scale"));
  if (window < 0) return fail(GQA_ERR_INVALID_ARG, "window %d is negative", window);
  if (sinks < 0) return fail(GQA_ERR_INVALID_ARG, "sinks %d is negative", sinks);
  if (!std::isfinite(softcap) || softcap < 0.f) return fail(GQA_ERR_INVALID_ARG, "softcap must be finite and >= 0");
  return GQA_OK;
}
int cache_type(const gqa_tensor* q, bool e4m3) {
  const bool bf16 = q->dtype == GQA_BF16;
  return e4m3 ? (bf16 ? gqa::kCacheE4m3 : gqa::kCacheE4m3F16) : bf16 ? gqa::kCacheBf16 : gqa::kCacheF16;
}

}  // namespace

extern "C" {

gqa_status gqa_paged_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_pages,
                              gqa_tensor* v_pages, const gqa_tensor* block_table, const gqa_tensor* kv_lens,
                              const gqa_tensor* qo_indptr, const gqa_tensor* rope, gqa_tensor* q_out, int interleaved,
                              float k_scale, float v_scale, gqa_stream_t stream) {
  return guarded([&] {
    return append_impl(q, k, v, k_pages, v_pages, block_table, kv_lens, qo_indptr, rope, q_out, interleaved, k_scale, v_scale,
                       {nullptr, nullptr, nullptr, 0.f}, stream);
  });
}

gqa_status gqa_paged_norm_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_pages,
                                   gqa_tensor* v_pages, const gqa_tensor* block_table, const gqa_tensor* kv_lens,
                                   const gqa_tensor* qo_indptr, const gqa_tensor* rope, const gqa_tensor* positions,
                                   const gqa_tensor* q_norm, const gqa_tensor* k_norm, gqa_tensor* q_out, int interleaved,
                                   float norm_eps, float k_scale, float v_scale, gqa_stream_t stream) {
  return guarded([&] {
    return append_impl(q, k, v, k_pages, v_pages, block_table, kv_lens, qo_indptr, rope, q_out, interleaved, k_scale, v_scale,
                       {positions, q_norm, k_norm, norm_eps}, stream);
  });
}

gqa_status nvfp4_paged_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_fp4,
                                gqa_tensor* k_sf, gqa_tensor* v_fp4, gqa_tensor* v_sf, const gqa_tensor* block_table,
                                const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, const gqa_tensor* rope,
                                gqa_tensor* q_out, int interleaved, float q_scale, gqa_stream_t stream) {
  return guarded([&] {
    return nvfp4_append_impl(q, k, v, k_fp4, k_sf, v_fp4, v_sf, block_table, qo_indptr, kv_lens, rope, q_out, interleaved, q_scale,
                             {nullptr, nullptr, nullptr, 0.f}, stream);
  });
}

gqa_status nvfp4_paged_norm_append_t(const gqa_tensor* q, const gqa_tensor* k, const gqa_tensor* v, gqa_tensor* k_fp4,
                                     gqa_tensor* k_sf, gqa_tensor* v_fp4, gqa_tensor* v_sf, const gqa_tensor* block_table,
                                     const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, const gqa_tensor* rope,
                                     const gqa_tensor* positions, const gqa_tensor* q_norm, const gqa_tensor* k_norm,
                                     gqa_tensor* q_out, int interleaved, float norm_eps, float q_scale, gqa_stream_t stream) {
  return guarded([&] {
    return nvfp4_append_impl(q, k, v, k_fp4, k_sf, v_fp4, v_sf, block_table, qo_indptr, kv_lens, rope, q_out, interleaved, q_scale,
                             {positions, q_norm, k_norm, norm_eps}, stream);
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
  return gqa_paged_window_attn_t(q, k_pages, v_pages, block_table, seq_lens, out, lse, q_scale, k_scale, v_scale, window, 0,
                                 softcap, workspace_, workspace_bytes, stream);
}

gqa_status gqa_paged_window_attn_t(const gqa_tensor* q, const gqa_tensor* k_pages, const gqa_tensor* v_pages,
                                   const gqa_tensor* block_table, const gqa_tensor* seq_lens, gqa_tensor* out, gqa_tensor* lse,
                                   float q_scale, float k_scale, float v_scale, int window, int sinks, float softcap, void* workspace_,
                                   int64_t workspace_bytes, gqa_stream_t stream) {
  return guarded([&]() -> gqa_status {
    AttnSizes z;
    if (!q || !k_pages || !out) return fail(GQA_ERR_INVALID_ARG, "q, k_pages or out: null descriptor");
    GQA_TRY(check_attn(q, k_pages, v_pages, block_table, -1, out, lse, &z));
    GQA_TRY(check_desc(seq_lens, "seq_lens", {GQA_I32}, {z.rows}));
    if (z.rows < 1 || z.rows > 65535) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 65535]", (long long)z.rows);
    GQA_TRY(check_layout(z));
    // (a block of the kernel counts the work of its share, in tiles of 32 tokens at least, in 31 bits)
    if (z.rows * z.hkv * ((z.hq / z.hkv + 7) / 8) > (int64_t(1) << 38) / (z.max_pages * z.page_size / 32 + 16))
      return fail(GQA_ERR_UNSUPPORTED, "batch %lld x %lld KV heads x %lld tokens of capacity are too many", (long long)z.rows,
                  (long long)z.hkv, (long long)(z.max_pages * z.page_size));
    GQA_TRY(check_numbers(q_scale, k_scale, v_scale, window, sinks, softcap));
    const int64_t need = gqa_paged_attn_workspace(z.hq, z.hkv, z.d);
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
    a.batch = z.rows;
    a.num_pages = z.num_pages;
    a.max_pages_per_seq = z.max_pages;
    a.hq = (int)z.hq;
    a.hkv = (int)z.hkv;
    a.d = (int)z.d;
    a.page_size = (int)z.page_size;
    a.cache = cache_type(q, z.e4m3);
    a.scale = (float)((double)q_scale * k_scale / std::sqrt((double)z.d));
    a.v_scale = v_scale;
    a.softcap = softcap;
    a.window = window;
    a.sinks = sinks;
    a.starve = gqa::starve_producers();
    if (!std::isfinite(a.scale) || (softcap > 0.f && !std::isfinite((float)(4.0 * a.scale / softcap))))
      return fail(GQA_ERR_INVALID_ARG, "q_scale * k_scale (over softcap) is out of range");
    ScopedDevice sd(where.device);
    if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // A call's two kernels follow each other on the stream: another thread's call on the
    // same stream, and so with the same workspace, must not come between them.
    std::lock_guard<std::mutex> lk(g_paged_launch_mu);
    if (!workspace_) GQA_TRY(own_workspace(where.device, s, gqa::paged_attn_workspace_bytes(1024, 1, 256), need, g_paged_ws, &workspace_));
    GQA_CUDA_TRY(gqa::launch_paged_attn(a, workspace_, s), "paged attention launch");
    return GQA_OK;
  });
}

gqa_status gqa_tree_mask_t(const gqa_tensor* parents, const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, gqa_tensor* mask,
                           gqa_tensor* positions, int window, int sinks, gqa_stream_t stream) {
  return guarded([&]() -> gqa_status {
    int64_t ps[1], ls[1], ms[2];
    // (empty tensors may have no data)
    gqa_tensor pa, ma, po;
    for (auto& c : {std::make_pair(parents, &pa), std::make_pair((const gqa_tensor*)mask, &ma),
                    std::make_pair((const gqa_tensor*)positions, &po)}) {
      if (!c.first) return fail(GQA_ERR_INVALID_ARG, "parents, mask or positions: null descriptor");
      *c.second = *c.first;
      if (!c.second->data && c.second->ndim > 0 && c.second->shape[0] == 0) c.second->data = c.second;
    }
    GQA_TRY(check_desc(&pa, "parents", {GQA_I32}, {-1}, ps));
    GQA_TRY(check_desc(kv_lens, "kv_lens", {GQA_I32}, {-1}, ls));
    if (ls[0] < 1 || ls[0] > (1 << 20)) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 2^20]", (long long)ls[0]);
    GQA_TRY(check_desc(qo_indptr, "qo_indptr", {GQA_I32}, {ls[0] + 1}));
    GQA_TRY(check_desc(&ma, "mask", {GQA_I32}, {ps[0], -1}, ms));
    GQA_TRY(check_desc(&po, "positions", {GQA_I32}, {ps[0]}));
    if (ms[1] < 1 || ms[1] > gqa::kMaxTreeTokens / 32)
      return fail(GQA_ERR_UNSUPPORTED_SHAPE, "%lld words of bits: 1 to %d are taken", (long long)ms[1], gqa::kMaxTreeTokens / 32);
    if (window < 0) return fail(GQA_ERR_INVALID_ARG, "window %d is negative", window);
    if (sinks < 0) return fail(GQA_ERR_INVALID_ARG, "sinks %d is negative", sinks);
    // (trees' blocks run at the same time; one reads all its parents before it writes)
    for (const Named& out : {Named{&ma, "mask"}, Named{&po, "positions"}})
      for (const Named& in : {Named{&pa, "parents"}, Named{qo_indptr, "qo_indptr"}, Named{kv_lens, "kv_lens"}, Named{&po, "positions"}})
        if (out.first != in.first && overlap(out.first, in.first) && !(out.first == &po && in.first == &pa && po.data == pa.data))
          return fail(GQA_ERR_INVALID_ARG, "%s overlaps %s: both are in use at once", out.second, in.second);
    if (ps[0] == 0) return GQA_OK;
    Where where;
    GQA_TRY(locate_tensors({{parents, "parents"}, {qo_indptr, "qo_indptr"}, {kv_lens, "kv_lens"}, {mask, "mask"}, {positions, "positions"}},
                           "gqa_tree_mask", &where));
    gqa::TreeMaskArgs a{};
    a.parents = static_cast<const int32_t*>(parents->data);
    a.indptr = static_cast<const int32_t*>(qo_indptr->data);
    a.kv_lens = static_cast<const int32_t*>(kv_lens->data);
    a.mask = static_cast<uint32_t*>(mask->data);
    a.positions = static_cast<int32_t*>(positions->data);
    a.total = ps[0];
    a.batch = ls[0];
    a.words = (int)ms[1];
    a.window = window;
    a.sinks = sinks;
    ScopedDevice sd(where.device);
    if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
    GQA_CUDA_TRY(gqa::launch_tree_mask(a, reinterpret_cast<cudaStream_t>(stream)), "tree mask launch");
    return GQA_OK;
  });
}

gqa_status gqa_paged_keep_t(const gqa_tensor* const* pages, int num_tensors, const gqa_tensor* block_table,
                            const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens, const gqa_tensor* kept,
                            const gqa_tensor* num_kept, gqa_tensor* new_lens, gqa_stream_t stream) {
  return guarded([&]() -> gqa_status {
    int64_t ls[1], bs[2], ks[2];
    if (!pages || num_tensors < 1 || num_tensors > gqa::kKeepTensors)
      return fail(GQA_ERR_INVALID_ARG, "%d tensors of pages: 1 to %d are taken", num_tensors, gqa::kKeepTensors);
    GQA_TRY(check_desc(kv_lens, "kv_lens", {GQA_I32}, {-1}, ls));
    if (ls[0] < 1 || ls[0] > 65535) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 65535]", (long long)ls[0]);
    GQA_TRY(check_desc(block_table, "block_table", {GQA_I32}, {ls[0], -1}, bs));
    GQA_TRY(check_desc(qo_indptr, "qo_indptr", {GQA_I32}, {ls[0] + 1}));
    GQA_TRY(check_desc(kept, "kept", {GQA_I32}, {ls[0], -1}, ks));
    GQA_TRY(check_desc(num_kept, "num_kept", {GQA_I32}, {ls[0]}));
    GQA_TRY(check_desc(new_lens, "new_lens", {GQA_I32}, {ls[0]}));
    if (new_lens->data == kv_lens->data) return fail(GQA_ERR_INVALID_ARG, "new_lens may not be kv_lens: both are in use at once");
    // (blocks that have yet to begin read what the first ones of a sequence would have written over)
    for (const Named& t : {Named{kv_lens, "kv_lens"}, Named{num_kept, "num_kept"}, Named{kept, "kept"}, Named{qo_indptr, "qo_indptr"},
                           Named{block_table, "block_table"}})
      if (overlap(new_lens, t.first)) return fail(GQA_ERR_INVALID_ARG, "new_lens overlaps %s: both are in use at once", t.second);
    if (bs[1] < 1) return fail(GQA_ERR_INVALID_ARG, "block_table has no column");
    if (ks[1] < 1) return fail(GQA_ERR_INVALID_ARG, "kept has no column");
    std::vector<Named> ts = {{block_table, "block_table"}, {qo_indptr, "qo_indptr"}, {kv_lens, "kv_lens"},
                             {kept, "kept"},               {num_kept, "num_kept"},   {new_lens, "new_lens"}};
    static const char* const names[gqa::kKeepTensors] = {"pages[0]", "pages[1]", "pages[2]", "pages[3]"};
    gqa::KeepArgs a{};
    std::vector<gqa_tensor> at(num_tensors);
    for (int i = 0; i < num_tensors; ++i) {
      const gqa_tensor* t = pages[i];
      if (!t) return fail(GQA_ERR_INVALID_ARG, "%s: null descriptor", names[i]);
      if (t->ndim != 4 && t->ndim != 5) return fail(GQA_ERR_INVALID_ARG, "%s has %d dimensions; expected 4 or 5", names[i], t->ndim);
      const int o = t->ndim - 4;
      int64_t s[5];
      GQA_TRY(o ? check_strided(t, names[i], {GQA_F16, GQA_BF16, GQA_E4M3, GQA_U8, GQA_F32}, {-1, -1, -1, -1, -1}, true, s, 8)
                : check_strided(t, names[i], {GQA_F16, GQA_BF16, GQA_E4M3, GQA_U8, GQA_F32}, {-1, -1, -1, -1}, true, s, 8));
      const int64_t layers = o ? s[0] : 1, num = s[o], heads = s[o + 1], size = s[o + 2], row = s[o + 3] * dtype_bytes(t->dtype);
      if (layers < 1 || num < 1 || heads < 1 || size < 1 || row < 1 || num > 2147483647LL || size > (1 << 20) || row > (1 << 20) ||
          layers * heads > (1 << 24))
        return fail(GQA_ERR_UNSUPPORTED_SHAPE, "%s is empty, or larger than is taken", names[i]);
      if (row % 8 != 0) return fail(GQA_ERR_UNSUPPORTED_SHAPE, "%s: rows of %lld bytes are no multiple of 8", names[i], (long long)row);
      if (i == 0) {
        a.num_pages = num;
        a.page_size = size;
      } else if (num != a.num_pages || size != a.page_size) {
        return fail(GQA_ERR_INVALID_ARG, "%s has %lld pages of %lld tokens; pages[0] has %lld of %lld", names[i], (long long)num,
                    (long long)size, (long long)a.num_pages, (long long)a.page_size);
      }
      const int64_t esz = dtype_bytes(t->dtype);
      gqa::KeepTensor& k = a.t[i];
      k.data = static_cast<uint8_t*>(t->data);
      k.s_layer = o ? stride_of(t, 0) * esz : 0;
      k.s_page = stride_of(t, o) * esz;
      k.s_head = stride_of(t, o + 1) * esz;
      k.s_slot = stride_of(t, o + 2) * esz;
      const int64_t all = k.s_layer | k.s_page | k.s_head | k.s_slot | row | (int64_t)reinterpret_cast<uintptr_t>(t->data);
      k.vec = all % 16 == 0 ? 16 : 8;
      k.heads = heads;
      k.pieces = row / k.vec;
      k.items = layers * heads * k.pieces;
      for (int j = 0; j < i; ++j)
        if (a.t[j].data == k.data) return fail(GQA_ERR_INVALID_ARG, "%s is %s again: its rows would move twice", names[i], names[j]);
      // (8-byte alignment is enough: it is looked at here)
      if (reinterpret_cast<uintptr_t>(t->data) % 8 != 0) return fail(GQA_ERR_INVALID_ARG, "%s is not 8-byte aligned", names[i]);
      at[i] = *t;
      at[i].dtype = GQA_I32;
      ts.push_back({&at[i], names[i]});
    }
    a.tensors = num_tensors;
    Where where;
    GQA_TRY(locate_tensors(ts, "gqa_paged_keep", &where));
    a.block_table = static_cast<const int32_t*>(block_table->data);
    a.indptr = static_cast<const int32_t*>(qo_indptr->data);
    a.kv_lens = static_cast<const int32_t*>(kv_lens->data);
    a.kept = static_cast<const int32_t*>(kept->data);
    a.num_kept = static_cast<const int32_t*>(num_kept->data);
    a.new_lens = static_cast<int32_t*>(new_lens->data);
    a.batch = ls[0];
    a.max_pages = bs[1];
    a.max_kept = ks[1];
    ScopedDevice sd(where.device);
    if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
    GQA_CUDA_TRY(gqa::launch_keep(a, reinterpret_cast<cudaStream_t>(stream)), "keep launch");
    return GQA_OK;
  });
}

int64_t gqa_paged_tree_attn_workspace(int64_t q_heads, int64_t kv_heads, int64_t d) {
  if (kv_heads < 1 || q_heads < 1 || q_heads > 1024 || q_heads % kv_heads != 0 || (d != 64 && d != 128 && d != 256)) return 0;
  return (int64_t)gqa::tree_attn_workspace_bytes((int)d);
}

gqa_status gqa_paged_tree_attn_t(const gqa_tensor* q, const gqa_tensor* k_pages, const gqa_tensor* v_pages,
                                 const gqa_tensor* block_table, const gqa_tensor* qo_indptr, const gqa_tensor* kv_lens,
                                 const gqa_tensor* mask, const gqa_tensor* positions, gqa_tensor* out, gqa_tensor* lse,
                                 float q_scale, float k_scale, float v_scale, int window, int sinks, float softcap,
                                 void* workspace_, int64_t workspace_bytes, gqa_stream_t stream) {
  return guarded([&]() -> gqa_status {
    AttnSizes z;
    int64_t ls[1], ms[2] = {0, 0};
    if (!q || !k_pages || !out) return fail(GQA_ERR_INVALID_ARG, "q, k_pages or out: null descriptor");
    GQA_TRY(check_desc(kv_lens, "kv_lens", {GQA_I32}, {-1}, ls));
    if (ls[0] < 1 || ls[0] > 65535) return fail(GQA_ERR_UNSUPPORTED, "batch %lld outside [1, 65535]", (long long)ls[0]);
    GQA_TRY(check_desc(qo_indptr, "qo_indptr", {GQA_I32}, {ls[0] + 1}));
    GQA_TRY(check_attn(q, k_pages, v_pages, block_table, ls[0], out, lse, &z));
    if (mask) {
      gqa_tensor m = *mask;
      if (!m.data && z.rows == 0) m.data = &m;
      GQA_TRY(check_desc(&m, "mask", {GQA_I32}, {z.rows, -1}, ms));
      if (ms[1] < 1 || ms[1] > gqa::kMaxTreeTokens / 32)
        return fail(GQA_ERR_UNSUPPORTED_SHAPE, "%lld words of bits: 1 to %d are taken", (long long)ms[1], gqa::kMaxTreeTokens / 32);
      if (window > 0 && !positions) return fail(GQA_ERR_INVALID_ARG, "a window over a tree needs the tokens' positions");
    }
    if (positions) {
      gqa_tensor x = *positions;
      if (!x.data && z.rows == 0) x.data = &x;
      GQA_TRY(check_desc(&x, "positions", {GQA_I32}, {z.rows}));
    }
    GQA_TRY(check_layout(z));
    GQA_TRY(check_numbers(q_scale, k_scale, v_scale, window, sinks, softcap));
    const int64_t group = z.hq / z.hkv, tiles = z.max_pages * z.page_size / 64 + 16;
    if (z.rows * group > 2147483647LL) return fail(GQA_ERR_UNSUPPORTED, "%lld tokens of %lld heads are too many", (long long)z.rows, (long long)group);
    // (tiles of 64 tokens at least; the kernel looks again, for offsets that fall)
    if (z.hkv * (ls[0] + z.rows * group / 128) > gqa::kTreeMostWork / tiles)
      return fail(GQA_ERR_UNSUPPORTED, "%lld sequences, %lld tokens x %lld KV heads x %lld tokens of capacity are too many",
                  (long long)ls[0], (long long)z.rows, (long long)z.hkv, (long long)(z.max_pages * z.page_size));
    const float scale = (float)((double)q_scale * k_scale / std::sqrt((double)z.d));
    if (!std::isfinite(scale) || (softcap > 0.f && !std::isfinite((float)(4.0 * scale / softcap))))
      return fail(GQA_ERR_INVALID_ARG, "q_scale * k_scale (over softcap) is out of range");
    const int64_t need = gqa_paged_tree_attn_workspace(z.hq, z.hkv, z.d);
    if (workspace_ && workspace_bytes < need)
      return fail(GQA_ERR_INVALID_ARG, "workspace of %lld bytes; %lld are needed", (long long)workspace_bytes, (long long)need);
    if (z.rows == 0) return GQA_OK;
    gqa_tensor ws = *q;  // the workspace's place is checked with the tensors'
    ws.data = workspace_;
    std::vector<Named> ts = {{q, "q"}, {k_pages, "k_pages"}, {v_pages, "v_pages"}, {block_table, "block_table"},
                             {qo_indptr, "qo_indptr"}, {kv_lens, "kv_lens"}, {out, "out"}};
    if (workspace_) ts.push_back({&ws, "workspace"});
    if (mask) ts.push_back({mask, "mask"});
    if (positions) ts.push_back({positions, "positions"});
    gqa_tensor l;
    if (lse) {
      l = *lse;
      l.dtype = GQA_I32;  // (4-byte alignment)
      ts.push_back({&l, "lse"});
    }
    Where where;
    GQA_TRY(locate_tensors(ts, "gqa_paged_tree_attn", &where));
    gqa::TreeAttnArgs a{};
    a.q = q->data;
    a.out = out->data;
    a.lse = lse ? static_cast<float*>(lse->data) : nullptr;
    a.k_pages = k_pages->data;
    a.v_pages = v_pages->data;
    a.block_table = static_cast<const int32_t*>(block_table->data);
    a.indptr = static_cast<const int32_t*>(qo_indptr->data);
    a.kv_lens = static_cast<const int32_t*>(kv_lens->data);
    a.mask = mask ? static_cast<const int32_t*>(mask->data) : nullptr;
    a.positions = positions ? static_cast<const int32_t*>(positions->data) : nullptr;
    a.q_tok = stride_of(q, 0);
    a.q_head = stride_of(q, 1);
    a.kp_page = k_pages->strides[0];
    a.kp_head = k_pages->strides[1];
    a.kp_slot = k_pages->strides[2];
    a.vp_page = v_pages->strides[0];
    a.vp_head = v_pages->strides[1];
    a.vp_slot = v_pages->strides[2];
    a.total = z.rows;
    a.batch = ls[0];
    a.num_pages = z.num_pages;
    a.max_pages_per_seq = z.max_pages;
    a.hq = (int)z.hq;
    a.hkv = (int)z.hkv;
    a.d = (int)z.d;
    a.page_size = (int)z.page_size;
    a.words = (int)ms[1];
    a.cache = cache_type(q, z.e4m3);
    a.scale = scale;
    a.v_scale = v_scale;
    a.softcap = softcap;
    a.window = window;
    a.sinks = sinks;
    a.starve = gqa::starve_producers();
    ScopedDevice sd(where.device);
    if (!sd.ok()) return fail(GQA_ERR_CUDA, "cannot switch to device %d", where.device);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // (two kernels that share a workspace, as the one-token attention's)
    std::lock_guard<std::mutex> lk(g_paged_launch_mu);
    if (!workspace_) GQA_TRY(own_workspace(where.device, s, gqa::tree_attn_workspace_bytes(256), need, g_tree_ws, &workspace_));
    GQA_CUDA_TRY(gqa::launch_tree_attn(a, workspace_, s), "tree attention launch");
    return GQA_OK;
  });
}

}  // extern "C"
