// paged_attn.cpp -- host side of the one-token paged attention: tensor maps,
// workspace layout, choice of the instance.
#include <cuda.h>  // CUtensorMap and the cuTensorMapEncodeTiled prototype (resolved at run time)

#include <algorithm>
#include <cmath>
#include <limits>
#include <mutex>

#include "paged_attn_host.h"

namespace gqa {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::once_flag g_encode_once;
EncodeTiledFn g_encode = nullptr;

// Tensor map over pages [num_pages, hkv, page_size, d] of any order in memory: a row
// of d elements is cut into chunks of at most 128 bytes, and a copy takes `box`
// tokens of one head of one page, chunk after chunk, swizzled.
cudaError_t make_map(const void* pages, const PagedAttnArgs& a, int64_t s_page, int64_t s_head, int64_t s_slot, int box,
                     CUtensorMap* map) {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  });
  if (!g_encode) return cudaErrorNotSupported;
  const int64_t esz = a.cache >= kCacheE4m3 ? 1 : 2;
  const int64_t row = a.d * esz, chunk = row < 128 ? row : 128;
  const cuuint64_t dims[5] = {(cuuint64_t)chunk, (cuuint64_t)a.page_size, (cuuint64_t)(row / chunk), (cuuint64_t)a.hkv,
                              (cuuint64_t)a.num_pages};
  // (a dimension of extent 1 may carry any stride; the map wants a multiple of 16)
  const cuuint64_t strides[4] = {(cuuint64_t)(s_slot * esz), (cuuint64_t)chunk,
                                 (cuuint64_t)(a.hkv > 1 ? s_head * esz : row), (cuuint64_t)(a.num_pages > 1 ? s_page * esz : row)};
  const cuuint32_t boxes[5] = {(cuuint32_t)chunk, (cuuint32_t)box, (cuuint32_t)(row / chunk), 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(pages), dims, strides, boxes, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              chunk == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              // (rows of one head apart: what lies behind 128 bytes may be another head's)
                              s_slot == a.d ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int rows_of(int group) { return group > 8 ? 16 : 8; }  // query heads of a unit

}  // namespace

size_t paged_attn_workspace_bytes(int hq, int hkv, int d) {
  const size_t rows = (size_t)pa::kGrid * 2 * rows_of(hq / hkv);
  return rows * d * sizeof(float) + rows * sizeof(float2) + pa::kGrid * sizeof(pa::Record);
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, void* workspace, cudaStream_t stream) {
  const int row_bytes = a.d * (a.cache >= kCacheE4m3 ? 1 : 2);
  const int tile = pa::tile_of(row_bytes);
  pa::Params p;
  p.q = a.q;
  p.out = a.out;
  p.lse = a.lse;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.group = a.hq / a.hkv;
  const int rows = rows_of(p.group);
  const size_t n = (size_t)pa::kGrid * 2 * rows;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + n * a.d);
  p.q_seq = a.q_seq;
  p.q_head = a.q_head;
  p.batch = a.batch;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages_per_seq;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.head_blocks = (p.group + rows - 1) / rows;
  for (p.gang_shift = 0; p.gang_shift < pa::kGangShift && ((a.hkv * p.head_blocks) >> p.gang_shift) % 2 == 0; ++p.gang_shift) {
  }
  const int box = a.page_size < tile ? a.page_size : tile;
  for (p.page_shift = 0; (1 << p.page_shift) < a.page_size; ++p.page_shift) {
  }
  for (p.box_shift = 0; (1 << p.box_shift) < box; ++p.box_shift) {
  }
  // No unit is split if there are no more than blocks and their sequences cannot be long
  // (the kernel's own rule, by the lengths themselves); then nothing is to be joined.
  const int64_t units = a.batch * a.hkv * p.head_blocks;
  const bool whole = units <= pa::kGrid && a.max_pages_per_seq * a.page_size <= (int64_t)pa::kWholeTiles * tile;
  p.record = whole ? nullptr : reinterpret_cast<pa::Record*>(p.part_ml + n);
  p.record_by_unit = units <= pa::kGrid;
  p.records = units <= pa::kGrid ? (int)units : pa::kGrid;
  const double log2e = 1.4426950408889634;
  p.scale_log2 = (float)(a.scale * log2e);
  // (a cap at the end of f32's range stays finite, twice itself too)
  const double cap = a.softcap * log2e, most = std::numeric_limits<float>::max() / 2;
  p.cap_out = a.softcap > 0.f ? (float)std::min(cap, most) : 0.f;
  p.cap_inv = a.softcap > 0.f ? (float)std::min(1.0 / cap, most) : 0.f;
  p.v_scale = a.v_scale;
  p.window = a.window;
  p.starve = a.starve;
  CUtensorMap k_map, v_map;
  cudaError_t e;
  if ((e = make_map(a.k_pages, a, a.kp_page, a.kp_head, a.kp_slot, box, &k_map)) != cudaSuccess) return e;
  if ((e = make_map(a.v_pages, a, a.vp_page, a.vp_head, a.vp_slot, box, &v_map)) != cudaSuccess) return e;
  switch (a.cache) {
    case kCacheF16: return pa::launch_f16(p, a.d, k_map, v_map, stream);
    case kCacheBf16: return pa::launch_bf16(p, a.d, k_map, v_map, stream);
    case kCacheE4m3: return pa::launch_e4m3(p, a.d, k_map, v_map, stream);
    default: return pa::launch_e4m3_f16(p, a.d, k_map, v_map, stream);
  }
}

cudaError_t paged_attn_read_errors(uint32_t* word) {
  cudaError_t e = cudaDeviceSynchronize();
  uint32_t w[3] = {0, 0, 0};
  if (e == cudaSuccess) e = pa::read_errors_f16(&w[0]);
  if (e == cudaSuccess) e = pa::read_errors_bf16(&w[1]);
  if (e == cudaSuccess) e = pa::read_errors_e4m3(&w[2]);
  *word = w[0] | w[1] | w[2];
  return e;
}

}  // namespace gqa
