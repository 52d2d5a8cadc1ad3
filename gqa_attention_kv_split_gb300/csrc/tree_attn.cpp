// tree_attn.cpp -- host side of the paged attention of several new tokens: tensor maps,
// workspace layout, choice of the instance.
#include <algorithm>
#include <cmath>
#include <limits>

#include "page_map.h"
#include "tree_attn_host.h"

namespace gqa {
namespace {

// Tensor map over pages [num_pages, hkv, page_size, d] of any order in memory.  16-bit pages: a
// copy takes 128 bytes of the rows of `box` tokens of one head of one page, swizzled; E4M3
// ones: the rows, as they are.
cudaError_t make_map(const void* pages, const TreeAttnArgs& a, int64_t s_page, int64_t s_head, int64_t s_slot, int box,
                     CUtensorMap* map) {
  const EncodeTiledFn encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  const bool e4m3 = a.cache >= kCacheE4m3;
  const int64_t esz = e4m3 ? 1 : 2, row = a.d * esz, chunk = e4m3 ? row : 128;
  const cuuint64_t dims[5] = {(cuuint64_t)chunk, (cuuint64_t)a.page_size, (cuuint64_t)(row / chunk), (cuuint64_t)a.hkv,
                              (cuuint64_t)a.num_pages};
  // (a dimension of extent 1 may carry any stride; the map wants a multiple of 16)
  const cuuint64_t strides[4] = {(cuuint64_t)(a.page_size > 1 ? s_slot * esz : row), (cuuint64_t)chunk,
                                 (cuuint64_t)(a.hkv > 1 ? s_head * esz : row), (cuuint64_t)(a.num_pages > 1 ? s_page * esz : row)};
  const cuuint32_t boxes[5] = {(cuuint32_t)chunk, (cuuint32_t)box, 1, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(pages), dims, strides, boxes, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                            // (rows of one head apart: what lies behind 128 bytes may be another head's)
                            s_slot == a.d ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

size_t tree_attn_workspace_bytes(int d) {
  const size_t rows = (size_t)ta::kGrid * 2 * ta::kRows;
  return rows * d * sizeof(float) + rows * sizeof(float2) + ta::kGrid * sizeof(ta::Record);
}

cudaError_t launch_tree_attn(const TreeAttnArgs& a, void* workspace, cudaStream_t stream) {
  const int tile = ta::tile_of(a.d);
  ta::Params p;
  p.q = a.q;
  p.out = a.out;
  p.lse = a.lse;
  p.block_table = a.block_table;
  p.indptr = a.indptr;
  p.kv_lens = a.kv_lens;
  p.mask = a.mask;
  p.positions = a.positions;
  const size_t n = (size_t)ta::kGrid * 2 * ta::kRows;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + n * a.d);
  p.q_tok = a.q_tok;
  p.q_head = a.q_head;
  p.total = a.total;
  p.batch = a.batch;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages_per_seq;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.group = a.hq / a.hkv;
  p.words = a.words;
  for (p.gang_shift = 0; p.gang_shift < ta::kGangShift && (a.hkv >> p.gang_shift) % 2 == 0; ++p.gang_shift) {
  }
  const int box = a.page_size < tile ? a.page_size : tile;
  for (p.page_shift = 0; (1 << p.page_shift) < a.page_size; ++p.page_shift) {
  }
  for (p.box_shift = 0; (1 << p.box_shift) < box; ++p.box_shift) {
  }
  // No unit is split if there are no more than blocks and their sequences cannot be long
  // (the kernel's own rule, by the lengths themselves); then nothing is to be joined.
  const int64_t rows = a.total * p.group;  // of a KV head; a sequence has ceil(its rows / kRows) blocks of them
  const int64_t units = a.hkv * (std::min(a.batch, a.total) + rows / ta::kRows);
  const bool whole = units <= (ta::kGrid >> p.gang_shift << p.gang_shift) &&
                     a.max_pages_per_seq * a.page_size <= (int64_t)ta::kWholeTiles * tile;
  p.record = whole ? nullptr : reinterpret_cast<ta::Record*>(p.part_ml + n);
  p.long_lists = units * 8 < ta::kGrid;
  const int64_t tiles = a.max_pages_per_seq * a.page_size / tile + 16;  // (of a unit, and what its ends count as)
  p.few = a.batch <= 32 && a.hkv * (rows / ta::kRows + 1) <= (int64_t(1) << 25) / tiles;
  p.row_groups = (int)((std::min<int64_t>(rows, ta::kRows) + 7) / 8);
  const double log2e = 1.4426950408889634;
  p.scale_log2 = (float)(a.scale * log2e);
  if (p.scale_log2 == 0.f) p.scale_log2 = std::numeric_limits<float>::min();  // (0 times a hidden score's infinity)
  // (a cap at the end of f32's range stays finite, twice itself too)
  const double cap = a.softcap * log2e, most = std::numeric_limits<float>::max() / 2;
  p.cap_out = a.softcap > 0.f ? (float)std::min(cap, most) : 0.f;
  p.cap_inv = a.softcap > 0.f ? (float)std::min(1.0 / cap, most) : 0.f;
  p.v_scale = a.v_scale;
  p.window = a.window;
  p.sinks = a.window > 0 ? a.sinks : 0;  // (without a window every token is visible)
  p.starve = a.starve;
  CUtensorMap k_map, v_map;
  cudaError_t e;
  if ((e = make_map(a.k_pages, a, a.kp_page, a.kp_head, a.kp_slot, box, &k_map)) != cudaSuccess) return e;
  if ((e = make_map(a.v_pages, a, a.vp_page, a.vp_head, a.vp_slot, box, &v_map)) != cudaSuccess) return e;
  static constexpr ta::Launch launch[4] = {ta::launch_f16, ta::launch_bf16, ta::launch_e4m3, ta::launch_e4m3_f16};
  return launch[a.cache](p, a.d, k_map, v_map, stream);
}

cudaError_t tree_attn_read_errors(uint32_t* word) {
  cudaError_t e = cudaDeviceSynchronize();
  *word = 0;
  for (auto read : {ta::read_errors_f16, ta::read_errors_bf16, ta::read_errors_e4m3, ta::read_errors_e4m3_f16}) {
    uint32_t w = 0;
    if (e == cudaSuccess) e = read(&w);
    *word |= w;
  }
  return e;
}

}  // namespace gqa
