// paged.h -- interface between the C-ABI host layer (api.cpp) and the kernels that fill
// and read paged caches of any layout: the append (append.cu) and the one-token
// attention (paged_attn.cpp).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace gqa {

// ---- append of new keys and values to a paged cache -------------------------

enum AppendMode { kAppendSame = 0, kAppendE4m3 = 1, kAppendNvfp4 = 2 };

// Strides are in elements (an E4M3 element is a byte).  q may be null: k and v only.
struct AppendArgs {
  const void *q, *k, *v;       // [total, heads, d] f16 or bf16, last dimension contiguous
  void* q_out;                 // the rotated queries: the inputs' type, or E4M3 (NVFP4 pages)
  void *k_pages, *v_pages;     // [num_pages, hkv, page_size, d], or NVFP4 codes [num_pages, 8, 64, 64]
  uint8_t *k_sf, *v_sf;        // NVFP4 scales [num_pages, 8, 64, 8]
  const int32_t* block_table;  // [batch, max_pages_per_seq]
  const int32_t* kv_lens;      // [batch], the new tokens included
  const int32_t* indptr;       // [batch + 1], or null: one token per sequence
  const float* rope;           // [rope_len, rot]: rot / 2 cosines, then rot / 2 sines; or null
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, qo_tok, qo_head;
  int64_t kp_page, kp_head, kp_slot, vp_page, vp_head, vp_slot;
  int64_t total, batch, num_pages, max_pages_per_seq, rope_len;
  int hq, hkv, d, page_size, rot, interleaved, bf16;
  int mode;                    // an AppendMode
  int tok_per_block;           // set by launch_append
  float inv_k, inv_v, inv_q;   // reciprocals of the scales of E4M3 values
};

cudaError_t launch_append(AppendArgs a, cudaStream_t stream);
cudaError_t append_read_errors(uint32_t* word);

// ---- one-token attention over a paged cache ---------------------------------

// The pages' type, and with it the queries' and outputs': f16 pages, bf16 pages, E4M3
// pages with bf16 queries, E4M3 pages with f16 queries.
enum CacheType { kCacheF16 = 0, kCacheBf16 = 1, kCacheE4m3 = 2, kCacheE4m3F16 = 3 };

struct PagedAttnArgs {
  const void* q;               // [batch, hq, d] f16 or bf16
  void* out;                   // [batch, hq, d], q's type, dense
  float* lse;                  // [batch, hq] or null
  const void *k_pages, *v_pages;
  const int32_t* block_table;  // [batch, max_pages_per_seq]
  const int32_t* seq_lens;     // [batch]
  int64_t q_seq, q_head;       // elements
  int64_t kp_page, kp_head, kp_slot, vp_page, vp_head, vp_slot;  // elements
  int64_t batch, num_pages, max_pages_per_seq;
  int hq, hkv, d, page_size;
  int cache;                   // a CacheType
  float scale, v_scale;        // of the scores (q_scale * k_scale / sqrt(d)) and of the output
  float softcap;               // 0: none
  int window;                  // 0: none
  int starve;
};

// Bytes of scratch of a call (a bound that depends on the head layout alone).
size_t paged_attn_workspace_bytes(int hq, int hkv, int d);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, void* workspace, cudaStream_t stream);
cudaError_t paged_attn_read_errors(uint32_t* word);

}  // namespace gqa
