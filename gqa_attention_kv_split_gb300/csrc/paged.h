// paged.h -- interface between the C-ABI host layer (api_paged.cpp) and the kernels that
// fill and read paged caches of any layout: the append (append.cuh), the one-token
// attention (paged_attn.cpp), and masks and compaction of drafted tokens (drafts.cu).
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
  const void *q_norm, *k_norm; // [d] weights of the heads' norms, the inputs' type or f32; or null: no norm
  const int32_t* positions;    // [total] rows of the rope table; or null: each token's place in the cache
  int norm_f32;
  float norm_eps;
};

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t append_read_errors(uint32_t* word);
// Of the instances with norms and positions (append_norm.cu).
cudaError_t launch_append_norm(const AppendArgs& a, cudaStream_t stream);
cudaError_t append_norm_read_errors(uint32_t* word);

// ---- drafted tokens: trees, compaction --------------------------------------

constexpr int kMaxTreeTokens = 1024;  // a row of bits has up to 32 words

struct TreeMaskArgs {
  const int32_t* parents;   // [total]
  const int32_t* indptr;    // [batch + 1]
  const int32_t* kv_lens;   // [batch], the drafted tokens included
  uint32_t* mask;           // [total, words]
  int32_t* positions;       // [total]
  int64_t total, batch;
  int words, window, sinks;
};
cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t stream);

// One tensor of pages [layers, num_pages, heads, page_size, row]; strides in bytes.
struct KeepTensor {
  uint8_t* data;
  int64_t s_layer, s_page, s_head, s_slot;
  int64_t items;    // layers * heads * pieces
  int64_t heads, pieces;  // pieces of `vec` bytes in a row
  int vec;          // 16 or 8
};
constexpr int kKeepTensors = 4;
struct KeepArgs {
  KeepTensor t[kKeepTensors];
  int tensors;
  const int32_t* block_table;  // [batch, max_pages]
  const int32_t* indptr;       // [batch + 1]
  const int32_t* kv_lens;      // [batch], the drafted tokens included
  const int32_t* kept;         // [batch, max_kept]
  const int32_t* num_kept;     // [batch]
  int32_t* new_lens;           // [batch]
  int64_t batch, max_pages, num_pages, max_kept, page_size;
};
cudaError_t launch_keep(const KeepArgs& a, cudaStream_t stream);
cudaError_t drafts_read_errors(uint32_t* word);

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
  int sinks;                   // first tokens that stay visible under a window
  int starve;
};

// Bytes of scratch of a call (a bound that depends on the head layout alone).
size_t paged_attn_workspace_bytes(int hq, int hkv, int d);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, void* workspace, cudaStream_t stream);
cudaError_t paged_attn_read_errors(uint32_t* word);

// ---- attention of several new tokens per sequence over a paged cache ---------

// The most work of a call, in tiles of K and V and what the units' ends count as: a block counts its share in 31 bits.
constexpr int64_t kTreeMostWork = int64_t(1) << 38;

struct TreeAttnArgs {
  const void* q;               // [total, hq, d] f16 or bf16
  void* out;                   // [total, hq, d], q's type, dense
  float* lse;                  // [total, hq] or null
  const void *k_pages, *v_pages;
  const int32_t* block_table;  // [batch, max_pages_per_seq]
  const int32_t* indptr;       // [batch + 1]
  const int32_t* kv_lens;      // [batch], the new tokens included
  const int32_t* mask;         // [total, words], or null: chains
  const int32_t* positions;    // [total], or null
  int64_t q_tok, q_head;       // elements
  int64_t kp_page, kp_head, kp_slot, vp_page, vp_head, vp_slot;  // elements
  int64_t total, batch, num_pages, max_pages_per_seq;
  int hq, hkv, d, page_size, words;
  int cache;                   // a CacheType
  float scale, v_scale;        // of the scores (q_scale * k_scale / sqrt(d)) and of the output
  float softcap;               // 0: none
  int window, sinks;           // 0: none
  int starve;
};

// Bytes of scratch of a call (a bound that depends on the head dim alone).
size_t tree_attn_workspace_bytes(int d);
cudaError_t launch_tree_attn(const TreeAttnArgs& a, void* workspace, cudaStream_t stream);
cudaError_t tree_attn_read_errors(uint32_t* word);

}  // namespace gqa
