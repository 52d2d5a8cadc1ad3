// tree_attn_host.h -- what the host side and the kernels of the paged attention of
// several new tokens (trees and chains of drafted ones) share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.h"

namespace gqa {
namespace ta {

constexpr int kGrid = 152;      // blocks: one per SM
constexpr int kGangShift = 3;   // log2 of the largest gang: 152 blocks are 19 gangs of 8
constexpr int kRows = 128;      // rows (tokens x heads of a KV head) of a unit: the MMA's M
constexpr int kWholeTiles = 4;  // sequences of up to so many tiles are not split if there is a block for each unit

// Tokens of a tile of K and V: what leaves room for two tiles and the queries at head dim 256.
constexpr int tile_of(int d) { return d > 128 ? 64 : 128; }

// For the joining kernel: a unit that begins in one block's share and ends in another's.
struct Record {
  int64_t row0;     // the sequence's first new token
  int kv_head, row; // the unit: rows [row, row + rows) of a KV head's
  int rows, lane;   // and its block's place in a gang
  int first, last;  // gangs that have a piece of it; last < 0: no such unit
  int first_slot;   // which of the first gang's two pieces it is (it is the first one of the others)
};

struct Params {
  const void* q;
  void* out;
  float* lse;
  const int32_t* block_table;
  const int32_t* indptr;
  const int32_t* kv_lens;
  const int32_t* mask;       // [total, words], or null: chains
  const int32_t* positions;  // [total], or null
  float* part_o;             // [kGrid][2][kRows][D]
  float2* part_ml;           // [kGrid][2][kRows]
  Record* record;            // [kGrid], or null: no unit can be split (there is no second kernel)
  int64_t q_tok, q_head, total, batch, num_pages, max_pages;
  int hq, hkv, group, words;
  int gang_shift;            // log2 of the blocks of a gang: the largest power of two up to 8 that divides the KV heads
  int page_shift, box_shift; // log2 of a page's tokens, and of those of one copy
  int row_groups;            // of 8 rows: what the joining kernel's grid covers
  float scale_log2;          // scores to the exp2 domain
  float cap_out, cap_inv;    // the cap of the scores in the exp2 domain (0: none), and its reciprocal
  float v_scale;
  int window, sinks, starve;
  int long_lists;            // so few units that one has more than about 8 pieces
  int few;                   // up to 32 sequences, and less than 2^31 of work whatever their offsets and lengths
};

// The instances of one cache type, each in a translation unit of its own.
using Launch = cudaError_t (*)(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_bf16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_e4m3(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_e4m3_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t read_errors_f16(uint32_t* word);
cudaError_t read_errors_bf16(uint32_t* word);
cudaError_t read_errors_e4m3(uint32_t* word);
cudaError_t read_errors_e4m3_f16(uint32_t* word);

}  // namespace ta
}  // namespace gqa
