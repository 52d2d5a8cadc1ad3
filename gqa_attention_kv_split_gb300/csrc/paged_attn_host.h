// paged_attn_host.h -- what the host side and the kernels of the one-token
// paged attention share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.h"

namespace gqa {
namespace pa {

constexpr int kGrid = 152;  // blocks: one per SM
constexpr int kGangShift = 3;  // log2 of the largest gang: 152 blocks are 19 gangs of 8
constexpr int kWholeTiles = 8;  // sequences of up to so many tiles are not split if there is a block for each unit

// Tokens per ring stage, from the bytes of a token's row: 16 to 32 KB of K and V a stage.
// (48 sequences of up to 16001 tokens in E4M3 pages, head dim 64: 90 us with 8 KB, 74 with
// 16; head dim 128: 124 us with 16 KB, 126 with 32; with one term a weight.)
constexpr int tile_of(int row_bytes) { return row_bytes > 256 ? 32 : row_bytes > 64 ? 64 : 128; }

// For the joining kernel: a unit and the gangs that have a piece of it.
struct Record {
  int b, unit;      // sequence, unit within it
  int first, last;  // last < 0: the unit lies inside one block (or there is no unit)
  int first_slot;   // which of the first gang's two pieces it is (it is the first one of the others)
};

struct Params {
  const void* q;
  void* out;
  float* lse;
  const int32_t* block_table;
  const int32_t* seq_lens;
  float* part_o;     // [kGrid][2][kRows][D]
  float2* part_ml;   // [kGrid][2][kRows]
  Record* record;    // [records], or null: no unit can be split (there is no second kernel)
  int records;       // one for each unit, or for each block the unit that begins there and
  int record_by_unit;  // ends elsewhere
  int64_t q_seq, q_head, batch, num_pages, max_pages;
  int hq, hkv, group, head_blocks;
  int gang_shift;    // log2 of the blocks of a gang: the largest power of two up to 8 that divides a sequence's units
  int page_shift, box_shift;  // log2 of a page's tokens, and of those of one copy
  float scale_log2;  // scores to the exp2 domain
  float cap_out, cap_inv;  // the cap of the scores in the exp2 domain (0: none), and its reciprocal
  float v_scale;
  int window, sinks, starve;
};

// The instances of one cache type, each in a translation unit of its own, and those with
// sinks in others.
using Launch = cudaError_t (*)(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_bf16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_e4m3(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_e4m3_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_sinks_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_sinks_bf16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_sinks_e4m3(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_sinks_e4m3_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t read_errors_f16(uint32_t* word);
cudaError_t read_errors_bf16(uint32_t* word);
cudaError_t read_errors_e4m3(uint32_t* word);
cudaError_t read_errors_sinks_f16(uint32_t* word);
cudaError_t read_errors_sinks_bf16(uint32_t* word);
cudaError_t read_errors_sinks_e4m3(uint32_t* word);

}  // namespace pa
}  // namespace gqa
