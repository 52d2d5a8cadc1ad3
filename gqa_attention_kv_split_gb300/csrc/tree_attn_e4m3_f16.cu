// tree_attn_e4m3_f16.cu -- the instances of tree_attn.cuh over E4M3 pages with f16 queries.
#include "tree_attn.cuh"

namespace gqa {
namespace ta {

cudaError_t launch_e4m3_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  return launch_cache<kCacheE4m3F16>(p, d, k_map, v_map, stream);
}

cudaError_t read_errors_e4m3_f16(uint32_t* word) { return read_errors_here(word); }

}  // namespace ta
}  // namespace gqa
