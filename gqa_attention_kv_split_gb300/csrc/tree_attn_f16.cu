// tree_attn_f16.cu -- the instances of tree_attn.cuh over f16 pages.
#include "tree_attn.cuh"

namespace gqa {
namespace ta {

cudaError_t launch_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  return launch_cache<kCacheF16>(p, d, k_map, v_map, stream);
}

cudaError_t read_errors_f16(uint32_t* word) { return read_errors_here(word); }

}  // namespace ta
}  // namespace gqa
