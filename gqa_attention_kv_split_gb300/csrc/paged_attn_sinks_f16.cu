// paged_attn_sinks_f16.cu -- the instances with sinks of paged_attn.cuh over f16 pages.
#include "paged_attn.cuh"

namespace gqa {
namespace pa {

cudaError_t launch_sinks_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  return launch_cache<kCacheF16, true>(p, d, k_map, v_map, stream);
}

cudaError_t read_errors_sinks_f16(uint32_t* word) { return read_errors_here(word); }

}  // namespace pa
}  // namespace gqa
