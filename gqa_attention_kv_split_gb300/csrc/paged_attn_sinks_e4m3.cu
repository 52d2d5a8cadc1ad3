// paged_attn_sinks_e4m3.cu -- the instances with sinks of paged_attn.cuh over E4M3 pages (bf16 and f16 queries).
#include "paged_attn.cuh"

namespace gqa {
namespace pa {

cudaError_t launch_sinks_e4m3(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  return launch_cache<kCacheE4m3, true>(p, d, k_map, v_map, stream);
}

cudaError_t launch_sinks_e4m3_f16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  return launch_cache<kCacheE4m3F16, true>(p, d, k_map, v_map, stream);
}

cudaError_t read_errors_sinks_e4m3(uint32_t* word) { return read_errors_here(word); }

}  // namespace pa
}  // namespace gqa
