// paged_attn_bf16.cu -- the instances of paged_attn.cuh over bf16 pages.
#include "paged_attn.cuh"

namespace gqa {
namespace pa {

cudaError_t launch_bf16(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  return launch_cache<kCacheBf16>(p, d, k_map, v_map, stream);
}

cudaError_t read_errors_bf16(uint32_t* word) { return read_errors_here(word); }

}  // namespace pa
}  // namespace gqa
