// append_norm.cu -- the instances of append.cuh with norms of the heads and given positions.
#include "append.cuh"

namespace gqa {

cudaError_t launch_append_norm(const AppendArgs& a, cudaStream_t stream) { return launch_here<true>(a, stream); }

cudaError_t append_norm_read_errors(uint32_t* word) { return read_errors_here(word); }

}  // namespace gqa
