// append.cu -- the instances of append.cuh without a norm, and the choice between the two.
#include "append.cuh"

namespace gqa {

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  // (positions without a norm: the other instances, whose weights are then left out)
  return a.q_norm || a.k_norm || a.positions ? launch_append_norm(a, stream) : launch_here<false>(a, stream);
}

cudaError_t append_read_errors(uint32_t* word) {
  uint32_t w[2] = {0, 0};
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = read_errors_here(&w[0]);
  if (e == cudaSuccess) e = append_norm_read_errors(&w[1]);
  *word = w[0] | w[1];
  return e;
}

}  // namespace gqa
