// The norm's backward for one element type (the directions and types compile in parallel).
#include "norm_kernels.cuh"

namespace r4 {

template <>
cudaError_t run_norm_bwd<float>(const NormArgs& a, int type, cudaStream_t st) {
  return bwd_type<float>(a, type, st);
}

}  // namespace r4
