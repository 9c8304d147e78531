// The norm's forward (the directions and types compile in parallel).
#include "norm_kernels.cuh"

namespace r4 {

template <>
cudaError_t run_norm_fwd<float>(const NormArgs& a, int type, cudaStream_t st) {
  return fwd_type<float>(a, type, st);
}
template <>
cudaError_t run_norm_fwd<__nv_bfloat16>(const NormArgs& a, int type, cudaStream_t st) {
  return fwd_type<__nv_bfloat16>(a, type, st);
}
template <>
cudaError_t run_norm_fwd<__half>(const NormArgs& a, int type, cudaStream_t st) {
  return fwd_type<__half>(a, type, st);
}

}  // namespace r4
