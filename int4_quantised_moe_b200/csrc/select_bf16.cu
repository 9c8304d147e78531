// Expert selection for scores of one type (the types compile in parallel).
#include "select_kernels.cuh"

namespace r4 {

template <>
cudaError_t run_select<__nv_bfloat16>(const SelectArgs& a, int sms, cudaStream_t st) {
  return select_type<__nv_bfloat16>(a, sms, st);
}
template <>
cudaError_t run_select_bwd<__nv_bfloat16>(const SelectArgs& a, cudaStream_t st) {
  return select_bwd_type<__nv_bfloat16>(a, st);
}

}  // namespace r4
