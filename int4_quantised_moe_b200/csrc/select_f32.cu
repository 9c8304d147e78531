// Expert selection for scores of one type (the types compile in parallel).
#include "select_kernels.cuh"

namespace r4 {

template <>
cudaError_t run_select<float>(const SelectArgs& a, int sms, cudaStream_t st) {
  return select_type<float>(a, sms, st);
}
template <>
cudaError_t run_select_bwd<float>(const SelectArgs& a, cudaStream_t st) {
  return select_bwd_type<float>(a, st);
}

}  // namespace r4
