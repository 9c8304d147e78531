#pragma once
#include "rows.cuh"

namespace r4 {

struct SelectArgs {
  const void* scores;
  int64_t ld;
  int Q, E, k;
  int groups, kept, group_top;
  int sigmoid, renorm;
  float scale;
  const float* bias;
  int64_t* ids;
  float* weights;
  int32_t* counts;
  // backward
  const int64_t* ids_in;
  const float* grad_route;
  void* grad;
};

// Selection and its backward for scores of one type (select_f32.cu, select_bf16.cu, select_f16.cu); a.Q > 0.
template <class T>
cudaError_t run_select(const SelectArgs& a, int sms, cudaStream_t st);
template <class T>
cudaError_t run_select_bwd(const SelectArgs& a, cudaStream_t st);

}  // namespace r4
