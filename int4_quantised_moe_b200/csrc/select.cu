// Expert selection and its backward: checks of arguments and entry points
// (kernels: select_kernels.cuh).
#include "prof.cuh"
#include "select.cuh"

namespace r4 {
namespace {

// A memset would end the chain of kernels that start early (8192 x 384 with
// counts: 2 us more).
__global__ void __launch_bounds__(256) clear_counts_kernel(int32_t* counts, int E) {
  begin_after_previous();
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e < E) counts[e] = 0;
}

bool cfg_ok(const rawint4_moe_select_cfg* c) {
  if (!c || c->experts < 1 || c->experts > 4096 || c->top_k < 1 || c->top_k > 32 || c->groups < 1 || c->groups > 32 ||
      c->experts % c->groups != 0 || c->groups_kept < 1 || c->groups_kept > c->groups)
    return false;
  const int size = c->experts / c->groups;
  return c->group_top >= 1 && c->group_top <= 2 && (c->groups == 1 || c->group_top <= size) &&
         c->top_k <= c->groups_kept * size && (c->score == RAWINT4_SCORE_SOFTMAX || c->score == RAWINT4_SCORE_SIGMOID) &&
         type_ok(c->type) && c->scale == c->scale && fabsf(c->scale) <= FLT_MAX;
}

SelectArgs common_args(const rawint4_moe_select_cfg* c, const void* scores, int64_t ld, int32_t qlen) {
  SelectArgs a{};
  a.scores = scores;
  a.ld = ld;
  a.Q = qlen;
  a.E = c->experts;
  a.k = c->top_k;
  a.groups = c->groups;
  a.kept = c->groups_kept;
  a.group_top = c->groups > 1 ? c->group_top : 1;
  a.sigmoid = c->score == RAWINT4_SCORE_SIGMOID;
  a.renorm = c->renormalise != 0;
  a.scale = c->scale;
  return a;
}

bool scores_ok(const rawint4_moe_select_cfg* c, const void* scores, int64_t ld, int32_t qlen) {
  return qlen >= 0 && qlen <= 1 << 30 && ld >= c->experts && ld <= kMaxPitch && (qlen == 0 || scores);
}

}  // namespace
}  // namespace r4

using namespace r4;

extern "C" {

RAWINT4_API int rawint4_moe_router_select(const rawint4_moe_select_cfg* cfg, const void* scores, int64_t ld, int32_t qlen,
                                          const float* bias, int64_t* ids, float* weights, int32_t* counts,
                                          void* stream_) {
  if (!cfg_ok(cfg) || !scores_ok(cfg, scores, ld, qlen) || (qlen > 0 && (!ids || !weights))) return RAWINT4_INVALID_ARGUMENT;
  const int64_t size = (int64_t)type_size(cfg->type), slots = (int64_t)qlen * cfg->top_k;
  if (!spans_ok({{scores, span_bytes(qlen, cfg->experts, ld, size), size}, {bias, cfg->experts * (int64_t)4, 4}},
                {{ids, slots * 8, 8}, {weights, slots * 4, 4}, {counts, cfg->experts * (int64_t)4, 4}}))
    return RAWINT4_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != RAWINT4_OK) return rc;
  SelectArgs a = common_args(cfg, scores, ld, qlen);
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.counts = counts;
  cudaStream_t st = static_cast<cudaStream_t>(stream_);
  if (counts && launch_early(clear_counts_kernel, (a.E + 255) / 256, 256, 0, st, counts, a.E) != cudaSuccess)
    return RAWINT4_CUDA_ERROR;
  if (qlen == 0) return RAWINT4_OK;
  R4_PROF("router_select", st);
  cudaError_t err;
  if (cfg->type == RAWINT4_TYPE_F32) err = run_select<float>(a, sms, st);
  else if (cfg->type == RAWINT4_TYPE_BF16) err = run_select<__nv_bfloat16>(a, sms, st);
  else err = run_select<__half>(a, sms, st);
  return err == cudaSuccess ? RAWINT4_OK : RAWINT4_CUDA_ERROR;
}

RAWINT4_API int rawint4_moe_router_select_bwd(const rawint4_moe_select_cfg* cfg, const void* scores, int64_t ld,
                                              int32_t qlen, const int64_t* ids, const float* grad_route,
                                              void* grad_scores, void* stream_) {
  if (!cfg_ok(cfg) || !scores_ok(cfg, scores, ld, qlen) || (qlen > 0 && (!ids || !grad_route || !grad_scores)))
    return RAWINT4_INVALID_ARGUMENT;
  if (qlen == 0) return RAWINT4_OK;
  const int64_t size = (int64_t)type_size(cfg->type), slots = (int64_t)qlen * cfg->top_k;
  if (!spans_ok({{scores, span_bytes(qlen, cfg->experts, ld, size), size}, {ids, slots * 8, 8}, {grad_route, slots * 4, 4}},
                {{grad_scores, (int64_t)qlen * cfg->experts * size, size}}))
    return RAWINT4_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != RAWINT4_OK) return rc;
  SelectArgs a = common_args(cfg, scores, ld, qlen);
  a.ids_in = ids;
  a.grad_route = grad_route;
  a.grad = grad_scores;
  cudaStream_t st = static_cast<cudaStream_t>(stream_);
  R4_PROF("router_select_bwd", st);
  cudaError_t err;
  if (cfg->type == RAWINT4_TYPE_F32) err = run_select_bwd<float>(a, st);
  else if (cfg->type == RAWINT4_TYPE_BF16) err = run_select_bwd<__nv_bfloat16>(a, st);
  else err = run_select_bwd<__half>(a, st);
  return err == cudaSuccess ? RAWINT4_OK : RAWINT4_CUDA_ERROR;
}

}  // extern "C"
