// The norm's checks of arguments and entry points, and the fold of the
// backward's partial sums (kernels: norm_kernels.cuh).
#include "norm.cuh"
#include "prof.cuh"

namespace r4 {
namespace {

// out = (accumulate ? out : 0) + the sum of the partial rows, rounded once.
// A warp reads 32 neighbouring columns of every 32nd row; the 32 sums are
// added in order. Latency is all it has: 32 warps a block with five rows each
// take 0.6 us less of a backward than 16, and 2.7 less than 4.
constexpr int kFoldWarps = 32;
constexpr int kFoldRows = (kBwdBlocks + kFoldWarps - 1) / kFoldWarps;
__global__ void __launch_bounds__(32 * kFoldWarps) norm_fold_kernel(const float* partial, int blocks,
                                                                    int width, void* gw, void* gb, int type,
                                                                    int accumulate) {
  __shared__ float sums[kFoldWarps][32];
  begin_after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  void* out = blockIdx.y ? gb : gw;
  if (!out) return;
  const float* p = partial + (int64_t)blockIdx.y * blocks * width + c;
  float v[kFoldRows];  // all on their way at once
#pragma unroll
  for (int i = 0; i < kFoldRows; ++i) {
    const int b = warp + i * kFoldWarps;
    v[i] = c < width && b < blocks ? p[(int64_t)b * width] : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kFoldRows; ++i) s += v[i];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= width) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kFoldWarps; ++i) s += sums[i][lane];
  if (accumulate) s += load_as(out, type, c);
  if (type == RAWINT4_TYPE_F32) static_cast<float*>(out)[c] = s;
  else if (type == RAWINT4_TYPE_BF16) static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
  else static_cast<__half*>(out)[c] = __float2half_rn(s);
}

bool cfg_ok(const rawint4_norm_cfg* c) {
  return c && c->rows >= 0 && c->rows <= 1 << 30 && c->width >= 1 && c->width <= kMaxWidth && type_ok(c->type) && type_ok(c->weight_type) &&
         (c->kind == RAWINT4_NORM_LAYER || c->kind == RAWINT4_NORM_RMS) && c->eps > 0.f && c->eps <= FLT_MAX;
}

// One of x and the checkpoint: fills the input fields of `a`.
bool input_ok(const rawint4_norm_cfg* c, const void* x, int64_t ldx, const rawint4_ckpt8* in, NormArgs& a) {
  if ((x != nullptr) == (in != nullptr)) return false;
  if (in) {
    if (!ckpt_format_ok(in->format) || !in->codes || !in->scales) return false;
    a.in_codes = in->codes;
    a.in_scales = in->scales;
    a.in_fmt = in->format;
    return true;
  }
  a.x = x;
  a.ldx = ldx;
  return ldx >= c->width && ldx <= kMaxPitch;
}

bool input_aligned(const NormArgs& a, int type) {
  return a.width % kChunk == 0 &&
         (a.in_codes ? reinterpret_cast<uintptr_t>(a.in_codes) % 8 == 0 : rows_aligned(a.x, a.ldx, type));
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

NormArgs common_args(const rawint4_norm_cfg* c, const void* weight) {
  NormArgs a{};
  a.rows = c->rows;
  a.width = c->width;
  a.groups = (int)ckpt_groups(c->width);
  a.layer = c->kind == RAWINT4_NORM_LAYER;
  a.w_type = c->weight_type;
  a.eps = c->eps;
  a.weight = weight;
  return a;
}

int64_t code_bytes(const NormArgs& a) { return (int64_t)a.rows * a.width; }
int64_t scale_bytes(const NormArgs& a) { return (int64_t)a.rows * a.groups; }

}  // namespace
}  // namespace r4

using namespace r4;

extern "C" {

RAWINT4_API int rawint4_norm_fwd(const rawint4_norm_cfg* cfg, const void* x, int64_t ldx, const rawint4_ckpt8* x_ckpt,
                                 const void* weight, const void* bias, void* y, float* mean, float* rstd,
                                 int32_t save_format, uint8_t* save_codes, uint8_t* save_scales, void* stream_) {
  if (!cfg_ok(cfg)) return RAWINT4_INVALID_ARGUMENT;
  if (cfg->rows == 0) return RAWINT4_OK;
  NormArgs a = common_args(cfg, weight);
  if (!input_ok(cfg, x, ldx, x_ckpt, a) || !y || !rstd || (a.layer ? mean == nullptr : mean != nullptr) ||
      (save_codes != nullptr) != (save_scales != nullptr) || (save_codes && (x_ckpt || !ckpt_format_ok(save_format))))
    return RAWINT4_INVALID_ARGUMENT;
  const int64_t size = (int64_t)type_size(cfg->type), wsize = (int64_t)type_size(cfg->weight_type);
  if (!spans_ok({{x, span_bytes(a.rows, a.width, a.ldx, size), size}, {a.in_codes, code_bytes(a), 1},
                 {a.in_scales, scale_bytes(a), 1}, {weight, a.width * wsize, wsize}, {bias, a.width * wsize, wsize}},
                {{y, code_bytes(a) * size, size}, {mean, a.rows * (int64_t)4, 4}, {rstd, a.rows * (int64_t)4, 4},
                 {save_codes, code_bytes(a), 1}, {save_scales, scale_bytes(a), 1}}))
    return RAWINT4_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != RAWINT4_OK) return rc;
  a.bias = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.codes = save_codes;
  a.scales = save_scales;
  a.fmt = save_format;
  a.vec = input_aligned(a, cfg->type) && rows_aligned(y, a.width, cfg->type) && aligned16(weight) &&
                   aligned16(bias) && reinterpret_cast<uintptr_t>(save_codes) % 8 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream_);
  R4_PROF("norm_fwd", st);
  cudaError_t err;
  if (cfg->type == RAWINT4_TYPE_F32) err = run_norm_fwd<float>(a, cfg->type, st);
  else if (cfg->type == RAWINT4_TYPE_BF16) err = run_norm_fwd<__nv_bfloat16>(a, cfg->type, st);
  else err = run_norm_fwd<__half>(a, cfg->type, st);
  return err == cudaSuccess ? RAWINT4_OK : RAWINT4_CUDA_ERROR;
}

RAWINT4_API int rawint4_norm_bwd_workspace_size(const rawint4_norm_cfg* cfg, size_t* bytes) {
  if (!cfg_ok(cfg) || !bytes) return RAWINT4_INVALID_ARGUMENT;
  const size_t blocks = cfg->rows < kBwdBlocks ? cfg->rows : kBwdBlocks;
  const size_t n = 2 * blocks * cfg->width * sizeof(float);
  *bytes = (n + 255) / 256 * 256;
  return RAWINT4_OK;
}

RAWINT4_API int rawint4_norm_bwd(const rawint4_norm_cfg* cfg, const void* x, int64_t ldx, const rawint4_ckpt8* x_ckpt,
                                 const void* grad_y, int64_t ldg, const void* weight, const float* mean,
                                 const float* rstd, void* grad_x, void* grad_weight, void* grad_bias, int accumulate,
                                 void* workspace, size_t ws_bytes, void* stream_) {
  size_t need = 0;
  if (rawint4_norm_bwd_workspace_size(cfg, &need) != RAWINT4_OK) return RAWINT4_INVALID_ARGUMENT;
  NormArgs a = common_args(cfg, weight);
  const bool sums = grad_weight || grad_bias;
  if (a.rows > 0 &&
      (!input_ok(cfg, x, ldx, x_ckpt, a) || !grad_y || !grad_x || !rstd || ldg < a.width || ldg > kMaxPitch ||
       (a.layer ? mean == nullptr : mean != nullptr) ||
       (sums && (!workspace || ws_bytes < need))))
    return RAWINT4_INVALID_ARGUMENT;
  const int64_t size = (int64_t)type_size(cfg->type), wsize = (int64_t)type_size(cfg->weight_type);
  if (!spans_ok({{x, span_bytes(a.rows, a.width, a.ldx, size), size}, {a.in_codes, code_bytes(a), 1},
                 {a.in_scales, scale_bytes(a), 1}, {grad_y, span_bytes(a.rows, a.width, ldg, size), size},
                 {weight, a.width * wsize, wsize}, {mean, a.rows * (int64_t)4, 4}, {rstd, a.rows * (int64_t)4, 4}},
                {{grad_x, code_bytes(a) * size, size}, {grad_weight, a.width * wsize, wsize},
                 {grad_bias, a.width * wsize, wsize}, {sums ? workspace : nullptr, (int64_t)need, 16}}))
    return RAWINT4_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != RAWINT4_OK) return rc;
  a.gy = grad_y;
  a.ldg = ldg;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.gx = grad_x;
  a.partial = static_cast<float*>(workspace);
  a.want_w = grad_weight != nullptr;
  a.want_b = grad_bias != nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream_);
  if (a.rows > 0) {
    a.vec = input_aligned(a, cfg->type) && rows_aligned(grad_y, ldg, cfg->type) &&
                     rows_aligned(grad_x, a.width, cfg->type) && aligned16(weight);
    R4_PROF("norm_bwd", st);
    cudaError_t err;
    if (cfg->type == RAWINT4_TYPE_F32) err = run_norm_bwd<float>(a, cfg->type, st);
    else if (cfg->type == RAWINT4_TYPE_BF16) err = run_norm_bwd<__nv_bfloat16>(a, cfg->type, st);
    else err = run_norm_bwd<__half>(a, cfg->type, st);
    if (err != cudaSuccess) return RAWINT4_CUDA_ERROR;
  }
  if (sums) {
    R4_PROF("norm_fold", st);
    if (launch_early(norm_fold_kernel, dim3(ceil_div(a.width, 32), 2), 32 * kFoldWarps, 0, st, a.partial,
                     bwd_blocks(bwd_shape(a), a.rows), a.width, grad_weight, grad_bias, cfg->weight_type,
                     accumulate) != cudaSuccess)
      return RAWINT4_CUDA_ERROR;
  }
  return RAWINT4_OK;
}

}  // extern "C"
