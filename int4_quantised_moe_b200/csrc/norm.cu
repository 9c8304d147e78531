// The norm in front of the layer, forward and backward, layer norm or RMS
// norm. With mu the row mean (0 for RMS), r = 1 / sqrt(mean((x - mu)^2) + eps)
// and xh = (x - mu) r:
//     y  = xh w + b
//     dx = r (w dy - mean(w dy) - xh mean(w dy xh))      (RMS: no middle term)
//     dw = sum over rows of dy xh,  db = sum over rows of dy
// x is a tensor, or the 8-bit checkpoint of one (rows.cuh), decoded on load;
// the forward can write x's checkpoint in the same pass.
//
// A row lies in the registers of one warp (narrow rows, several warps a
// block) or of one block, so each input is read once: the mean, then the
// centred squares, are summed from registers in fp32. The backward keeps the
// sums of dw and db over a block's rows in registers as well; each block
// writes one partial row to the workspace and a second kernel adds the
// partials in block order, so the result does not depend on timing.
#include "prof.cuh"
#include "rows.cuh"

namespace r4 {
namespace {

constexpr int kMaxWidth = 16384;
constexpr int kWarpRows = 4;        // rows a block works on at a time when a row lies in one warp
constexpr int kMaxPartials = 296;   // blocks of the backward at most (two on each of 148 SMs): rows of partial sums

struct NormArgs {
  const void* x;            // elements of type T, or
  const uint8_t* in_codes;  // an 8-bit checkpoint
  const uint8_t* in_scales;
  int64_t ldx;
  int in_fmt;
  int rows, width, groups;
  int layer;                // subtract the mean
  int w_type;
  float eps;
  const void *weight, *bias;
  void* y;
  float *mean, *rstd;
  uint8_t *codes, *scales;  // checkpoint to write (null: none)
  int fmt;
  // backward
  const void* gy;
  int64_t ldg;
  const float *mean_in, *rstd_in;
  void* gx;
  float* partial;           // [2][blocks][width]: dw, db
  int want_w, want_b;
};

// Columns of this thread's element j of chunk i, in either layout.
template <bool VEC>
__device__ __forceinline__ int column(int i, int j, int t, int threads) {
  return VEC ? (i * threads + t) * kChunk + j : (i * kChunk + j) * threads + t;
}

template <class T>
__device__ __forceinline__ float any_load(const void* p, int64_t i) {
  return Elem<T>::to(static_cast<const T*>(p)[i]);
}
__device__ __forceinline__ float vec_load(const void* p, int type, int i) {
  if (type == RAWINT4_TYPE_F32) return any_load<float>(p, i);
  if (type == RAWINT4_TYPE_BF16) return any_load<__nv_bfloat16>(p, i);
  return any_load<__half>(p, i);
}

// Elements of one row of a tensor; columns past the width read as 0.
template <class T, int NV, bool VEC>
__device__ __forceinline__ void load_row(const T* row, int width, int t, int threads, float (&f)[NV * kChunk]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (VEC) {
      const int c0 = column<VEC>(i, 0, t, threads);
      if (c0 < width) {
        const RawChunk<T> r = load_chunk(row + c0);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) f[i * kChunk + j] = Elem<T>::to(r.v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) f[i * kChunk + j] = 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const int c = column<VEC>(i, j, t, threads);
        f[i * kChunk + j] = c < width ? Elem<T>::to(row[c]) : 0.f;
      }
    }
  }
}

template <class T, int NV, bool VEC>
__device__ __forceinline__ void store_row(T* row, int width, int t, int threads, const float (&f)[NV * kChunk]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (VEC) {
      const int c0 = column<VEC>(i, 0, t, threads);
      if (c0 < width) {
        float v[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) v[j] = f[i * kChunk + j];
        store_chunk(row + c0, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const int c = column<VEC>(i, j, t, threads);
        if (c < width) row[c] = Elem<T>::from(f[i * kChunk + j]);
      }
    }
  }
}

// The same from a checkpoint; values past fp32 saturate.
template <int NV, bool VEC>
__device__ __forceinline__ void load_ckpt_row(const uint8_t* codes, const uint8_t* scales, int fmt, int width, int t,
                                              int threads, float (&f)[NV * kChunk]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (VEC) {
      const int c0 = column<VEC>(i, 0, t, threads);
      if (c0 < width) {
        const uint2 w = *reinterpret_cast<const uint2*>(codes + c0);
        const float s = ckpt_scale(scales[c0 / kCkptGroup]);
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
          f[i * kChunk + j] = ckpt_saturate(ckpt_value(((j < 4 ? w.x : w.y) >> (8 * (j % 4))) & 0xFFu, s, fmt), FLT_MAX);
      } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) f[i * kChunk + j] = 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const int c = column<VEC>(i, j, t, threads);
        f[i * kChunk + j] =
            c < width ? ckpt_saturate(ckpt_value(codes[c], ckpt_scale(scales[c / kCkptGroup]), fmt), FLT_MAX) : 0.f;
      }
    }
  }
}

// Sum over the threads of a row: a warp, or the block (through `buf`, which
// the caller alternates so that one barrier a sum is enough).
__device__ __forceinline__ float2 row_sum2(float a, float b, int threads, float2* buf) {
  a = row_warp_sum(a);
  b = row_warp_sum(b);
  if (threads == 32) return make_float2(a, b);
  const int warps = threads >> 5;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const float2 v = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
  return make_float2(row_warp_sum(v.x), row_warp_sum(v.y));
}

// Writes the checkpoint of the row held in f. Called by all lanes of a warp.
template <int NV, bool VEC>
__device__ __forceinline__ void save_row(const float (&f)[NV * kChunk], uint8_t* codes, uint8_t* scales, int fmt,
                                         int width, int t, int threads) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (VEC) {
      const int c0 = column<VEC>(i, 0, t, threads);
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < kChunk; ++j) amax = max(amax, finite_abs_bits(f[i * kChunk + j]));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      if (c0 < width) {
        const uint32_t byte = ckpt_scale_byte(amax, fmt);
        const float inv = ckpt_inv_scale(byte);
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < kChunk; ++j) w[j / 4] |= ckpt_code(f[i * kChunk + j], inv, fmt) << (8 * (j % 4));
        *reinterpret_cast<uint2*>(codes + c0) = make_uint2(w[0], w[1]);
        if (c0 % kCkptGroup == 0) scales[c0 / kCkptGroup] = (uint8_t)byte;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const int c = column<VEC>(i, j, t, threads);
        const float v = f[i * kChunk + j];
        const uint32_t byte = ckpt_scale_byte(__reduce_max_sync(0xffffffffu, finite_abs_bits(v)), fmt);
        if (c < width) {
          codes[c] = (uint8_t)ckpt_code(v, ckpt_inv_scale(byte), fmt);
          if (c % kCkptGroup == 0) scales[c / kCkptGroup] = (uint8_t)byte;
        }
      }
    }
  }
}

// blockDim = (threads of a row, rows): the threads of a row are a warp when
// blockDim.y > 1, else the block.
template <class T, int NV, bool VEC, bool CKPT>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormArgs a) {
  __shared__ float2 buf[2][16];
  const int t = threadIdx.x, threads = blockDim.x;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;  // whole warps leave; a block-wide row never does
  float f[NV * kChunk];
  if (CKPT)
    load_ckpt_row<NV, VEC>(a.in_codes + (int64_t)row * a.width, a.in_scales + (int64_t)row * a.groups, a.in_fmt, a.width,
                           t, threads, f);
  else
    load_row<T, NV, VEC>(static_cast<const T*>(a.x) + row * a.ldx, a.width, t, threads, f);
  if (!CKPT && a.codes)
    save_row<NV, VEC>(f, a.codes + (int64_t)row * a.width, a.scales + (int64_t)row * a.groups, a.fmt, a.width, t, threads);
  const float inv_n = 1.0f / (float)a.width;
  float mu = 0.f;
  if (a.layer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV * kChunk; ++i) s += f[i];
    mu = row_sum2(s, 0.f, threads, buf[0]).x * inv_n;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const float d = column<VEC>(i, j, t, threads) < a.width ? f[i * kChunk + j] - mu : 0.f;
      f[i * kChunk + j] = d;
      q += d * d;
    }
  const float r = 1.0f / sqrtf(row_sum2(q, 0.f, threads, buf[1]).x * inv_n + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const int c = column<VEC>(i, j, t, threads);
      if (c < a.width) {
        float v = f[i * kChunk + j] * r;
        if (a.weight) v *= vec_load(a.weight, a.w_type, c);
        if (a.bias) v += vec_load(a.bias, a.w_type, c);
        f[i * kChunk + j] = v;
      }
    }
  store_row<T, NV, VEC>(static_cast<T*>(a.y) + (int64_t)row * a.width, a.width, t, threads, f);
  if (t == 0) {
    if (a.mean) a.mean[row] = mu;
    a.rstd[row] = r;
  }
}

template <class T, int NV, bool VEC, bool CKPT>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormArgs a) {
  __shared__ float2 buf[2][16];
  extern __shared__ float fold[];  // narrow rows: the warps' sums, [rows - 1][width] at a time
  const int t = threadIdx.x, threads = blockDim.x;
  const float inv_n = 1.0f / (float)a.width;
  float dw[NV * kChunk], db[NV * kChunk], w[NV * kChunk];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const int c = column<VEC>(i, j, t, threads);
      dw[i * kChunk + j] = db[i * kChunk + j] = 0.f;
      w[i * kChunk + j] = c < a.width ? (a.weight ? vec_load(a.weight, a.w_type, c) : 1.f) : 0.f;
    }
  int turn = 0;
  for (int row = blockIdx.x * blockDim.y + threadIdx.y; row < a.rows; row += gridDim.x * blockDim.y, turn ^= 1) {
    float f[NV * kChunk], g[NV * kChunk];
    if (CKPT)
      load_ckpt_row<NV, VEC>(a.in_codes + (int64_t)row * a.width, a.in_scales + (int64_t)row * a.groups, a.in_fmt,
                             a.width, t, threads, f);
    else
      load_row<T, NV, VEC>(static_cast<const T*>(a.x) + row * a.ldx, a.width, t, threads, f);
    load_row<T, NV, VEC>(static_cast<const T*>(a.gy) + row * a.ldg, a.width, t, threads, g);
    const float r = a.rstd_in[row], mu = a.layer ? a.mean_in[row] : 0.f;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV * kChunk; ++i) {
      const float xh = (f[i] - mu) * r, p = g[i] * w[i];
      dw[i] += g[i] * xh;
      db[i] += g[i];
      f[i] = xh;
      g[i] = p;
      s1 += p;
      s2 += p * xh;
    }
    const float2 s = row_sum2(s1, s2, threads, buf[turn]);
    const float m1 = a.layer ? s.x * inv_n : 0.f, m2 = s.y * inv_n;
#pragma unroll
    for (int i = 0; i < NV * kChunk; ++i) f[i] = r * (g[i] - m1 - f[i] * m2);
    store_row<T, NV, VEC>(static_cast<T*>(a.gx) + (int64_t)row * a.width, a.width, t, threads, f);
  }
  if (!a.want_w && !a.want_b) return;
  for (int pass = 0; pass < 2; ++pass) {
    if (!(pass ? a.want_b : a.want_w)) continue;
    if (blockDim.y > 1) {  // add the block's rows in order
      __syncthreads();
      for (int y = 0; y < (int)blockDim.y; ++y) {
        if ((int)threadIdx.y == y)
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < kChunk; ++j) {
              const int c = column<VEC>(i, j, t, threads);
              if (c < a.width) fold[c] = (y ? fold[c] : 0.f) + (pass ? db : dw)[i * kChunk + j];
            }
        __syncthreads();
      }
      float* out = a.partial + ((int64_t)pass * gridDim.x + blockIdx.x) * a.width;
      for (int c = threadIdx.y * threads + t; c < a.width; c += threads * blockDim.y) out[c] = fold[c];
    } else {
      float* out = a.partial + ((int64_t)pass * gridDim.x + blockIdx.x) * a.width;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          const int c = column<VEC>(i, j, t, threads);
          if (c < a.width) out[c] = (pass ? db : dw)[i * kChunk + j];
        }
    }
  }
}

// out = (accumulate ? out : 0) + the partial rows in order, rounded once.
__global__ void __launch_bounds__(256) norm_fold_kernel(const float* __restrict__ partial, int blocks, int width,
                                                        void* gw, void* gb, int type, int accumulate) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  void* out = blockIdx.y ? gb : gw;
  if (c >= width || !out) return;
  const float* p = partial + (int64_t)blockIdx.y * blocks * width + c;
  float s = accumulate ? vec_load(out, type, c) : 0.f;
  for (int b = 0; b < blocks; ++b) s += p[(int64_t)b * width];
  if (type == RAWINT4_TYPE_F32) static_cast<float*>(out)[c] = s;
  else if (type == RAWINT4_TYPE_BF16) static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
  else static_cast<__half*>(out)[c] = __float2half_rn(s);
}

struct Shape {
  int nv, threads, rows;  // chunks a thread, threads a row, rows a block
};

Shape shape_for(int width) {
  const int chunks = (width + kChunk - 1) / kChunk;
  if (chunks <= 32) return {1, 32, kWarpRows};
  if (chunks <= 64) return {2, 32, kWarpRows};
  if (chunks <= 128) return {4, 32, kWarpRows};
  const int nv = chunks <= 512 ? 2 : 4;
  return {nv, (chunks + nv * 32 - 1) / (nv * 32) * 32, 1};
}

int bwd_blocks(const Shape& s, int rows) {
  const int need = (rows + s.rows - 1) / s.rows;
  return need < kMaxPartials ? need : kMaxPartials;
}

template <class T, int NV, bool VEC, bool CKPT>
cudaError_t launch(const NormArgs& a, const Shape& s, bool bwd, cudaStream_t st) {
  const dim3 block(s.threads, s.rows);
  if (bwd)
    norm_bwd_kernel<T, NV, VEC, CKPT>
        <<<bwd_blocks(s, a.rows), block, s.rows > 1 ? a.width * sizeof(float) : 0, st>>>(a);
  else
    norm_fwd_kernel<T, NV, VEC, CKPT><<<(a.rows + s.rows - 1) / s.rows, block, 0, st>>>(a);
  return cudaGetLastError();
}

template <class T, int NV>
cudaError_t pick(const NormArgs& a, const Shape& s, bool vec, bool bwd, cudaStream_t st) {
  if (a.in_codes)
    return vec ? launch<T, NV, true, true>(a, s, bwd, st) : launch<T, NV, false, true>(a, s, bwd, st);
  return vec ? launch<T, NV, true, false>(a, s, bwd, st) : launch<T, NV, false, false>(a, s, bwd, st);
}

template <class T>
cudaError_t pick_nv(const NormArgs& a, const Shape& s, bool vec, bool bwd, cudaStream_t st) {
  if (s.nv == 1) return pick<T, 1>(a, s, vec, bwd, st);
  if (s.nv == 2) return pick<T, 2>(a, s, vec, bwd, st);
  return pick<T, 4>(a, s, vec, bwd, st);
}

cudaError_t run(const NormArgs& a, int type, bool vec, bool bwd, cudaStream_t st) {
  const Shape s = shape_for(a.width);
  if (type == RAWINT4_TYPE_F32) return pick_nv<float>(a, s, vec, bwd, st);
  if (type == RAWINT4_TYPE_BF16) return pick_nv<__nv_bfloat16>(a, s, vec, bwd, st);
  return pick_nv<__half>(a, s, vec, bwd, st);
}

bool cfg_ok(const rawint4_norm_cfg* c) {
  return c && c->rows >= 0 && c->width >= 1 && c->width <= kMaxWidth && type_ok(c->type) && type_ok(c->weight_type) &&
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
  const bool vec = input_aligned(a, cfg->type) && rows_aligned(y, a.width, cfg->type) &&
                   reinterpret_cast<uintptr_t>(save_codes) % 8 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream_);
  R4_PROF("norm_fwd", st);
  return run(a, cfg->type, vec, false, st) == cudaSuccess ? RAWINT4_OK : RAWINT4_CUDA_ERROR;
}

RAWINT4_API int rawint4_norm_bwd_workspace_size(const rawint4_norm_cfg* cfg, size_t* bytes) {
  if (!cfg_ok(cfg) || !bytes) return RAWINT4_INVALID_ARGUMENT;
  const size_t n = (size_t)2 * bwd_blocks(shape_for(cfg->width), cfg->rows) * cfg->width * sizeof(float);
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
    const bool vec = input_aligned(a, cfg->type) && rows_aligned(grad_y, ldg, cfg->type) &&
                     rows_aligned(grad_x, a.width, cfg->type);
    R4_PROF("norm_bwd", st);
    if (run(a, cfg->type, vec, true, st) != cudaSuccess) return RAWINT4_CUDA_ERROR;
  }
  if (sums) {
    R4_PROF("norm_fold", st);
    norm_fold_kernel<<<dim3((a.width + 255) / 256, 2), 256, 0, st>>>(
        a.partial, bwd_blocks(shape_for(a.width), a.rows), a.width, grad_weight, grad_bias, cfg->weight_type, accumulate);
    if (cudaGetLastError() != cudaSuccess) return RAWINT4_CUDA_ERROR;
  }
  return RAWINT4_OK;
}

}  // extern "C"
