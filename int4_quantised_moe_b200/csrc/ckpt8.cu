// Activation checkpoints in 8 bits: rows [rows, width] of fp32, bf16 or fp16
// kept as one code per element and one power-of-two scale per 32 neighbours
// of a row (format: rows.cuh), and read back.
//
// Both directions are one pass: 32 neighbours sit in four lanes (vector
// layout) or in one warp (scalar layout), so a group's largest magnitude
// needs shuffles only and every byte moves once.
#include "prof.cuh"
#include "rows.cuh"

namespace r4 {
namespace {

constexpr int kThreads = 256;

// Vector layout: `cpr` chunks a row, padded to a multiple of four so that the
// four lanes of a group never straddle rows.
template <class T>
__global__ void __launch_bounds__(kThreads) ckpt8_save_vec(const T* __restrict__ x, int64_t ldx, int64_t rows, int width,
                                                           int cpr, int fmt, uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales, int groups) {
  const int64_t n = rows * cpr;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  // every lane of a warp runs the same number of turns: n is a multiple of four and
  // the lanes past it take part in the shuffles with zeros
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads; i0 < n; i0 += stride) {
    const int64_t i = i0 + threadIdx.x;
    const int64_t row = i / cpr;
    const int c = (int)(i - row * cpr);
    const bool mine = i < n && c * kChunk < width;
    float f[kChunk];
    uint32_t amax = 0;
    if (mine) {
      const RawChunk<T> r = load_chunk(x + row * ldx + c * kChunk);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        f[j] = Elem<T>::to(r.v[j]);
        amax = max(amax, finite_abs_bits(f[j]));
      }
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    if (mine) {
      const uint32_t byte = ckpt_scale_byte(amax, fmt);
      const float inv = ckpt_inv_scale(byte);
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < kChunk; ++j) w[j / 4] |= ckpt_code(f[j], inv, fmt) << (8 * (j % 4));
      *reinterpret_cast<uint2*>(codes + row * width + c * kChunk) = make_uint2(w[0], w[1]);
      if (c % 4 == 0) scales[row * groups + c / 4] = (uint8_t)byte;
    }
  }
}

// Scalar layout: one warp per group.
template <class T>
__global__ void __launch_bounds__(kThreads) ckpt8_save_any(const T* __restrict__ x, int64_t ldx, int64_t rows, int width,
                                                           int fmt, uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales, int groups) {
  const int lane = threadIdx.x & 31;
  const int64_t n = rows * groups;
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n;
       i += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t row = i / groups;
    const int g = (int)(i - row * groups);
    const int col = g * kCkptGroup + lane;
    const bool mine = col < width;
    const float f = mine ? Elem<T>::to(x[row * ldx + col]) : 0.f;
    const uint32_t byte = ckpt_scale_byte(__reduce_max_sync(0xffffffffu, finite_abs_bits(f)), fmt);
    if (mine) codes[row * width + col] = (uint8_t)ckpt_code(f, ckpt_inv_scale(byte), fmt);
    if (lane == 0) scales[i] = (uint8_t)byte;
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) ckpt8_load_vec(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t rows, int width,
                                                           int groups, int fmt, T* __restrict__ out) {
  const int cpr = width / kChunk;
  const int64_t n = rows * cpr;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / cpr;
    const int c = (int)(i - row * cpr);
    const uint2 w = *reinterpret_cast<const uint2*>(codes + i * kChunk);
    const float scale = ckpt_scale(scales[row * groups + c / 4]);
    float f[kChunk];
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
      f[j] = ckpt_saturate(ckpt_value(((j < 4 ? w.x : w.y) >> (8 * (j % 4))) & 0xFFu, scale, fmt), Elem<T>::kMax);
    store_chunk(out + i * kChunk, f);
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) ckpt8_load_any(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t rows, int width,
                                                           int groups, int fmt, T* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const int64_t n = rows * groups;
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n;
       i += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t row = i / groups;
    const int col = (int)(i - row * groups) * kCkptGroup + lane;
    if (col < width) {
      const float v = ckpt_value(codes[row * width + col], ckpt_scale(scales[i]), fmt);
      out[row * width + col] = Elem<T>::from(ckpt_saturate(v, Elem<T>::kMax));
    }
  }
}

int blocks_for(int64_t units, int per_block, int sms) {
  const int64_t need = (units + per_block - 1) / per_block;
  const int64_t most = (int64_t)sms * 16;
  return (int)(need < most ? need : most);
}

template <class T>
cudaError_t save(int fmt, int type, const void* x, int64_t ldx, int64_t rows, int width, uint8_t* codes, uint8_t* scales,
                 int sms, cudaStream_t st) {
  const int groups = (int)ckpt_groups(width);
  const T* p = static_cast<const T*>(x);
  if (width % kChunk == 0 && rows_aligned(x, ldx, type) && reinterpret_cast<uintptr_t>(codes) % 8 == 0) {
    const int cpr = groups * (kCkptGroup / kChunk);
    ckpt8_save_vec<T><<<blocks_for(rows * cpr, kThreads, sms), kThreads, 0, st>>>(p, ldx, rows, width, cpr, fmt, codes,
                                                                                  scales, groups);
  } else {
    ckpt8_save_any<T><<<blocks_for(rows * groups, kThreads / 32, sms), kThreads, 0, st>>>(p, ldx, rows, width, fmt, codes,
                                                                                          scales, groups);
  }
  return cudaGetLastError();
}

template <class T>
cudaError_t load(int fmt, int type, const uint8_t* codes, const uint8_t* scales, int64_t rows, int width, void* out,
                 int sms, cudaStream_t st) {
  const int groups = (int)ckpt_groups(width);
  T* p = static_cast<T*>(out);
  if (width % kChunk == 0 && rows_aligned(out, width, type) && reinterpret_cast<uintptr_t>(codes) % 8 == 0) {
    ckpt8_load_vec<T><<<blocks_for(rows * (width / kChunk), kThreads, sms), kThreads, 0, st>>>(codes, scales, rows, width,
                                                                                               groups, fmt, p);
  } else {
    ckpt8_load_any<T><<<blocks_for(rows * groups, kThreads / 32, sms), kThreads, 0, st>>>(codes, scales, rows, width,
                                                                                          groups, fmt, p);
  }
  return cudaGetLastError();
}

bool sizes_ok(int fmt, int type, int64_t rows, int width, int64_t ld) {
  return ckpt_format_ok(fmt) && type_ok(type) && rows >= 0 && rows < (int64_t)1 << 31 && width >= 1 && width <= 1 << 20 &&
         ld >= width && ld <= kMaxPitch;
}

}  // namespace
}  // namespace r4

using namespace r4;

extern "C" {

RAWINT4_API int rawint4_ckpt8_save(int32_t format, int32_t type, const void* x, int64_t ldx, int64_t rows, int32_t width,
                                   uint8_t* codes, uint8_t* scales, void* stream_) {
  if (!sizes_ok(format, type, rows, width, ldx)) return RAWINT4_INVALID_ARGUMENT;
  if (rows == 0) return RAWINT4_OK;
  const int64_t size = (int64_t)type_size(type);
  if (!x || !codes || !scales ||
      !spans_ok({{x, span_bytes(rows, width, ldx, size), size}},
                {{codes, rows * width, 1}, {scales, rows * ckpt_groups(width), 1}}))
    return RAWINT4_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != RAWINT4_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream_);
  R4_PROF("ckpt8_save", st);
  cudaError_t err;
  if (type == RAWINT4_TYPE_F32) err = save<float>(format, type, x, ldx, rows, width, codes, scales, sms, st);
  else if (type == RAWINT4_TYPE_BF16) err = save<__nv_bfloat16>(format, type, x, ldx, rows, width, codes, scales, sms, st);
  else err = save<__half>(format, type, x, ldx, rows, width, codes, scales, sms, st);
  return err == cudaSuccess ? RAWINT4_OK : RAWINT4_CUDA_ERROR;
}

RAWINT4_API int rawint4_ckpt8_load(int32_t format, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                   int32_t width, int32_t type, void* out, void* stream_) {
  if (!sizes_ok(format, type, rows, width, width)) return RAWINT4_INVALID_ARGUMENT;
  if (rows == 0) return RAWINT4_OK;
  const int64_t size = (int64_t)type_size(type);
  if (!out || !codes || !scales ||
      !spans_ok({{codes, rows * width, 1}, {scales, rows * ckpt_groups(width), 1}}, {{out, rows * width * size, size}}))
    return RAWINT4_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != RAWINT4_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream_);
  R4_PROF("ckpt8_load", st);
  cudaError_t err;
  if (type == RAWINT4_TYPE_F32) err = load<float>(format, type, codes, scales, rows, width, out, sms, st);
  else if (type == RAWINT4_TYPE_BF16) err = load<__nv_bfloat16>(format, type, codes, scales, rows, width, out, sms, st);
  else err = load<__half>(format, type, codes, scales, rows, width, out, sms, st);
  return err == cudaSuccess ? RAWINT4_OK : RAWINT4_CUDA_ERROR;
}

}  // extern "C"
