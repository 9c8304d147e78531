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
constexpr int kUnroll = 4;  // chunks a thread holds at once: 64 bytes of loads in flight

// Where chunk i of a tensor lies. Chunks are counted over rows padded to
// whole groups, so that the four lanes of a group never straddle rows; a
// dense tensor of whole groups is one long row (cpr = 0) and needs no division.
struct Place {
  int64_t x, code, scale;  // element of x, code, scale byte
  bool mine;
};
__device__ __forceinline__ Place place(int64_t i, uint32_t cpr, int width, int64_t ldx, int groups) {
  if (cpr == 0) return {i * kChunk, i * kChunk, i / 4, true};
  const uint32_t row = (uint32_t)i / cpr, c = (uint32_t)i - row * cpr;
  return {row * ldx + c * kChunk, (int64_t)row * width + c * kChunk, (int64_t)row * groups + c / 4,
          (int)(c * kChunk) < width};
}

// Vector layout.
template <class T, int FMT>
__global__ void __launch_bounds__(kThreads) ckpt8_save_vec(const T* x, int64_t ldx, int64_t n, int width,
                                                           uint32_t cpr, uint8_t* codes,
                                                           uint8_t* scales, int groups) {
  begin_after_previous();
  const int64_t i0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  RawChunk<T> r[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = i0 + u * kThreads;
    r[u] = RawChunk<T>{};
    if (i < n) {
      const Place p = place(i, cpr, width, ldx, groups);
      if (p.mine) r[u] = load_chunk(x + p.x);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = i0 + u * kThreads;
    uint32_t byte;
    const uint2 w = ckpt_encode8(widen<T>(r[u]), abs_max_bits<T>(r[u]), FMT, &byte);
    if (i < n) {
      const Place p = place(i, cpr, width, ldx, groups);
      if (p.mine) {
        *reinterpret_cast<uint2*>(codes + p.code) = w;
        if (threadIdx.x % 4 == 0) scales[p.scale] = (uint8_t)byte;
      }
    }
  }
}

// Scalar layout: a warp takes a segment of a row, up to kAnyUnroll groups that
// lie at constant distances; n segments, `segments` a row.
constexpr int kAnyUnroll = 8;

template <class T, int FMT>
__global__ void __launch_bounds__(kThreads) ckpt8_save_any(const T* x, int64_t ldx, int64_t n, int width,
                                                           uint8_t* codes, uint8_t* scales,
                                                           uint32_t segments, int groups) {
  begin_after_previous();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (i >= n) return;
  const uint32_t row = (uint32_t)i / segments;
  const int g0 = (int)((uint32_t)i - row * segments) * kAnyUnroll;
  const int col = g0 * kCkptGroup + lane;
  x += row * ldx + col;
  codes += (int64_t)row * width + col;
  const int left = width - col;  // columns from the lane's first one on
  float f[kAnyUnroll];
#pragma unroll
  for (int u = 0; u < kAnyUnroll; ++u) f[u] = u * kCkptGroup < left ? Elem<T>::to(x[u * kCkptGroup]) : 0.f;
  uint32_t mine = 0;  // lane u: the scale byte of group u
#pragma unroll
  for (int u = 0; u < kAnyUnroll; ++u) {
    if (g0 + u >= groups) break;
    const uint32_t byte = ckpt_scale_byte(__reduce_max_sync(0xffffffffu, finite_abs_bits(f[u])), FMT);
    if (u * kCkptGroup < left) codes[u * kCkptGroup] = (uint8_t)ckpt_code(f[u], ckpt_inv_scale(byte), FMT);
    if (lane == u) mine = byte;
  }
  if (lane < kAnyUnroll && g0 + lane < groups) scales[(int64_t)row * groups + g0 + lane] = (uint8_t)mine;
}

template <class T, int FMT>
__global__ void __launch_bounds__(kThreads) ckpt8_load_vec(const uint8_t* codes,
                                                           const uint8_t* scales, int64_t n, int width,
                                                           uint32_t cpr, int groups, T* out) {
  begin_after_previous();
  const int64_t i0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  uint2 w[kUnroll];
  uint32_t byte[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = i0 + u * kThreads;
    w[u] = make_uint2(0u, 0u);
    byte[u] = 1u;
    if (i < n) {
      const Place p = place(i, cpr, width, width, groups);
      if (p.mine) {
        w[u] = *reinterpret_cast<const uint2*>(codes + p.code);
        byte[u] = scales[p.scale];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = i0 + u * kThreads;
    const Chunk f = ckpt_decode8<T>(w[u], byte[u], FMT);
    if (i < n) {
      const Place p = place(i, cpr, width, width, groups);
      if (p.mine) store_chunk(out + p.x, f);
    }
  }
}

template <class T, int FMT>
__global__ void __launch_bounds__(kThreads) ckpt8_load_any(const uint8_t* codes,
                                                           const uint8_t* scales, int64_t n, int width,
                                                           uint32_t segments, int groups, T* out) {
  begin_after_previous();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (i >= n) return;
  const uint32_t row = (uint32_t)i / segments;
  const int g0 = (int)((uint32_t)i - row * segments) * kAnyUnroll;
  const int col = g0 * kCkptGroup + lane;
  codes += (int64_t)row * width + col;
  out += (int64_t)row * width + col;
  const int left = width - col;
  const uint32_t mine = lane < kAnyUnroll && g0 + lane < groups ? scales[(int64_t)row * groups + g0 + lane] : 1u;
  uint32_t code[kAnyUnroll];
#pragma unroll
  for (int u = 0; u < kAnyUnroll; ++u) code[u] = u * kCkptGroup < left ? codes[u * kCkptGroup] : 0u;
#pragma unroll
  for (int u = 0; u < kAnyUnroll; ++u) {
    if (g0 + u >= groups) break;
    const uint32_t byte = __shfl_sync(0xffffffffu, mine, u);
    float v = ckpt_value(code[u], ckpt_scale(byte), FMT);
    if (byte > ckpt_safe_byte<T>(FMT)) v = ckpt_saturate(v, Elem<T>::kMax);
    if (u * kCkptGroup < left) out[u * kCkptGroup] = Elem<T>::from(v);
  }
}

// Calls run(first row, units, blocks) for slices of at most 2^31 units (the
// kernels' unit-to-row division is 32 bits wide), `per_row` units a row and
// `per_block` a block.
template <class F>
cudaError_t slices(int64_t rows, int64_t per_row, int64_t per_block, F run) {
  const int64_t step = ((int64_t)1 << 31) / per_row;
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t n = (rows - r < step ? rows - r : step) * per_row;
    const cudaError_t err = run(r, n, (unsigned)((n + per_block - 1) / per_block));
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

constexpr int kGroupChunks = kCkptGroup / kChunk;
constexpr int kVecUnits = kThreads * kUnroll;       // chunks of a block
constexpr int kAnyUnits = kThreads / 32;        // segments of a block

int segments_of(int groups) { return (groups + kAnyUnroll - 1) / kAnyUnroll; }

uint32_t chunks_per_row(int width, int64_t ld) {
  return ld == width && width % kCkptGroup == 0 ? 0u : (uint32_t)ckpt_groups(width) * kGroupChunks;
}

template <class T, int FMT>
cudaError_t save(int type, const void* x, int64_t ldx, int64_t rows, int width, uint8_t* codes, uint8_t* scales,
                 cudaStream_t st) {
  const int groups = (int)ckpt_groups(width);
  const T* p = static_cast<const T*>(x);
  if (width % kChunk == 0 && rows_aligned(x, ldx, type) && reinterpret_cast<uintptr_t>(codes) % 8 == 0)
    return slices(rows, groups * kGroupChunks, kVecUnits, [&](int64_t r, int64_t n, unsigned blocks) {
      return launch_early(ckpt8_save_vec<T, FMT>, blocks, kThreads, 0, st, p + r * ldx, ldx, n, width, chunks_per_row(width, ldx),
                                                          codes + r * width, scales + r * groups, groups);
    });
  return slices(rows, segments_of(groups), kAnyUnits, [&](int64_t r, int64_t n, unsigned blocks) {
    return launch_early(ckpt8_save_any<T, FMT>, blocks, kThreads, 0, st, p + r * ldx, ldx, n, width, codes + r * width,
                        scales + r * groups, (uint32_t)segments_of(groups), groups);
  });
}

template <class T, int FMT>
cudaError_t load(int type, const uint8_t* codes, const uint8_t* scales, int64_t rows, int width, void* out,
                 cudaStream_t st) {
  const int groups = (int)ckpt_groups(width);
  T* p = static_cast<T*>(out);
  if (width % kChunk == 0 && rows_aligned(out, width, type) && reinterpret_cast<uintptr_t>(codes) % 8 == 0)
    return slices(rows, groups * kGroupChunks, kVecUnits, [&](int64_t r, int64_t n, unsigned blocks) {
      return launch_early(ckpt8_load_vec<T, FMT>, blocks, kThreads, 0, st, codes + r * width, scales + r * groups, n, width,
                                                          chunks_per_row(width, width), groups, p + r * width);
    });
  return slices(rows, segments_of(groups), kAnyUnits, [&](int64_t r, int64_t n, unsigned blocks) {
    return launch_early(ckpt8_load_any<T, FMT>, blocks, kThreads, 0, st, codes + r * width, scales + r * groups, n, width,
                        (uint32_t)segments_of(groups), groups, p + r * width);
  });
}

template <class T>
cudaError_t save_fmt(int fmt, int type, const void* x, int64_t ldx, int64_t rows, int width, uint8_t* codes,
                     uint8_t* scales, cudaStream_t st) {
  return fmt == RAWINT4_CKPT_E4M3 ? save<T, RAWINT4_CKPT_E4M3>(type, x, ldx, rows, width, codes, scales, st)
                                  : save<T, RAWINT4_CKPT_INT8>(type, x, ldx, rows, width, codes, scales, st);
}

template <class T>
cudaError_t load_fmt(int fmt, int type, const uint8_t* codes, const uint8_t* scales, int64_t rows, int width, void* out,
                     cudaStream_t st) {
  return fmt == RAWINT4_CKPT_E4M3 ? load<T, RAWINT4_CKPT_E4M3>(type, codes, scales, rows, width, out, st)
                                  : load<T, RAWINT4_CKPT_INT8>(type, codes, scales, rows, width, out, st);
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
  if (type == RAWINT4_TYPE_F32) err = save_fmt<float>(format, type, x, ldx, rows, width, codes, scales, st);
  else if (type == RAWINT4_TYPE_BF16) err = save_fmt<__nv_bfloat16>(format, type, x, ldx, rows, width, codes, scales, st);
  else err = save_fmt<__half>(format, type, x, ldx, rows, width, codes, scales, st);
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
  if (type == RAWINT4_TYPE_F32) err = load_fmt<float>(format, type, codes, scales, rows, width, out, st);
  else if (type == RAWINT4_TYPE_BF16) err = load_fmt<__nv_bfloat16>(format, type, codes, scales, rows, width, out, st);
  else err = load_fmt<__half>(format, type, codes, scales, rows, width, out, st);
  return err == cudaSuccess ? RAWINT4_OK : RAWINT4_CUDA_ERROR;
}

}  // extern "C"
