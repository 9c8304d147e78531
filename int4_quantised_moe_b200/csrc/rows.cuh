// Helpers shared by the row kernels around the layer (norm.cu, ckpt8.cu,
// select.cu): element types, vector loads and stores, and the 8-bit
// checkpoint code of a group of 32 values.
//
// Two layouts of a row over T threads:
//   vector   thread t holds chunks t, t + T, ... of kChunk consecutive
//            elements, moved with 16-byte accesses; needs every row to start
//            on a 16-byte boundary and a width that is a multiple of kChunk.
//   scalar   thread t holds elements t, t + T, ...; any width and pitch. A
//            warp reads 32 neighbours at a time, so the accesses stay coalesced.
#pragma once
#include <cuda_fp8.h>
#include <float.h>

#include <initializer_list>

#include "common.cuh"

namespace r4 {

constexpr int kChunk = 8;        // elements of one vector chunk
constexpr int kCkptGroup = 32;   // columns under one scale of an 8-bit checkpoint

template <class T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
  static constexpr float kMax = FLT_MAX;
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ float2 widen(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t narrow(float2 v) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  static constexpr float kMax = 3.3895313892515355e38f;
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ float2 widen(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t narrow(float2 v) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static constexpr float kMax = 65504.f;
};

// Two fp32 operations in one instruction (f32x2), each rounded by itself.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\n"
      "mul.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\n"
      "add.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A chunk in fp32, as the pairs the arithmetic works on.
struct Chunk {
  float2 p[kChunk / 2];
  __device__ __forceinline__ float& operator[](int j) { return j & 1 ? p[j / 2].y : p[j / 2].x; }
  __device__ __forceinline__ float operator[](int j) const { return j & 1 ? p[j / 2].y : p[j / 2].x; }
};
__device__ __forceinline__ Chunk chunk_of(float v) {
  Chunk c;
#pragma unroll
  for (int j = 0; j < kChunk / 2; ++j) c.p[j] = both(v);
  return c;
}

// A chunk as it lies in memory (16 bytes for the 16-bit types, 32 for fp32).
template <class T>
struct alignas(16) RawChunk {
  uint32_t w[kChunk * sizeof(T) / 4];
};

template <class T>
__device__ __forceinline__ RawChunk<T> load_chunk(const T* p) {
  RawChunk<T> r;
  const uint4* s = reinterpret_cast<const uint4*>(p);
  uint4* d = reinterpret_cast<uint4*>(&r);
#pragma unroll
  for (int i = 0; i < (int)sizeof(r) / 16; ++i) d[i] = s[i];
  return r;
}

template <class T>
__device__ __forceinline__ Chunk widen(const RawChunk<T>& r) {
  Chunk c;
#pragma unroll
  for (int j = 0; j < kChunk / 2; ++j) {
    if constexpr (sizeof(T) == 4)
      c.p[j] = make_float2(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
    else
      c.p[j] = Elem<T>::widen(r.w[j]);
  }
  return c;
}

template <class T>
__device__ __forceinline__ RawChunk<T> narrow(const Chunk& c) {
  RawChunk<T> r;
#pragma unroll
  for (int j = 0; j < kChunk / 2; ++j) {
    if constexpr (sizeof(T) == 4) {
      r.w[2 * j] = __float_as_uint(c.p[j].x);
      r.w[2 * j + 1] = __float_as_uint(c.p[j].y);
    } else {
      r.w[j] = Elem<T>::narrow(c.p[j]);
    }
  }
  return r;
}

template <class T>
__device__ __forceinline__ void store_chunk(T* p, const Chunk& c) {
  const RawChunk<T> r = narrow<T>(c);
  const uint4* s = reinterpret_cast<const uint4*>(&r);
  uint4* d = reinterpret_cast<uint4*>(p);
#pragma unroll
  for (int i = 0; i < (int)sizeof(r) / 16; ++i) d[i] = s[i];
}

// ------------------------------------------------------- 8-bit checkpoints
// A group of 32 neighbours shares the scale 2^e, e the smallest exponent
// >= -126 for which its largest finite magnitude fits the code: at most 448
// (E4M3) or below 127.5 (INT8, so that it rounds to at most 127). It is kept
// as the byte e + 127, the exponent field of the fp32 number 2^e. A power of
// two makes x 2^-e exact, so the code is the one rounding of the true value.
// Values that are not finite become the NaN code (E4M3 0x7f, INT8 0x80).
__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
  const uint32_t a = __float_as_uint(v) & 0x7FFFFFFFu;
  return a < 0x7F800000u ? a : 0u;
}

__device__ __forceinline__ uint32_t ckpt_scale_byte(uint32_t amax_bits, int fmt) {
  const int top = fmt == RAWINT4_CKPT_E4M3 ? 8 : 6;
  const uint32_t limit = fmt == RAWINT4_CKPT_E4M3 ? 0x600000u : 0x7EFFFFu;  // mantissa bits of 1.75, just under 1.9921875
  const int over = (amax_bits & 0x7FFFFFu) > limit ? 1 : 0;
  return (uint32_t)max(1, (int)(amax_bits >> 23) - top + over);
}

// 2^-e of a scale byte written by ckpt_scale_byte (1 .. 249)
__device__ __forceinline__ float ckpt_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float ckpt_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ uint32_t ckpt_code(float x, float inv, int fmt) {
  const bool finite = (__float_as_uint(x) & 0x7FFFFFFFu) < 0x7F800000u;
  const float v = x * inv;
  if (fmt == RAWINT4_CKPT_E4M3)
    return finite ? (uint32_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3) : 0x7Fu;
  return finite ? (uint32_t)__float2int_rn(v) & 0xFFu : 0x80u;
}

// Eight codes of finite values (INT8: adding 1.5 2^23 leaves the rounded
// integer in the low mantissa bits).
__device__ __forceinline__ uint2 ckpt_codes8(const Chunk& f, float inv, int fmt) {
  uint32_t w[2];
  if (fmt == RAWINT4_CKPT_E4M3) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 a = mul2(f.p[2 * h], both(inv)), b = mul2(f.p[2 * h + 1], both(inv));
      asm("{\n.reg .b16 lo, hi;\ncvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
          "mov.b32 %0, {lo, hi};\n}"
          : "=r"(w[h])
          : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // an exact product and one rounding
      const float2 a = fma2(f.p[2 * h], both(inv), both(12582912.f)), b = fma2(f.p[2 * h + 1], both(inv), both(12582912.f));
      w[h] = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                         __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
    }
  }
  return make_uint2(w[0], w[1]);
}

// Codes and scale byte of a chunk whose group lies in four neighbouring
// lanes; called by all lanes of a warp (a lane without a chunk passes zeros).
// `amax`: the chunk's largest |x| as fp32 bits, infinities and NaN included.
__device__ __forceinline__ uint2 ckpt_encode8(const Chunk& f, uint32_t amax, int fmt, uint32_t* byte) {
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  if (__any_sync(0xffffffffu, amax >= 0x7F800000u)) {  // rare: leave such values out of the scale, code them as NaN
    amax = 0;
#pragma unroll
    for (int j = 0; j < kChunk; ++j) amax = max(amax, finite_abs_bits(f[j]));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    *byte = ckpt_scale_byte(amax, fmt);
    const float inv = ckpt_inv_scale(*byte);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < kChunk; ++j) w[j / 4] |= ckpt_code(f[j], inv, fmt) << (8 * (j % 4));
    return make_uint2(w[0], w[1]);
  }
  *byte = ckpt_scale_byte(amax, fmt);
  return ckpt_codes8(f, ckpt_inv_scale(*byte), fmt);
}

// The chunk's largest |x| as fp32 bits; 16-bit types compare two at a time.
template <class T>
__device__ __forceinline__ uint32_t abs_max_bits(const RawChunk<T>& r) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kChunk; ++j) m = max(m, r.w[j] & 0x7FFFFFFFu);
    return m;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kChunk / 2; ++j) m = __vmaxu2(m, r.w[j] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    return __float_as_uint(Elem<T>::widen(m).x);
  }
}

// Value of a code; |code| 2^e beyond fp32 gives an infinity.
__device__ __forceinline__ float ckpt_value(uint32_t code, float scale, int fmt) {
  if (fmt == RAWINT4_CKPT_E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
    return __half2float(__half(h)) * scale;
  }
  const float v = (float)(int8_t)code * scale;
  return code == 0x80u ? __uint_as_float(0x7FC00000u) : v;
}

// The group's largest value can round up past the type's largest number:
// finite codes stay finite.
__device__ __forceinline__ float ckpt_saturate(float v, float limit) {
  return fabsf(v) > limit ? copysignf(limit, v) : v;
}

// The largest scale byte under which every finite code stays below `limit`:
// 448 2^e and 127 2^e fit fp16 up to e = 7 and 9, fp32 and bf16 up to 119 and 121.
template <class T>
__device__ __forceinline__ uint32_t ckpt_safe_byte(int fmt) {
  return (sizeof(T) == 2 && Elem<T>::kMax < 1e5f ? 127u + 7u : 127u + 119u) + (fmt == RAWINT4_CKPT_E4M3 ? 0u : 2u);
}

// The numbers that eight codes stand for, without their scale, in fp16 (exact;
// INT8 through 1024 + (code + 128), which fp16 holds in its low bits).
__device__ __forceinline__ RawChunk<__half> ckpt_numbers8(uint2 w, int fmt) {
  RawChunk<__half> r;
  if (fmt == RAWINT4_CKPT_E4M3) {
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(r.w[0]), "=r"(r.w[1])
        : "r"(w.x));
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(r.w[2]), "=r"(r.w[3])
        : "r"(w.y));
  } else {
    const uint32_t u[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t v = __byte_perm(u[q / 2], 0x64006400u, (q & 1) ? 0x7372 : 0x7170);
      const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), __half2half2(__ushort_as_half(0x6480)));  // 1152
      r.w[q] = *reinterpret_cast<const uint32_t*>(&d);
    }
    if (__vcmpeq4(w.x, 0x80808080u) | __vcmpeq4(w.y, 0x80808080u)) {  // rare: NaN codes
#pragma unroll
      for (int j = 0; j < kChunk; ++j)
        if ((u[j / 4] >> (8 * (j % 4)) & 0xFFu) == 0u) r.w[j / 2] |= 0x7FFFu << (16 * (j & 1));
    }
  }
  return r;
}

// Eight values of a checkpoint, saturated for type T.
template <class T>
__device__ __forceinline__ Chunk ckpt_decode8(uint2 w, uint32_t byte, int fmt) {
  Chunk f = widen<__half>(ckpt_numbers8(w, fmt));
  const float2 scale = both(ckpt_scale(byte));
#pragma unroll
  for (int q = 0; q < 4; ++q) f.p[q] = mul2(f.p[q], scale);
  if (byte > ckpt_safe_byte<T>(fmt)) {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) f[j] = ckpt_saturate(f[j], Elem<T>::kMax);
  }
  return f;
}

// Kernels of this kind follow one another in a stream within microseconds, so
// each may be launched while the one before it drains: begin_after_previous()
// stands before a kernel's first access to memory and returns when everything
// before it in the stream is complete and visible; it also lets the next
// kernel's blocks take the places that this one's last blocks leave.
// Such a kernel is resident while the one before it still writes its inputs,
// so none of its pointers is __restrict__ and nothing is read with __ldg: both
// say that the data stays as it is for as long as the kernel lives, and loads
// marked so may be moved in front of the wait.
__device__ __forceinline__ void begin_after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // after the wait: one kernel ahead, no more
}

__device__ __forceinline__ float row_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------- host side
// Launch of a kernel that starts with begin_after_previous().
template <class... P, class... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, int smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

constexpr int64_t kMaxPitch = (int64_t)1 << 28;  // elements of a row pitch

inline size_t type_size(int type) { return type == RAWINT4_TYPE_F32 ? 4 : 2; }
inline bool type_ok(int type) {
  return type == RAWINT4_TYPE_F32 || type == RAWINT4_TYPE_BF16 || type == RAWINT4_TYPE_F16;
}
inline bool ckpt_format_ok(int fmt) { return fmt == RAWINT4_CKPT_E4M3 || fmt == RAWINT4_CKPT_INT8; }
inline int64_t ckpt_groups(int64_t width) { return (width + kCkptGroup - 1) / kCkptGroup; }

// Every row of a [rows, width] tensor with row pitch ld starts on a 16-byte boundary.
inline bool rows_aligned(const void* p, int64_t ld, int type) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)type_size(type) % 16 == 0;
}
// Bytes from the first to the last element of such a tensor.
inline int64_t span_bytes(int64_t rows, int64_t width, int64_t ld, int64_t size) {
  return rows > 0 ? ((rows - 1) * ld + width) * size : 0;
}

// A buffer of a call: its n bytes at p (null: absent) and the alignment of its elements.
struct Span {
  const void* p;
  int64_t n;
  int64_t align;
};

// Every buffer is aligned to its elements, and no output touches an input or another output.
inline bool spans_ok(std::initializer_list<Span> in, std::initializer_list<Span> out) {
  auto aligned = [](const Span& s) { return reinterpret_cast<uintptr_t>(s.p) % s.align == 0; };
  auto apart = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return !a.p || !b.p || a.n <= 0 || b.n <= 0 || x >= y + (uintptr_t)b.n || y >= x + (uintptr_t)a.n;
  };
  for (const Span& s : in)
    if (!aligned(s)) return false;
  for (const Span* o = out.begin(); o != out.end(); ++o) {
    if (!aligned(*o)) return false;
    for (const Span& s : in)
      if (!apart(*o, s)) return false;
    for (const Span* q = out.begin(); q != o; ++q)
      if (!apart(*o, *q)) return false;
  }
  return true;
}

}  // namespace r4
