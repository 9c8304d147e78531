// The norm in front of the layer, forward and backward, layer norm or RMS
// norm. With mu the row mean (0 for RMS), r = 1 / sqrt(mean((x - mu)^2) + eps)
// and xh = (x - mu) r:
//     y  = xh w + b
//     dx = r (w dy - mean(w dy) - xh mean(w dy xh))      (RMS: no middle term)
//     dw = sum over rows of dy xh,  db = sum over rows of dy
// x is a tensor, or the 8-bit checkpoint of one (rows.cuh), decoded on load;
// the forward can write x's checkpoint in the same pass.
//
// Forward: a row lies in the registers of one warp (narrow rows, several rows
// a block) or of one block, so the input is read once: the mean, then the
// centred squares, are summed from registers in fp32. The sum over a row's bf16
// values or a checkpoint's (8 bits each) is exact where they are of one size, and
// so is the mean. With more bits (fp32, fp16) the centred values are summed along
// with their squares, and what their mean lacks of 0 corrects the mean. A row of
// one value has that value for its mean in either case.
//
// xh is formed as (x - mu) r in both directions. x r - mu r would save an
// instruction a pair, but the rounding of mu r stays when x - mu is small: rows of
// the value 5 would get 2e-4 in place of 0.
//
// Backward: a fixed grid of blocks walks the rows. The threads of a row copy
// their own chunks of the coming rows into shared memory (cp.async, a ring of
// a few rows), so no barrier guards the ring and several rows are in flight
// while one is computed. dw and db of a thread's columns stay in its
// registers; each block writes one partial row of sums, and a second kernel
// adds the partials in block order, so the result does not depend on timing.
#pragma once
#include <type_traits>

#include "norm.cuh"

namespace r4 {
namespace {

// Column of this thread's element j of chunk i, in either layout.
template <bool VEC>
__device__ __forceinline__ int column(int i, int j, int t, int threads) {
  return VEC ? (i * threads + t) * kChunk + j : (i * kChunk + j) * threads + t;
}

// The weight or bias of chunk i's columns; `none` where there is no tensor.
template <bool VEC>
__device__ __forceinline__ Chunk load_vector(const void* p, int type, int i, int t, int threads, int width, float none) {
  if (!p) return chunk_of(none);
  if constexpr (VEC) {
    const int c = column<true>(i, 0, t, threads);
    if (c >= width) return chunk_of(0.f);
    if (type == RAWINT4_TYPE_F32) return widen<float>(load_chunk(static_cast<const float*>(p) + c));
    if (type == RAWINT4_TYPE_BF16) return widen<__nv_bfloat16>(load_chunk(static_cast<const __nv_bfloat16*>(p) + c));
    return widen<__half>(load_chunk(static_cast<const __half*>(p) + c));
  } else {
    Chunk v;
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const int c = column<false>(i, j, t, threads);
      v[j] = c < width ? load_as(p, type, c) : 0.f;
    }
    return v;
  }
}

// Chunk i of a row in memory, in the scalar layout; columns past the width read as 0.
template <class T>
__device__ __forceinline__ Chunk any_chunk(const T* row, int i, int t, int threads, int width) {
  Chunk v;
#pragma unroll
  for (int j = 0; j < kChunk; ++j) {
    const int c = column<false>(i, j, t, threads);
    v[j] = c < width ? Elem<T>::to(row[c]) : 0.f;
  }
  return v;
}

// Chunk i of a checkpointed row in the scalar layout.
__device__ __forceinline__ Chunk any_ckpt_chunk(const uint8_t* codes, const uint8_t* scales, int fmt, int i, int t,
                                                int threads, int width) {
  Chunk v;
#pragma unroll
  for (int j = 0; j < kChunk; ++j) {
    const int c = column<false>(i, j, t, threads);
    v[j] = c < width ? ckpt_saturate(ckpt_value(codes[c], ckpt_scale(scales[c / kCkptGroup]), fmt), FLT_MAX) : 0.f;
  }
  return v;
}

template <class T>
__device__ __forceinline__ void store_any_chunk(T* row, int i, int t, int threads, int width, const Chunk& v) {
#pragma unroll
  for (int j = 0; j < kChunk; ++j) {
    const int c = column<false>(i, j, t, threads);
    if (c < width) row[c] = Elem<T>::from(v[j]);
  }
}

// Writes the checkpoint of chunk i. Called by all lanes of a warp.
template <class R, bool VEC>
__device__ __forceinline__ void save_chunk(const RawChunk<R>& raw, uint8_t* codes, uint8_t* scales, int fmt, int i, int t,
                                           int threads, int width) {
  const Chunk v = widen<R>(raw);
  if (VEC) {
    const int c = column<true>(i, 0, t, threads);
    uint32_t byte;
    const uint2 w = ckpt_encode8(v, abs_max_bits<R>(raw), fmt, &byte);
    if (c < width) {
      *reinterpret_cast<uint2*>(codes + c) = w;
      if (c % kCkptGroup == 0) scales[c / kCkptGroup] = (uint8_t)byte;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const int c = column<false>(i, j, t, threads);
      const uint32_t byte = ckpt_scale_byte(__reduce_max_sync(0xffffffffu, finite_abs_bits(v[j])), fmt);
      if (c < width) {
        codes[c] = (uint8_t)ckpt_code(v[j], ckpt_inv_scale(byte), fmt);
        if (c % kCkptGroup == 0) scales[c / kCkptGroup] = (uint8_t)byte;
      }
    }
  }
}

// Sums over the `threads` threads of a row: one warp, or several that meet at
// the named barrier `bar` (each sum has its own `buf`, or the callers alternate
// between two).
__device__ __forceinline__ void row_barrier(int bar, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
}
__device__ __forceinline__ float row_sum(float a, int threads, int bar, float* buf) {
  a = row_warp_sum(a);
  if (threads == 32) return a;
  const int lane = threadIdx.x & 31;
  if (lane == 0) buf[threadIdx.x >> 5] = a;
  row_barrier(bar, threads);
  return row_warp_sum(lane < threads >> 5 ? buf[lane] : 0.f);
}
__device__ __forceinline__ float2 row_sum2(float a, float b, int threads, int bar, float2* buf) {
  a = row_warp_sum(a);
  b = row_warp_sum(b);
  if (threads == 32) return make_float2(a, b);
  const int lane = threadIdx.x & 31;
  if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
  row_barrier(bar, threads);
  const float2 v = lane < threads >> 5 ? buf[lane] : make_float2(0.f, 0.f);
  return make_float2(row_warp_sum(v.x), row_warp_sum(v.y));
}

// CKPT: 0 for a tensor, 1 + its format for a checkpoint (a format decided at
// run time cost the backward 9 of 79 us).

// ------------------------------------------------------------------ forward
// blockDim = (threads of a row, rows): the threads of a row are a warp when
// blockDim.y > 1, else the block. R is how a row waits in registers: in the
// vector layout as it came (16-bit elements, or a checkpoint's numbers in fp16
// with a scale a chunk), else as fp32.
template <class T, class R, int NV, bool VEC, int CKPT>
__global__ void __launch_bounds__(512, VEC ? 2 : 1) norm_fwd_kernel(const NormArgs a) {
  __shared__ float buf[16];
  __shared__ float2 buf2[16];
  constexpr bool kScaled = VEC && CKPT;
  constexpr int kFormat = CKPT - 1;
  constexpr bool kCorrect = !kScaled && !std::is_same<R, __nv_bfloat16>::value;
  begin_after_previous();
  const int t = threadIdx.x, threads = blockDim.x;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;  // whole warps leave; a block-wide row never does
  const int stride = threads * kChunk;  // from a thread's chunk to its next one, in the vector layout
  bool in[NV];
  RawChunk<R> x[NV];
  float scale[kScaled ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    in[i] = column<VEC>(i, 0, t, threads) < a.width;
    if constexpr (kScaled) {
      uint2 codes = make_uint2(0u, 0u);
      scale[i] = 0.f;
      if (in[i]) {
        codes = *reinterpret_cast<const uint2*>(a.in_codes + (int64_t)row * a.width + t * kChunk + i * stride);
        scale[i] = ckpt_scale(a.in_scales[(int64_t)row * a.groups + (t * kChunk + i * stride) / kCkptGroup]);
      }
      x[i].w[0] = codes.x;  // decoded once all loads are on their way
      x[i].w[1] = codes.y;
    } else if constexpr (CKPT) {
      x[i] = RawChunk<R>{};
      if (in[i]) x[i] = narrow<R>(any_ckpt_chunk(a.in_codes + (int64_t)row * a.width, a.in_scales + (int64_t)row * a.groups, kFormat,
                                                 i, t, threads, a.width));
    } else if constexpr (VEC) {
      x[i] = RawChunk<R>{};
      if (in[i]) x[i] = load_chunk(static_cast<const T*>(a.x) + row * a.ldx + t * kChunk + i * stride);
    } else {
      x[i] = RawChunk<R>{};
      if (in[i]) x[i] = narrow<R>(any_chunk(static_cast<const T*>(a.x) + row * a.ldx, i, t, threads, a.width));
    }
  }
  if constexpr (kScaled) {
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = ckpt_numbers8(make_uint2(x[i].w[0], x[i].w[1]), kFormat);
  }
  if (!CKPT && a.codes)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (VEC || __any_sync(0xffffffffu, in[i]))
        save_chunk<R, VEC>(x[i], a.codes + (int64_t)row * a.width, a.scales + (int64_t)row * a.groups, a.fmt, i, t,
                           threads, a.width);

  const float inv_n = 1.0f / (float)a.width;
  float mu = 0.f;
  // x - mu of pair j of chunk i
  auto centred = [&](float2 x, int i) {
    if constexpr (kScaled) return fma2(x, both(scale[i]), both(-mu));
    else return add2(x, both(-mu));
  };
  float2 q = both(0.f);
  float var;
  if (a.layer) {
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Chunk v = widen<R>(x[i]);
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) s = kScaled ? fma2(v.p[j], both(scale[kScaled ? i : 0]), s) : add2(s, v.p[j]);
    }
    const float total = row_sum(s.x + s.y, threads, 1, buf);
    mu = total * inv_n;
    mu = fmaf(fmaf(-mu, (float)a.width, total), inv_n, mu);  // the quotient, to its last bit if it ends there
    s = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      Chunk d = widen<R>(x[i]);
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) d.p[j] = centred(d.p[j], i);
      if (!VEC)
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
          if (column<false>(i, j, t, threads) >= a.width) d[j] = 0.f;
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) {
        if (kCorrect) s = add2(s, d.p[j]);
        q = fma2(d.p[j], d.p[j], q);
      }
    }
    if constexpr (kCorrect) {
      const float2 sums = row_sum2(s.x + s.y, q.x + q.y, threads, 1, buf2);
      const float shift = sums.x * inv_n;
      mu += shift;
      var = fmaxf(sums.y * inv_n - shift * shift, 0.f);
      if (!(sums.y < INFINITY)) var = sums.y;  // infinities and NaN stay what they are
    } else {
      var = row_sum(q.x + q.y, threads, 1, reinterpret_cast<float*>(buf2)) * inv_n;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Chunk v = widen<R>(x[i]);
      float2 s = kScaled ? both(0.f) : q;
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) s = fma2(v.p[j], v.p[j], s);
      q = kScaled ? fma2(mul2(s, both(scale[kScaled ? i : 0])), both(scale[kScaled ? i : 0]), q) : s;
    }
    var = row_sum(q.x + q.y, threads, 1, buf) * inv_n;
  }
  const float r = 1.0f / sqrtf(var + a.eps);
  T* const y = static_cast<T*>(a.y) + (int64_t)row * a.width;
  // y of chunk i, given the weight's and bias's tensor type
  auto finish = [&](auto wt) {
    using W = decltype(wt);
    const W* const w = static_cast<const W*>(a.weight);
    const W* const b = static_cast<const W*>(a.bias);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      Chunk v = widen<R>(x[i]);
      if (a.layer) {
#pragma unroll
        for (int j = 0; j < kChunk / 2; ++j) v.p[j] = mul2(centred(v.p[j], i), both(r));
      } else {
        const float2 rx = both(kScaled ? r * scale[kScaled ? i : 0] : r);
#pragma unroll
        for (int j = 0; j < kChunk / 2; ++j) v.p[j] = mul2(v.p[j], rx);
      }
      if (w) {
        const Chunk f = VEC ? widen<W>(load_chunk(w + t * kChunk + i * stride)) : any_chunk(w, i, t, threads, a.width);
#pragma unroll
        for (int j = 0; j < kChunk / 2; ++j) v.p[j] = mul2(v.p[j], f.p[j]);
      }
      if (b) {
        const Chunk f = VEC ? widen<W>(load_chunk(b + t * kChunk + i * stride)) : any_chunk(b, i, t, threads, a.width);
#pragma unroll
        for (int j = 0; j < kChunk / 2; ++j) v.p[j] = add2(v.p[j], f.p[j]);
      }
      if (VEC) store_chunk(y + t * kChunk + i * stride, v);
      else store_any_chunk(y, i, t, threads, a.width, v);
    }
  };
  if (a.w_type == RAWINT4_TYPE_F32) finish(float());
  else if (a.w_type == RAWINT4_TYPE_BF16) finish(__nv_bfloat16());
  else finish(__half());
  if (t == 0) {
    if (a.mean) a.mean[row] = mu;
    a.rstd[row] = r;
  }
}

// ----------------------------------------------------------------- backward
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Until at most n of this thread's groups are still on their way.
__device__ __forceinline__ void copy_wait_but(int n) {
  if (n >= 3) copy_wait<3>();
  else if (n == 2) copy_wait<2>();
  else if (n == 1) copy_wait<1>();
  else copy_wait<0>();
}

// blockDim = (threads of a row, row groups); each group walks rows on its own
// and meets at its own barrier. VEC: a thread's chunks of x and dy of a row lie
// in its slots of the ring and are read from there twice, for the sums and for
// dx; otherwise they are read from memory (a row ahead into registers where a
// thread has one chunk, else twice, the second time from cache).
// The scale bytes of a checkpoint are fetched one row ahead into registers.
// One block an SM runs, and the bounds say so: left open, four chunks from E4M3
// with db and a mean were compiled for two, at 64 registers and 956 bytes of
// spills a thread (4096 x 12288: 270 us, now 146; RMS of 4096 x 9001: 165, now
// 131). Not so the vector layout's plain RMS, which loses its place for the four
// chunks' numbers by it (8192 x 7168 from E4M3: 69 us, with the bound 85).
template <class T, int NV, bool VEC, int CKPT, bool SUMB, bool LAYER>
__global__ void __launch_bounds__(bwd_threads(NV), VEC && !SUMB && !LAYER ? 0 : 1) norm_bwd_kernel(const NormArgs a) {
  __shared__ float2 buf[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kFormat = CKPT - 1;
  constexpr int kXBytes = CKPT ? kChunk : (int)sizeof(RawChunk<T>);
  const int t = threadIdx.x, threads = blockDim.x, group = threadIdx.y;
  const int warp0 = group * (threads >> 5);  // a group's part of buf
  const int step = gridDim.x * blockDim.y;
  const float inv_n = 1.0f / (float)a.width;
  begin_after_previous();

  // slots of this thread: [stage][chunk][thread], x behind dy
  constexpr int kG = (int)sizeof(RawChunk<T>);
  const int all = threads * blockDim.y;
  uint8_t* const my_g = ring + (group * threads + t) * kG;
  uint8_t* const my_x = ring + a.stages * NV * all * kG + (group * threads + t) * kXBytes;
  // offsets of chunk 0 of the stage at hand; chunks lie all * size apart
  int at_g = 0, at_x = 0;
  const int step_g = all * kG, step_x = all * kXBytes;
  bool in[NV];  // the thread's chunks that the row has
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = column<VEC>(i, 0, t, threads) < a.width;
  // this thread's place in the rows that are fetched next, at hand and written
  const int first = blockIdx.x * blockDim.y + group;
  const T* fetch_g = static_cast<const T*>(a.gy) + first * a.ldg + t * kChunk;
  const T* fetch_x = static_cast<const T*>(a.x) + first * a.ldx + t * kChunk;
  const uint8_t* fetch_codes = a.in_codes + (int64_t)first * a.width + t * kChunk;
  const int64_t hop_g = step * a.ldg, hop_x = step * a.ldx, hop = (int64_t)step * a.width;
  const int stride = threads * kChunk;  // from a thread's chunk to its next one
  int fetch_row = first;
  auto fetch = [&] {
    if (fetch_row < a.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i]) {
          uint8_t* const sg = my_g + at_g + i * step_g;
          uint8_t* const sx = my_x + at_x + i * step_x;
          copy_async16(sg, fetch_g + i * stride);
          if (sizeof(T) == 4) copy_async16(sg + 16, fetch_g + i * stride + 4);
          if (CKPT) {
            copy_async8(sx, fetch_codes + i * stride);
          } else {
            copy_async16(sx, fetch_x + i * stride);
            if (sizeof(T) == 4) copy_async16(sx + 16, fetch_x + i * stride + 4);
          }
        }
    }
    copy_commit();
    fetch_row += step;
    fetch_g += hop_g;
    if (CKPT) fetch_codes += hop;
    else fetch_x += hop_x;
  };
  auto next_stage = [&] {
    at_g += NV * step_g;
    at_x += NV * step_x;
    if (at_g == a.stages * NV * step_g) at_g = at_x = 0;
  };

  Chunk dw[NV], db[SUMB ? NV : 1], w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    dw[i] = chunk_of(0.f);
    if (SUMB) db[i] = chunk_of(0.f);
  }
  if (VEC)
    for (int s = 0; s < a.stages; ++s) {
      fetch();
      next_stage();
    }
#pragma unroll
  for (int i = 0; i < NV; ++i) w[i] = load_vector<VEC>(a.weight, a.w_type, i, t, threads, a.width, 1.f);

  // statistics and scale bytes, fetched a row ahead
  const uint8_t* next_scales = a.in_scales + (int64_t)first * a.groups + t / (kCkptGroup / kChunk);
  const int hop_groups = step * a.groups;
  float next_r = 0.f, next_mu = 0.f;
  uint32_t next_bytes[NV] = {};
  auto fetch_stats = [&](int row) {
    if (row < a.rows) {
      next_r = a.rstd_in[row];
      if (LAYER) next_mu = a.mean_in[row];
      if (CKPT && VEC) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (in[i]) next_bytes[i] = next_scales[i * (stride / kCkptGroup)];
        next_scales += hop_groups;
      }
    }
  };
  fetch_stats(first);
  T* out = static_cast<T*>(a.gx) + (int64_t)first * a.width;

  // the scalar layout with one chunk a thread: the next row's elements, as they come, wait in registers. They are
  // asked for at once, or behind the row's sums where db leaves too few registers (loads on their way would be
  // spilled and waited for: 4096 x 3329 bf16 layer norm with db 41 us, asked for at once 63)
  constexpr bool kKept = !VEC && NV == 1;
  constexpr int kAhead = kKept ? kChunk : 1, kAheadX = kKept && !CKPT ? kChunk : 1, kAheadC = kKept && CKPT ? kChunk : 1;
  T ahead_g[kAhead], ahead_x[kAheadX];
  uint8_t ahead_code[kAheadC], ahead_byte[kAheadC];
  auto fetch_any = [&](int row) {
    if (row >= a.rows) return;
    const T* const g = static_cast<const T*>(a.gy) + row * a.ldg;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = column<false>(0, j, t, threads);
      if (c >= a.width) continue;
      ahead_g[j] = g[c];
      if constexpr (CKPT) {
        ahead_code[kKept ? j : 0] = a.in_codes[(int64_t)row * a.width + c];
        ahead_byte[kKept ? j : 0] = a.in_scales[(int64_t)row * a.groups + c / kCkptGroup];
      } else {
        ahead_x[kKept ? j : 0] = static_cast<const T*>(a.x)[row * a.ldx + c];
      }
    }
  };
  auto take_any = [&](Chunk& xv, Chunk& gv, float mean) {  // x - mean and dy; columns past the width give 0
    xv = gv = chunk_of(0.f);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (column<false>(0, j, t, threads) >= a.width) continue;
      gv[j] = Elem<T>::to(ahead_g[j]);
      if constexpr (CKPT)
        xv[j] = ckpt_saturate(ckpt_value(ahead_code[kKept ? j : 0], ckpt_scale(ahead_byte[kKept ? j : 0]), kFormat), FLT_MAX);
      else
        xv[j] = Elem<T>::to(ahead_x[kKept ? j : 0]);
      if (LAYER) xv[j] -= mean;
    }
  };
  if (kKept) fetch_any(first);

  int turn = 0;
  for (int row = first; row < a.rows; row += step) {
    RawChunk<__half> numbers[CKPT && VEC ? NV : 1];  // a checkpoint's, decoded once; its scale goes into the factor of xh
    Chunk kept_x, kept_g;
    if (kKept) {
      take_any(kept_x, kept_g, next_mu);
      if (!SUMB) fetch_any(row + step);
    }
    // x and dy of a chunk that the row has; in the scalar layout, columns past the width give 0
    auto chunk = [&](int i, Chunk& xv, Chunk& gv) {
      if (VEC) {
        gv = widen<T>(*reinterpret_cast<const RawChunk<T>*>(my_g + at_g + i * step_g));
        if (CKPT) xv = widen<__half>(numbers[CKPT ? i : 0]);
        else xv = widen<T>(*reinterpret_cast<const RawChunk<T>*>(my_x + at_x + i * step_x));
      } else {
        gv = any_chunk(static_cast<const T*>(a.gy) + row * a.ldg, i, t, threads, a.width);
        if (CKPT)
          xv = any_ckpt_chunk(a.in_codes + (int64_t)row * a.width, a.in_scales + (int64_t)row * a.groups, kFormat, i, t,
                              threads, a.width);
        else
          xv = any_chunk(static_cast<const T*>(a.x) + row * a.ldx, i, t, threads, a.width);
      }
    };
    const float r = next_r, mu = next_mu;
    uint32_t bytes[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) bytes[i] = next_bytes[i];
    fetch_stats(row + step);
    if (VEC) copy_wait_but(a.stages - 1);

    // in the scalar layout not as pairs, which want their factors twice in neighbouring registers
    auto mul = [](float2 a, float2 b) {
      if constexpr (VEC) return mul2(a, b);
      else return make_float2(a.x * b.x, a.y * b.y);
    };
    auto add = [](float2 a, float2 b) {
      if constexpr (VEC) return add2(a, b);
      else return make_float2(a.x + b.x, a.y + b.y);
    };
    auto fma = [](float2 a, float2 b, float2 c) {
      if constexpr (VEC) return fma2(a, b, c);
      else return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
    };
    float2 s1 = both(0.f), s2 = both(0.f);
    constexpr bool kLate = LAYER || !(CKPT && VEC);
    const float2 r2 = both(r), minus_mu = both(-mu);
    // factor(i) times off_mean(x, i) is xh
    auto off_mean = [&](float2 x, int i) {
      if (!LAYER || kKept) return x;
      return CKPT && VEC ? fma(x, both(ckpt_scale(bytes[i])), minus_mu) : add(x, minus_mu);
    };
    auto factor = [&](int i) { return CKPT && VEC && !LAYER ? both(r * ckpt_scale(bytes[i])) : r2; };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      Chunk xv, gv;
      if (CKPT && VEC) numbers[CKPT && VEC ? i : 0] = ckpt_numbers8(*reinterpret_cast<const uint2*>(my_x + at_x + i * step_x), kFormat);
      if (kKept) {
        xv = kept_x;
        gv = kept_g;
      } else {
        chunk(i, xv, gv);
      }
      const float2 rx = factor(i);
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) {
        if (kLate) {  // dy (x - mu): r comes in with dw's sum and, for the row, behind its sum
          const float2 gx = mul(gv.p[j], off_mean(xv.p[j], i));
          dw[i].p[j] = fma(gx, r2, dw[i].p[j]);
          s2 = fma(gx, w[i].p[j], s2);
        } else {  // a checkpoint's scales differ within the row: dy xh
          const float2 gx = mul(gv.p[j], mul(xv.p[j], rx));
          dw[i].p[j] = add(dw[i].p[j], gx);
          s2 = fma(gx, w[i].p[j], s2);
        }
        if (SUMB) db[i].p[j] = add(db[i].p[j], gv.p[j]);
        if (LAYER) s1 = fma(gv.p[j], w[i].p[j], s1);
      }
    }
    float2 s;
    if (LAYER) s = row_sum2(s1.x + s1.y, s2.x + s2.y, threads, 1 + group, buf[turn] + warp0);
    else s = make_float2(0.f, row_sum(s2.x + s2.y, threads, 1 + group, reinterpret_cast<float*>(buf[turn] + warp0)));
    if (kKept && SUMB) fetch_any(row + step);
    // dx = r w dy + xh c1 + c0, from dx = r (w dy - m1 - xh m2)
    if (kLate) s.y *= r;
    const float c1 = -r * (s.y * inv_n);
    const float2 c0 = both(-r * (s.x * inv_n));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      Chunk xv, gv;
      if (kKept) {
        xv = kept_x;
        gv = kept_g;
      } else {
        chunk(i, xv, gv);
      }
      const float2 cx = both(factor(i).x * c1);
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j)
        xv.p[j] = fma(mul(gv.p[j], w[i].p[j]), r2, LAYER ? fma(off_mean(xv.p[j], i), cx, c0) : mul(xv.p[j], cx));
      if (VEC) store_chunk(out + t * kChunk + i * stride, xv);
      else store_any_chunk(out, i, t, threads, a.width, xv);
    }
    out += hop;
    if (VEC) {
      fetch();
      next_stage();
    }
    turn ^= 1;
  }
  if (VEC) copy_wait<0>();  // nothing but empty groups is left
  if (!a.want_w && !a.want_b) return;

  // the sums of the block's groups side by side in shared memory (the rings are done with), added in order
  float* const fold = reinterpret_cast<float*>(ring);
  __syncthreads();
  auto put = [&](float* row, int i, const Chunk& v) {
    if (VEC) {
      if (in[i]) store_chunk(row + column<true>(i, 0, t, threads), v);
    } else {
      store_any_chunk(row, i, t, threads, a.width, v);
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    put(fold + group * a.width, i, dw[i]);
    if (SUMB) put(fold + (blockDim.y + group) * a.width, i, db[SUMB ? i : 0]);
  }
  __syncthreads();
  for (int c = group * threads + t; c < a.width; c += all) {
    for (int pass = 0; pass < (SUMB ? 2 : 1); ++pass) {
      float s = 0.f;
      for (int y = 0; y < (int)blockDim.y; ++y) s += fold[(pass * blockDim.y + y) * a.width + c];
      a.partial[((int64_t)pass * gridDim.x + blockIdx.x) * a.width + c] = s;
    }
  }
}

// ------------------------------------------------------------- launch shapes
// Forward: eight chunks of a 16-bit row a thread keep a block's warps, and the
// time they wait for one another, few (8192 x 7168 bf16 RMS: 38 us, with four
// 45); with a mean (layer norm with bias: 65 us, with four 52) or a checkpoint's
// numbers eight do not fit the registers, so four (4096 x 2816 from INT8: 11.3 us,
// with two 13.0). Few rows want many threads each (1 x 7168: eight chunks 3.8 us,
// four 2.9, two 2.4).
Shape fwd_shape(const NormArgs& a, int type) {
  if (!a.vec) {
    // scalar layout: two chunks a thread (8192 x 2817 bf16 RMS: one 44 us, two 33, four 37; 4096 x 8191: two 60, four
    // 63), one where rows are few (400 x 2817: one 3.5 us, two 3.9); a block has at most 512 threads
    int most = a.rows <= kFewRows ? 1 : 2;
    while (a.width > most * kChunk * 512) most *= 2;
    return shape_for(a.width, most, a.rows <= kFewRows ? 1 : kFwdWarps);
  }
  int most = !a.in_codes && type != RAWINT4_TYPE_F32 && !a.layer ? 8 : 4;
  if (a.rows <= kFewRows && a.width <= 2 * kChunk * 512) most = 2;
  return shape_for(a.width, most, a.rows <= kFewRows ? 1 : kFwdWarps);
}

// Bytes of one stage of a block's rings.
int stage_bytes(const Shape& s, int type, bool ckpt) {
  const int chunk = kChunk * (int)type_size(type);
  return s.nv * s.threads * s.rows * (chunk + (ckpt ? kChunk : chunk));
}

template <class T, int NV, bool VEC, int CKPT, bool SUMB, bool LAYER>
cudaError_t launch_bwd(NormArgs a, int type, cudaStream_t st) {
  const Shape s = bwd_shape(a);
  const int stage = stage_bytes(s, type, CKPT);
  a.stages = VEC ? kBwdRing / stage : 1;
  if (a.stages > kBwdMaxStages) a.stages = kBwdMaxStages;
  const int sums = (SUMB ? 2 : 1) * s.rows * a.width * (int)sizeof(float);
  int smem = VEC ? a.stages * stage : 0;
  if (smem < sums) smem = sums;
  static std::atomic<unsigned long long> opted{0};
  int dev = 0;
  if (!device_flag_test(opted, &dev)) {
    const cudaError_t err = cudaFuncSetAttribute(norm_bwd_kernel<T, NV, VEC, CKPT, SUMB, LAYER>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdRing);
    if (err != cudaSuccess) return err;
    device_flag_set(opted, dev);
  }
  return launch_early(norm_bwd_kernel<T, NV, VEC, CKPT, SUMB, LAYER>, bwd_blocks(s, a.rows), dim3(s.threads, s.rows), smem, st, a);
}

template <class T, class R, int NV, bool VEC, int CKPT>
cudaError_t launch_fwd(const NormArgs& a, const Shape& s, cudaStream_t st) {
  return launch_early(norm_fwd_kernel<T, R, NV, VEC, CKPT>, ceil_div(a.rows, s.rows), dim3(s.threads, s.rows), 0, st, a);
}

template <class T, int NV, int CKPT>
cudaError_t pick_ckpt_fwd(const NormArgs& a, const Shape& s, bool vec, cudaStream_t st) {
  return vec ? launch_fwd<T, __half, NV, true, CKPT>(a, s, st) : launch_fwd<T, float, NV, false, CKPT>(a, s, st);
}

template <class T, int NV>
cudaError_t pick_fwd(const NormArgs& a, const Shape& s, bool vec, cudaStream_t st) {
  if (a.in_codes)
    return a.in_fmt == RAWINT4_CKPT_E4M3 ? pick_ckpt_fwd<T, NV, 1 + RAWINT4_CKPT_E4M3>(a, s, vec, st)
                                         : pick_ckpt_fwd<T, NV, 1 + RAWINT4_CKPT_INT8>(a, s, vec, st);
  return vec ? launch_fwd<T, T, NV, true, 0>(a, s, st) : launch_fwd<T, float, NV, false, 0>(a, s, st);
}

template <class T>
cudaError_t fwd_type(const NormArgs& a, int type, cudaStream_t st) {
  const Shape s = fwd_shape(a, type);
  const bool vec = a.vec;
  if constexpr (sizeof(T) == 2)
    if (s.nv == 8) return launch_fwd<T, T, 8, true, 0>(a, s, st);
  if (s.nv == 1) return pick_fwd<T, 1>(a, s, vec, st);
  if (s.nv == 2) return pick_fwd<T, 2>(a, s, vec, st);
  return pick_fwd<T, 4>(a, s, vec, st);
}

template <class T, int NV, bool VEC, int CKPT>
cudaError_t pick_sums(const NormArgs& a, int type, cudaStream_t st) {
  if (a.layer)
    return a.want_b ? launch_bwd<T, NV, VEC, CKPT, true, true>(a, type, st)
                    : launch_bwd<T, NV, VEC, CKPT, false, true>(a, type, st);
  return a.want_b ? launch_bwd<T, NV, VEC, CKPT, true, false>(a, type, st)
                  : launch_bwd<T, NV, VEC, CKPT, false, false>(a, type, st);
}

template <class T, int NV, bool VEC>
cudaError_t pick_source(const NormArgs& a, int type, cudaStream_t st) {
  if (!a.in_codes) return pick_sums<T, NV, VEC, 0>(a, type, st);
  return a.in_fmt == RAWINT4_CKPT_E4M3 ? pick_sums<T, NV, VEC, 1 + RAWINT4_CKPT_E4M3>(a, type, st)
                                       : pick_sums<T, NV, VEC, 1 + RAWINT4_CKPT_INT8>(a, type, st);
}

template <class T, int NV>
cudaError_t pick_bwd(const NormArgs& a, int type, bool vec, cudaStream_t st) {
  return vec ? pick_source<T, NV, true>(a, type, st) : pick_source<T, NV, false>(a, type, st);
}

template <class T>
cudaError_t bwd_type(const NormArgs& a, int type, cudaStream_t st) {
  const bool vec = a.vec;
  const int nv = bwd_shape(a).nv;
  if (nv == 1) return pick_bwd<T, 1>(a, type, vec, st);
  if (nv == 2) return pick_bwd<T, 2>(a, type, vec, st);
  return pick_bwd<T, 4>(a, type, vec, st);
}

}  // namespace
}  // namespace r4
