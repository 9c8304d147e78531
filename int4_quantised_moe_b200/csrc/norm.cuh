#pragma once
#include "rows.cuh"

namespace r4 {

constexpr int kMaxWidth = 16384;
constexpr int kFewRows = 296;        // two rows an SM
constexpr int kFwdWarps = 8;         // rows of a forward block when a row lies in one warp
// Threads of a backward block at most: 128, 96 and 72 registers a thread. w, dw
// and db take 8 a chunk each. Spills in bytes a thread, vector layout: none to 24
// without db; with it none at one chunk, up to 48 at two, 12 to 84 at four from a
// tensor and 156 to 300 from a checkpoint. Scalar layout, whose next row waits in
// registers too: none to 88 without db, up to 108, 60 and 240 with it.
__host__ __device__ constexpr int bwd_threads(int nv) { return nv == 4 ? 512 : nv == 2 ? 640 : 896; }
constexpr int kBwdBlocks = 148;      // blocks of the backward at most, one an SM: rows of partial sums
constexpr int kBwdMaxStages = 4;     // rows in a thread group's ring
constexpr int kBwdRing = 200 * 1024; // bytes of shared memory for the rings

struct NormArgs {
  const void* x;            // elements of type T, or
  const uint8_t* in_codes;  // an 8-bit checkpoint
  const uint8_t* in_scales;
  int64_t ldx;
  int in_fmt;
  int rows, width, groups;
  int vec;                  // every row, weight and bias may move with vector accesses
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
  int stages;
};

__device__ __forceinline__ float load_as(const void* p, int type, int64_t i) {
  if (type == RAWINT4_TYPE_F32) return static_cast<const float*>(p)[i];
  if (type == RAWINT4_TYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

struct Shape {
  int nv, threads, rows;  // chunks a thread, threads a row, rows (row groups) a block
};

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The smallest of `most`, most / 2, ... chunks a thread that a row of one warp
// needs, else `most` and as many warps as that takes.
inline Shape shape_for(int width, int most, int warps_rows) {
  const int chunks = ceil_div(width, kChunk);
  for (int nv = 1; nv <= most && nv <= 4; nv *= 2)
    if (chunks <= 32 * nv) return {nv, 32, warps_rows};
  return {most, ceil_div(chunks, most * 32) * 32, 1};
}

// Backward: four chunks a thread, fewer where db needs registers too: two, or
// one next to a checkpoint's numbers, if the row's threads then fit a block
// (with the fold, 8192 x 7168 bf16 RMS: four 61 us, two 70; 4095 x 704 fp32 with
// db: two 13.3 us, one 14.2; 4096 x 2816 bf16 with db: four 26 us, two 21, from
// INT8: four 36, two 26, one 24). The scalar layout takes one, the next row's
// elements waiting beside it (8192 x 2817 bf16 RMS: four 106 us, two 102, one 54).
inline Shape bwd_shape(const NormArgs& a) {
  int most = !a.vec ? 1 : !a.want_b ? 4 : a.in_codes ? 1 : 2;
  Shape s = shape_for(a.width, most, 1);
  while (s.threads > bwd_threads(s.nv) / (s.nv == 1 ? 2 : 1)) s = shape_for(a.width, most *= 2, 1);
  s.rows = bwd_threads(s.nv) / s.threads;
  if (s.threads > 32 && s.rows > 15) s.rows = 15;  // named barriers
  return s;
}

inline int bwd_blocks(const Shape& s, int rows) {
  const int need = ceil_div(rows, s.rows);
  return need < kBwdBlocks ? need : kBwdBlocks;
}

// The kernels for one element type (norm_fwd.cu, norm_bwd_f32.cu, norm_bwd_bf16.cu, norm_bwd_f16.cu). a.rows > 0.
template <class T>
cudaError_t run_norm_fwd(const NormArgs& a, int type, cudaStream_t st);
template <class T>
cudaError_t run_norm_bwd(const NormArgs& a, int type, cudaStream_t st);

}  // namespace r4
