// Expert selection from router scores s [Q, E], and its backward:
//     p   = sigmoid(s) or softmax(s),  key = p + balance bias
//     groups: a group's score is the sum of its best one or two keys, the
//             groups_kept best groups stay in
//     ids = the k experts of largest key, ties to the lower index
//     w   = scale p_i / (sum of the k p)   or   scale p_i
// The bias ranks only; it has no gradient. A score of -inf (or NaN) has
// p = 0 and ranks last.
//
// Selection decides between real numbers, so it must not depend on how fp32
// rounds p + bias. Without a bias p grows with s and the scores themselves are
// compared. With one (and for sums of two keys) the keys are formed in fp32
// with an error bound. Where the gaps between the best keys exceed the bound
// the selection stands; experts or groups whose order is open (about one token
// in a hundred has some) are ordered again by their keys in double. Tokens that
// the fp32 form cannot hold (too few scores left, keys out of range, more than
// 31 candidates of open order) are selected in double as a whole. That is slow
// where it is every token: 8192 x 384 fp32 sigmoid with a bias takes 14 us, with
// four scores left a token 42, with equal keys everywhere (a router's start) 64.
//
// One warp a token, scores in registers, four neighbours a lane and step. A
// key becomes one 32-bit number: its place in the range of possible keys (23
// bits of a float in [1, 2)) above the expert's index, counted down, so that a
// round of the top-k is one warp-wide integer maximum that names the expert as
// well. 16-bit scores that are ranked as they are keep all their bits there.
// Each lane keeps its best two numbers at hand; only a lane that has given away
// both looks at its scores again. Warps walk over tokens, the next token's
// scores already on their way, and count the routed slots in shared memory.
//
// Backward, with a_i = p_i / (sum of the k p) and gbar = sum of g_i a_i:
//     sigmoid: ds_i = scale a_i (1 - p_i) (g_i - gbar)   or  scale g_i p_i (1 - p_i)
//     softmax: ds_i = scale a_i (g_i - gbar)             or
//              ds_j = scale p_j ([j selected] g_j - sum of g_i p_i)  for every expert j
// Products like a_i and the sigmoid's tails are formed from exponents scaled
// by the largest selected one, so they do not underflow together.
#pragma once
#include <type_traits>

#include "select.cuh"

namespace r4 {
namespace {

constexpr int kWarps = 16;    // warps of a block at most, one token each at a time
constexpr int kBwdThreads = 128;

// Floats as unsigned integers of the same order (not for NaN).
__device__ __forceinline__ uint32_t ordered32(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered32(uint32_t u) {
  return __uint_as_float(u ^ ((uint32_t)((int32_t)~u >> 31) | 0x80000000u));
}
__device__ __forceinline__ float warp_max_f(float v) {
  return from_ordered32(__reduce_max_sync(0xffffffffu, ordered32(v)));
}
// A 16-bit score (in fp32) as a 16-bit integer of the same order, at least 0x7f.
template <class T>
__device__ __forceinline__ uint32_t ordered16(float v) {
  const T h = Elem<T>::from(v);
  const uint32_t b = *reinterpret_cast<const uint16_t*>(&h);
  return b & 0x8000u ? b ^ 0xFFFFu : b | 0x8000u;
}
__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum and maximum over the LANES lanes of a token.
template <int LANES>
__device__ __forceinline__ float part_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float part_max(float v) {
  if constexpr (LANES == 32) {
    return warp_max_f(v);
  } else {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}

// Two of them at once (NaN becomes -inf, -0 becomes +0), and back.
template <class T>
__device__ __forceinline__ uint32_t ordered16_pair(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 low = __half2half2(__ushort_as_half(0xFC00));
    const __half2 v = __hmax2(__hadd2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(0.f)), low);
    w = *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 low = __bfloat162bfloat162(__ushort_as_bfloat16(0xFF80));
    const __nv_bfloat162 v =
        __hmax2(__hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(0.f)), low);
    w = *reinterpret_cast<const uint32_t*>(&v);
  }
  return w ^ ((w >> 15 & 0x00010001u) * 0x7FFFu + 0x80008000u);
}
template <class T>
__device__ __forceinline__ float from_ordered16(uint32_t o) {
  const uint16_t b = (uint16_t)(o & 0x8000u ? o ^ 0x8000u : o ^ 0xFFFFu);
  return Elem<T>::to(*reinterpret_cast<const T*>(&b));
}

// A score as the ranking sees it: NaN counts as -inf, -0 as +0.
template <class T>
__device__ __forceinline__ float clean_score(T v) {
  const float s = Elem<T>::to(v);
  return s == s ? s + 0.0f : -INFINITY;
}

// Doubles as unsigned integers of the same order; all are above 0, which
// marks an expert that is out.
__device__ __forceinline__ uint64_t ordered(double v) {
  if (!(v == v)) v = -INFINITY;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double from_ordered(uint64_t u) {
  return __longlong_as_double((long long)(u >> 63 ? u & 0x7FFFFFFFFFFFFFFFull : ~u));
}

// exp(s - m) with the convention that an infinite maximum is shared by those that reach it.
__device__ __forceinline__ float shifted_exp(float s, float m) { return s == m ? 1.f : expf(s - m); }

// Lane j < k holds the score of slot j (-inf otherwise). Returns the slot's
// unnormalised probability and, in *total, its sum over the k slots.
__device__ __forceinline__ float slot_share(float s, int sigmoid, float* total) {
  const float top = warp_max_f(s);
  float q = 0.f;
  if (top > -INFINITY && s > -INFINITY) {
    if (sigmoid) q = expf(fminf(s, 0.f) - fminf(top, 0.f)) / (1.f + expf(-fabsf(s)));
    else q = shifted_exp(s, top);
  }
  *total = row_warp_sum(q);
  return q;
}

// ------------------------------------------------------- selection in double
// The expert of slot `lane` (lane < k) of token t; `key` is the warp's scratch,
// one key an expert. Also for rows too wide for registers.
template <class T>
__device__ __noinline__ int select_double(const SelectArgs& a, int t, uint64_t* key) {
  const int lane = threadIdx.x & 31;
  const T* z = static_cast<const T*>(a.scores) + t * a.ld;
  double m = 0.0, denom = 1.0;  // softmax: largest score and sum of exponentials
  if (!a.sigmoid && (a.bias || a.group_top > 1)) {
    float mf = -INFINITY;
    for (int e = lane; e < a.E; e += 32) mf = fmaxf(mf, clean_score(z[e]));
    m = warp_max_f(mf);
    double sum = 0.0;
    for (int e = lane; e < a.E; e += 32) {
      const double s = clean_score(z[e]);
      sum += s == m ? 1.0 : exp(s - m);
    }
    denom = warp_sum_d(sum);
  }
  auto prob = [&](double s) {
    if (s == -INFINITY) return 0.0;
    return a.sigmoid ? 1.0 / (1.0 + exp(-s)) : (s == m ? 1.0 : exp(s - m)) / denom;
  };
  __syncwarp();
  for (int e = lane; e < a.E; e += 32) {
    const double s = clean_score(z[e]);
    key[e] = ordered(a.bias && s > -INFINITY ? prob(s) + (double)a.bias[e] : s);
  }
  __syncwarp();

  if (a.groups > 1) {
    const int size = a.E / a.groups;
    uint64_t mine = 0;  // lane g: score of group g
    for (int g = 0; g < a.groups; ++g) {
      uint64_t b1 = 0, b2 = 0;
      for (int e = lane; e < size; e += 32) {
        const uint64_t u = key[g * size + e];
        if (u > b1) {
          b2 = b1;
          b1 = u;
        } else if (u > b2) {
          b2 = u;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
        b2 = c1 > b1 ? max(b1, c2) : max(b2, c1);
        b1 = max(b1, c1);
      }
      if (a.group_top > 1) {  // b2 exists: groups hold at least two experts
        double v1 = from_ordered(b1), v2 = from_ordered(b2);
        if (!a.bias) {
          v1 = v1 > -INFINITY ? prob(v1) : v1;
          v2 = v2 > -INFINITY ? prob(v2) : v2;
        }
        b1 = ordered(v2 > -INFINITY ? v1 + v2 : v1);
      }
      if (lane == g) mine = b1;
    }
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t u = __shfl_sync(0xffffffffu, mine, g);
      better += u > mine || (u == mine && g < lane);
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, lane < a.groups && better < a.kept);
    for (int e = lane; e < a.E; e += 32)
      if (!((kept >> (e / size)) & 1u)) key[e] = 0;
    __syncwarp();
  }

  int id = 0;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = 0;
    int at = 0x7fffffff;
    for (int e = lane; e < a.E; e += 32) {
      const uint64_t u = key[e];
      if (u > best) {
        best = u;
        at = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t u = __shfl_xor_sync(0xffffffffu, best, o);
      const int i = __shfl_xor_sync(0xffffffffu, at, o);
      if (u > best || (u == best && i < at)) {
        best = u;
        at = i;
      }
    }
    if (lane == j) id = at;
    if (lane == (at & 31)) key[at] = 0;
    __syncwarp();
  }
  return id;
}

// ------------------------------------------------------ scores in registers
// Lane l holds experts 128 i + 4 l + j, j < 4, i < NI; places past the last
// expert hold -inf.
template <class T>
struct alignas(4 * sizeof(T)) Four {
  T v[4];
};

template <class T, int NI, bool VEC>
__device__ __forceinline__ void fetch_scores(const T* z, int E, int lane, Four<T> (&r)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = 128 * i + 4 * lane;
    if (VEC) {  // E % 4 == 0 and every row aligned to four scores
      if (e < E) r[i] = *reinterpret_cast<const Four<T>*>(z + e);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < E) r[i].v[j] = z[e + j];
    }
  }
}
__device__ __forceinline__ int expert_at(int slot, int lane) { return 128 * (slot >> 2) + 4 * lane + (slot & 3); }

// Keys further than this below the largest possible one share the lowest place.
constexpr float kSpread = 60.f;

// p by the fast exponential (relative error 2^-22, and the rounding of its
// argument, below 1.2 |s| 2^-23) and reciprocal (1 ulp): p (1 - p) |s| < 1/4, so
// the error of p is below 2^-21. A softmax adds its sum's E / 32 + 5 roundings
// (`key_error`).
__device__ __forceinline__ float fast_sigmoid(float s) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// A gap between two fp32 keys that their errors cannot close; p + bias rounds
// by 2^-24 of its size.
__device__ __forceinline__ bool apart(float hi, float lo, float err, float size) {
  return lo == -INFINITY || hi - lo > 2.f * err + 0x1p-22f * size;
}

// Lane l < n holds a candidate e of token t; those whose order the fp32 keys
// leave open are put in order by their keys in double. Returns the expert of
// slot `lane`. m: the largest score.
template <class T>
__device__ __noinline__ int order_double(const SelectArgs& a, int t, int e, int n, float m, int* place) {
  const int lane = threadIdx.x & 31;
  const T* z = static_cast<const T*>(a.scores) + t * a.ld;
  double exact = lane < n ? (double)clean_score(z[e]) : -INFINITY;
  if (a.bias) {
    double sum = 1.0;
    if (!a.sigmoid) {
      sum = 0.0;
      for (int q = lane; q < a.E; q += 32) {
        const double v = clean_score(z[q]);
        sum += v == (double)m ? 1.0 : exp(v - (double)m);
      }
      sum = warp_sum_d(sum);
    }
    if (lane < n) {
      exact = a.sigmoid ? 1.0 / (1.0 + exp(-exact)) : (exact == (double)m ? 1.0 : exp(exact - (double)m)) / sum;
      exact += (double)a.bias[e];
    }
  }
  int rank = 0;
  for (int o = 0; o < n; ++o) {
    const double u = __shfl_sync(0xffffffffu, exact, o);
    const int eo = __shfl_sync(0xffffffffu, e, o);
    rank += u > exact || (u == exact && eo < e);
  }
  __syncwarp();
  if (lane < n && rank < a.k) place[rank] = e;
  __syncwarp();
  const int id = lane < a.k ? place[lane] : 0;
  __syncwarp();
  return id;
}

// Of the groups marked in `open` (bit g << share for group g), the `need` best
// by their scores in double, marked the same way.
template <class T>
__device__ __noinline__ uint32_t groups_double(const SelectArgs& a, int t, uint32_t open, int need, int share, float m) {
  const int lane = threadIdx.x & 31, size = a.E / a.groups;
  const T* z = static_cast<const T*>(a.scores) + t * a.ld;
  double denom = 1.0;
  if (!a.sigmoid) {
    denom = 0.0;
    for (int e = lane; e < a.E; e += 32) {
      const double v = clean_score(z[e]);
      denom += v == (double)m ? 1.0 : exp(v - (double)m);
    }
    denom = warp_sum_d(denom);
  }
  auto prob = [&](double s) {
    return a.sigmoid ? 1.0 / (1.0 + exp(-s)) : (s == (double)m ? 1.0 : exp(s - (double)m)) / denom;
  };
  double mine = -INFINITY;  // lane g << share: the score of group g
  for (uint32_t left = open; left; left &= left - 1) {
    const int at = __ffs(left) - 1;
    double b1 = -INFINITY, b2 = -INFINITY;
    for (int i = lane; i < size; i += 32) {
      const int e = (at >> share) * size + i;
      double v = clean_score(z[e]);
      if (a.bias && v > -INFINITY) {
        const double b = a.bias[e];
        v = b == b ? prob(v) + b : -INFINITY;
      }
      b2 = fmax(b2, fmin(b1, v));
      b1 = fmax(b1, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
      b2 = fmax(fmin(b1, c1), fmax(b2, c2));
      b1 = fmax(b1, c1);
    }
    if (a.group_top > 1) {
      if (!a.bias) {
        b1 = b1 > -INFINITY ? prob(b1) : b1;
        b2 = b2 > -INFINITY ? prob(b2) : b2;
      }
      b1 = b2 > -INFINITY ? b1 + b2 : b1;
    }
    if (lane == at) mine = b1;
  }
  int better = 0;
  for (uint32_t left = open; left; left &= left - 1) {
    const int at = __ffs(left) - 1;
    const double u = __shfl_sync(0xffffffffu, mine, at);
    better += u > mine || (u == mine && at < lane);
  }
  return __ballot_sync(0xffffffffu, (open >> lane & 1u) && better < need);
}

// The group stage: experts outside the groups_kept best groups are closed (their
// bits of the result cleared). Groups whose order around the border the fp32
// keys leave open are ordered in double. `row`: the warp's scratch.
template <class T, int NP, class Prob>
__device__ __forceinline__ uint32_t open_experts(const SelectArgs& a, int t, const float (&s)[NP], float* row, int lane,
                                                 float key_error, float m, Prob prob) {
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (expert_at(i, lane) < a.E) row[expert_at(i, lane)] = s[i];
  __syncwarp();
  const int size = a.E / a.groups;
  // 2^share lanes a group, each with every 2^share-th of its experts
  const int share = 31 - __clz(32 / a.groups);
  const int g = lane >> share, part = lane & ((1 << share) - 1);
  float b1 = -INFINITY, b2 = -INFINITY;
  if (g < a.groups)
    for (int e = part; e < size; e += 1 << share) {
      const float u = row[g * size + e];
      b2 = fmaxf(b2, fminf(b1, u));
      b1 = fmaxf(b1, u);
    }
  for (int o = 1; o < 1 << share; o <<= 1) {
    const float c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
    b2 = fmaxf(fminf(b1, c1), fmaxf(b2, c2));
    b1 = fmaxf(b1, c1);
  }
  float magnitude = fabsf(b1);
  if (a.group_top > 1) {
    if (!a.bias) {  // a softmax's denominator is common to all groups
      b1 = b1 > -INFINITY ? prob(b1) : b1;
      b2 = b2 > -INFINITY ? prob(b2) : b2;
    }
    magnitude = fabsf(b1) + (b2 > -INFINITY ? fabsf(b2) : 0.f);
    b1 = b2 > -INFINITY ? b1 + b2 : b1;
  }
  int better = 0;  // groups ahead of the lane's
  for (int o = 0; o < a.groups; ++o) {
    const float u = __shfl_sync(0xffffffffu, b1, o << share);
    better += u > b1 || (u == b1 && o < g);
  }
  const bool first = part == 0 && g < a.groups;  // one lane speaks for a group
  const bool in = first && better < a.kept;
  uint32_t kept = __ballot_sync(0xffffffffu, in);
  if (a.kept < a.groups && (a.bias || a.group_top > 1)) {
    const float lo = -warp_max_f(in ? -b1 : -INFINITY), hi = warp_max_f(first && !in ? b1 : -INFINITY);
    const float most = warp_max_f(first && magnitude < INFINITY ? magnitude : 0.f);
    const bool sure = in ? apart(b1, hi, 2.f * key_error, 4.f * most) : apart(lo, b1, 2.f * key_error, 4.f * most);
    const uint32_t open = __ballot_sync(0xffffffffu, first && !sure);
    if (open) {
      kept &= ~open;
      kept |= groups_double<T>(a, t, open, a.kept - __popc(kept), share, m);
    }
  }
  const float inv_size = 1.f / (float)size;  // (e + 0.5) / size truncates to e / size for e < 4096
  uint32_t mask = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int of = (int)(((float)expert_at(i, lane) + 0.5f) * inv_size);
    if (!((kept >> ((of << share) & 31)) & 1u)) mask &= ~(1u << i);
  }
  __syncwarp();
  return mask;
}

template <class T, int NI, bool VEC, bool BIAS, bool GROUPS>
__global__ void __launch_bounds__(32 * kWarps, NI <= 4 ? 2 : 1) select_kernel(const SelectArgs a) {
  begin_after_previous();
  constexpr int NP = 4 * NI;
  constexpr bool kWhole = sizeof(T) == 2 && !BIAS;  // 16-bit scores ranked as they are: all their bits, no rounding
  constexpr int kIndexBits = NI == 1 ? 7 : NI == 2 ? 8 : NI <= 4 ? 9 : 10;
  constexpr uint32_t kIndex = (1u << kIndexBits) - 1;
  constexpr int kShift = kIndexBits > 9 ? kIndexBits : 9;  // ten index bits cost the place its lowest bit
  constexpr float kStep = 0x1p-23f * (1 << (kShift - 9));  // of a place, in [1, 2)
  constexpr float kFloor = 1.f + 0x1p-8f;
  constexpr uint32_t kFloorPlace = (1u << 15) >> (kShift - 9);
  extern __shared__ uint64_t keys[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* const scratch = keys + (size_t)warp * a.E;
  int* const tally = reinterpret_cast<int*>(keys + (size_t)warps * a.E);
  const int step = gridDim.x * warps;
  int t = blockIdx.x * warps + warp;
  const T* const all = static_cast<const T*>(a.scores);

  Four<T> ahead[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) ahead[i].v[j] = Elem<T>::from(-INFINITY);
  if (t < a.Q) fetch_scores<T, NI, VEC>(all + t * a.ld, a.E, lane, ahead);
  if (a.counts) {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) tally[e] = 0;
    __syncthreads();
  }
  // the bias of the lane's experts, and the range of keys p + bias
  float bias[BIAS ? NP : 1], low = 0.f, range = 1.f;
  if constexpr (BIAS) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int e = expert_at(i, lane);
      const float b = e < a.E ? a.bias[e] : -INFINITY;
      bias[i] = b == b ? b : -INFINITY;
      hi = fmaxf(hi, bias[i]);
      lo = bias[i] > -INFINITY ? fminf(lo, bias[i]) : lo;
    }
    hi = warp_max_f(hi);
    low = fmaxf(-warp_max_f(-lo), hi - kSpread);
    range = hi + 1.f - low;
  }
  const float key_error = a.sigmoid ? 0x1p-21f : 0x1p-21f + (NP + 16) * 0x1p-23f;

  for (; t < a.Q; t += step) {
    float s[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) s[i] = fmaxf(Elem<T>::to(ahead[i >> 2].v[i & 3]), -INFINITY);  // NaN counts as -inf
    const T* z = all + t * a.ld;
    if (t + step < a.Q) fetch_scores<T, NI, VEC>(all + (t + step) * a.ld, a.E, lane, ahead);

    float m = -INFINITY, denom = 1.f;
    if ((!BIAS && !kWhole) || !a.sigmoid) {
#pragma unroll
      for (int i = 0; i < NP; ++i) m = fmaxf(m, s[i]);
      m = warp_max_f(m);
    }
    if (!a.sigmoid && (BIAS || !a.renorm)) {
      denom = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) denom += s[i] > -INFINITY ? shifted_exp(s[i], m) : 0.f;
      denom = row_warp_sum(denom);
    }
    auto prob = [&](float v) { return a.sigmoid ? fast_sigmoid(v) : shifted_exp(v, m) / denom; };
    if constexpr (BIAS) {  // from here on s is what is ranked: the key, -inf where it ranks last
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NP; ++i) s[i] = s[i] > -INFINITY ? fast_sigmoid(s[i]) + bias[i] : -INFINITY;
      } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) s[i] = s[i] > -INFINITY ? shifted_exp(s[i], m) / denom + bias[i] : -INFINITY;
      }
    }
    bool sure = true;
    uint32_t open = 0xffffffffu;  // bit i: the lane's expert i lies in a kept group
    if constexpr (GROUPS) {
      open = open_experts<T, NP>(a, t, s, reinterpret_cast<float*>(scratch), lane, key_error, m, prob);
      if (!kWhole)
#pragma unroll
        for (int i = 0; i < NP; ++i) s[i] = open >> i & 1u ? s[i] : -INFINITY;
    }

    uint32_t u[NP];  // the numbers; 0 is no candidate
    float number_error = 0.f;
    if constexpr (kWhole) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        u[i] = ordered16<T>(s[i] + 0.f) << 16 | (kIndex - (uint32_t)expert_at(i, lane));
        if (GROUPS) u[i] = open >> i & 1u ? u[i] : 0u;
      }
    } else {
      if constexpr (!BIAS) {
        float least = INFINITY;
#pragma unroll
        for (int i = 0; i < NP; ++i) least = s[i] > -INFINITY ? fminf(least, s[i]) : least;
        low = fmaxf(-warp_max_f(-least), m - kSpread);
        range = m - low;
      }
      // [low, low + range] to [1 + 2^-7, 2 - 2^-6]; what lies below shares the lowest place (closed groups and
      // scores of -inf among it), and a token that would give that place a slot is selected in double
      const float scale = range > 0.f ? __fdividef(1.f - 0x1p-5f, range) : 0.f, offset = fmaf(-low, scale, 1.f + 0x1p-7f);
      number_error = range * 0x1p-20f;  // of a place, as a key: the product's rounding and the cut
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint32_t f = __float_as_uint(fmaxf(fmaf(s[i], scale, offset), kFloor));
        u[i] = (f << 9 & ~kIndex) | (kIndex - (uint32_t)expert_at(i, lane));
      }
    }

    // each lane's best numbers at hand: all four in order, or two
    uint32_t b1 = 0u, b2 = 0u, b3 = 0u, b4 = 0u;
    auto look = [&](uint32_t below) {
      b1 = b2 = 0u;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint32_t v = u[i] < below ? u[i] : 0u;
        b2 = max(b2, min(b1, v));
        b1 = max(b1, v);
      }
    };
    if constexpr (NI == 1) {
      const uint32_t h1 = max(u[0], u[1]), l1 = min(u[0], u[1]), h2 = max(u[2], u[3]), l2 = min(u[2], u[3]);
      b1 = max(h1, h2);
      b4 = min(l1, l2);
      const uint32_t x = min(h1, h2), y = max(l1, l2);
      b2 = max(x, y);
      b3 = min(x, y);
    } else {
      look(0xffffffffu);
    }
    auto round = [&]() {
      const uint32_t best = __reduce_max_sync(0xffffffffu, b1);
      const bool mine = b1 == best;
      if constexpr (NI == 1) {
        b1 = mine ? b2 : b1;
        b2 = mine ? b3 : b2;
        b3 = mine ? b4 : b3;
        b4 = mine ? 0u : b4;
      } else {
        if (__any_sync(0xffffffffu, mine && b2 == 0u)) {
          if (mine) look(best);
        } else {
          b1 = mine ? b2 : b1;
          b2 = mine ? 0u : b2;
        }
      }
      return best;
    };
    uint32_t won = 0u;
    for (int j = 0; j < a.k; ++j) {
      const uint32_t best = round();
      if (lane == j) won = best;
    }
    int id = (int)(kIndex - (won & kIndex));
    if constexpr (!kWhole) {
      // the slot behind (behind the last slot: the best that is left); n steps between two places are at least
      // n - 1 steps of the keys, and both keys' errors have to fit
      const uint32_t rest = __reduce_max_sync(0xffffffffu, b1);
      const uint32_t behind = __shfl_down_sync(0xffffffffu, won, 1);
      const uint32_t next = lane + 1 < a.k ? behind : rest;
      const float unit = kStep * range;
      const float need = 2.f * number_error + (BIAS ? 2.f * key_error + 0x1p-21f * (fabsf(low) + range) : 0.f);
      const bool clear = (float)((won >> kShift) - (next >> kShift)) * unit > need;
      const bool floored = won >> kShift <= kFloorPlace;
      // ranges that the places cannot hold: infinite, or far away from 0 for their size
      if (__any_sync(0xffffffffu, lane < a.k && floored) || !(range < INFINITY) || fabsf(low) > 0x1p14f * range) {
        sure = false;
      } else if (__any_sync(0xffffffffu, lane < a.k && !clear)) {
        const uint32_t last = __shfl_sync(0xffffffffu, won, a.k - 1);
        int n = a.k;
        while (n < 32) {  // all that may belong to the slots
          const uint32_t top = __reduce_max_sync(0xffffffffu, b1);
          if (top >> kShift <= kFloorPlace || (float)((last >> kShift) - (top >> kShift)) * unit > need) break;
          round();
          if (lane == n) won = top;
          ++n;
        }
        if (n < 32 && sure) id = order_double<T>(a, t, (int)(kIndex - (won & kIndex)), n, m, reinterpret_cast<int*>(scratch));
        sure = sure && n < 32;
      }
    }
    if (!sure) id = select_double<T>(a, t, scratch);

    const float v = lane < a.k ? clean_score(z[id]) : -INFINITY;
    float w;
    if (a.renorm) {
      float total;
      const float q = slot_share(v, a.sigmoid, &total);
      w = total > 0.f ? a.scale * (q / total) : 0.f;
    } else {
      w = v > -INFINITY ? a.scale * (a.sigmoid ? 1.f / (1.f + expf(-v)) : shifted_exp(v, m) / denom) : 0.f;
    }
    if (lane < a.k) {
      a.ids[(int64_t)t * a.k + lane] = id;
      a.weights[(int64_t)t * a.k + lane] = w;
      if (a.counts) atomicAdd(tally + id, 1);
    }
  }
  if (a.counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
      if (tally[e]) atomicAdd(a.counts + e, tally[e]);
  }
}

// ------------------------------------------------- many tokens, few experts
// 16-bit scores ranked as they are, at most 128 experts, eight slots, no
// groups: four tokens a warp, eight lanes each, so what a token costs beside
// its scores (rounds, weights, stores) is shared by four. Lane l of a token
// holds experts 64 i + 8 l + j, i < 2, j < 8, sorts their numbers and keeps the
// best eight in order; a round is three exchanges and a shift. (Keys that need
// the error bound lose this way: 65536 x 128 fp32 with bias 37 us, 31 one a warp.)
constexpr int kManyExperts = 128;
constexpr uint32_t kManyIndex = kManyExperts - 1;

__device__ __forceinline__ void order_two(uint32_t& a, uint32_t& b) {  // a >= b
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
// Descending order of eight numbers (Batcher's odd-even merge sort).
__device__ __forceinline__ void order_eight(uint32_t (&v)[8]) {
#pragma unroll
  for (int p = 1; p < 8; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < 8; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < 8 && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order_two(v[i + j], v[i + j + k]);
}

template <class T, bool VEC>
__global__ void __launch_bounds__(32 * kWarps, 2) select_many_kernel(const SelectArgs a) {
  begin_after_previous();
  extern __shared__ int tally[];
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, l = lane & 7;
  const int step = gridDim.x * warps * 4;
  int t = (blockIdx.x * warps + (threadIdx.x >> 5)) * 4 + (lane >> 3);
  const T* const all = static_cast<const T*>(a.scores);

  RawChunk<T> ahead[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) ahead[i] = narrow<T>(chunk_of(-INFINITY));
  auto fetch = [&](int t) {
    if (t >= a.Q) return;
    const T* z = all + t * a.ld;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 64 * i + 8 * l;
      if (VEC) {
        if (e < a.E) ahead[i] = load_chunk(z + e);
      } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
          if (e + j < a.E) reinterpret_cast<T*>(&ahead[i])[j] = z[e + j];
      }
    }
  };
  fetch(t);
  if (a.counts) {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) tally[e] = 0;
    __syncthreads();
  }
  // indexes of the lane's experts counted down, two 16-bit halves a register
  uint32_t index[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t e = 64 * (i >> 2) + 8 * l + 2 * (i & 3);
    index[i] = (kManyIndex - e) | (kManyIndex - e - 1) << 16;
  }

  // all lanes of a warp make the same turns: the last token of each may lie past the end
  for (; t - (lane >> 3) < a.Q; t += step) {
    const RawChunk<T> raw[2] = {ahead[0], ahead[1]};
    fetch(t + step);
    uint32_t u[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t o = ordered16_pair<T>(raw[i].w[j]);
        u[i][2 * j] = __byte_perm(o, index[4 * i + j], 0x1054);
        u[i][2 * j + 1] = __byte_perm(o, index[4 * i + j], 0x3276);
      }
    // the lane's best eight in order: of two descending eights, the larger of each pair from opposite ends
    // is a bitonic sequence
    uint32_t b[8];
    order_eight(u[0]);
    order_eight(u[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = max(u[0][i], u[1][7 - i]);
#pragma unroll
    for (int k = 4; k > 0; k >>= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(i & k)) order_two(b[i], b[i + k]);
    uint32_t won = 0u, top = 0u;
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = b[0];
      best = max(best, __shfl_xor_sync(0xffffffffu, best, 4));
      best = max(best, __shfl_xor_sync(0xffffffffu, best, 2));
      best = max(best, __shfl_xor_sync(0xffffffffu, best, 1));
      if (l == j) won = best;
      if (j == 0) top = best;
      const bool mine = b[0] == best;
#pragma unroll
      for (int i = 0; i < 7; ++i) b[i] = mine ? b[i + 1] : b[i];
      b[7] = mine ? 0u : b[7];
    }
    const int id = (int)(kManyIndex - (won & kManyIndex));
    const float v = l < a.k ? from_ordered16<T>(won >> 16) : -INFINITY, m = from_ordered16<T>(top >> 16);
    float w = 0.f;
    if (a.renorm) {
      if (v > -INFINITY)
        w = a.sigmoid ? expf(fminf(v, 0.f) - fminf(m, 0.f)) / (1.f + expf(-fabsf(v))) : shifted_exp(v, m);
      const float total = part_sum<8>(w);
      w = total > 0.f ? a.scale * (w / total) : 0.f;
    } else if (a.sigmoid) {
      w = v > -INFINITY ? a.scale / (1.f + expf(-v)) : 0.f;
    } else {
      float denom = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Chunk s = widen<T>(raw[i]);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) denom += s[j] > -INFINITY ? shifted_exp(s[j], m) : 0.f;  // not for NaN either
      }
      denom = part_sum<8>(denom);
      w = v > -INFINITY ? a.scale * (shifted_exp(v, m) / denom) : 0.f;
    }
    if (t < a.Q && l < a.k) {
      a.ids[(int64_t)t * a.k + l] = id;
      a.weights[(int64_t)t * a.k + l] = w;
      if (a.counts) atomicAdd(tally + id, 1);
    }
  }
  if (a.counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
      if (tally[e]) atomicAdd(a.counts + e, tally[e]);
  }
}

// Rows of more than 1024 experts: the keys lie in shared memory, in double, and
// every round of the top-k looks at all of them (8192 x 1025 fp32 with a bias
// 117 us, x 4096 1140; 1024 experts in registers take 26). Built to be right, not
// to be quick.
template <class T>
__global__ void __launch_bounds__(32 * kWarps) select_wide_kernel(const SelectArgs a) {
  begin_after_previous();
  extern __shared__ uint64_t keys[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t = blockIdx.x * warps + warp; t < a.Q; t += gridDim.x * warps) {
    const T* z = static_cast<const T*>(a.scores) + t * a.ld;
    const int id = select_double<T>(a, t, keys + (size_t)warp * a.E);
    const float s = lane < a.k ? clean_score(z[id]) : -INFINITY;
    float w;
    if (a.renorm) {
      float total;
      const float q = slot_share(s, a.sigmoid, &total);
      w = total > 0.f ? a.scale * (q / total) : 0.f;
    } else if (a.sigmoid) {
      w = s > -INFINITY ? a.scale / (1.f + expf(-s)) : 0.f;
    } else {
      float m = -INFINITY, denom = 0.f;
      for (int e = lane; e < a.E; e += 32) m = fmaxf(m, clean_score(z[e]));
      m = warp_max_f(m);
      for (int e = lane; e < a.E; e += 32) denom += shifted_exp(clean_score(z[e]), m);
      denom = row_warp_sum(denom);
      w = s > -INFINITY ? a.scale * (shifted_exp(s, m) / denom) : 0.f;
    }
    if (lane < a.k) {
      a.ids[(int64_t)t * a.k + lane] = id;
      a.weights[(int64_t)t * a.k + lane] = w;
      if (a.counts) atomicAdd(a.counts + id, 1);
    }
  }
}

// ----------------------------------------------------------------- backward
// LANES (8 or 32, at least k) lanes a token, so that small selections share a
// warp's instructions. Experts lie in chunks of eight, chunk c in lane c %
// LANES. NI > 0: a softmax over all experts keeps the lane's NI chunks in
// registers; NI = 0: no such gradient, or any number of experts, read again
// from cache.
template <class T, bool VEC>
__device__ __forceinline__ Chunk score_chunk(const T* z, int e, int E) {
  Chunk c = chunk_of(-INFINITY);
  if (VEC) {
    if (e < E) c = widen<T>(load_chunk(z + e));
  } else {
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
      if (e + j < E) c[j] = Elem<T>::to(z[e + j]);
  }
#pragma unroll
  for (int j = 0; j < kChunk; ++j) c[j] = fmaxf(c[j], -INFINITY);  // NaN counts as -inf
  return c;
}

template <class T, int LANES, int NI, bool VEC>
__global__ void __launch_bounds__(kBwdThreads) select_bwd_kernel(const SelectArgs a) {
  begin_after_previous();
  const int lane = threadIdx.x % LANES;
  const int t = blockIdx.x * (kBwdThreads / LANES) + threadIdx.x / LANES;
  const bool live = t < a.Q;
  const T* z = static_cast<const T*>(a.scores) + t * a.ld;
  T* dz = static_cast<T*>(a.grad) + (int64_t)t * a.E;
  const bool softmax_all = !a.sigmoid && !a.renorm;  // the gradient reaches every expert
  Chunk s[NI ? NI : 1];
  if (NI > 0)
#pragma unroll
    for (int i = 0; i < NI; ++i) s[i] = score_chunk<T, VEC>(z, (i * LANES + lane) * kChunk, live ? a.E : 0);

  int id = -1;
  float g = 0.f, v = -INFINITY;
  if (live && lane < a.k) {
    const int64_t wide = a.ids_in[(int64_t)t * a.k + lane];
    const float gr = a.grad_route[(int64_t)t * a.k + lane];
    if (wide >= 0 && wide < a.E) {  // any other id contributes nothing
      id = (int)wide;
      v = clean_score(z[id]);
      g = gr * a.scale;
    }
  }
  float d = 0.f, m = -INFINITY, every = 0.f;  // d: the slot's share of the gradient
  if (!softmax_all) {
    if (live) {  // zeros everywhere, while the slots' loads are on their way
      if (VEC) {
        for (int e = lane * kChunk; e < a.E; e += LANES * kChunk) store_chunk(dz + e, chunk_of(0.f));
      } else {
        for (int e = lane; e < a.E; e += LANES) dz[e] = Elem<T>::from(0.f);
      }
    }
    float q = 0.f;
    if (a.renorm) {
      const float top = part_max<LANES>(v);
      if (v > -INFINITY)
        q = a.sigmoid ? expf(fminf(v, 0.f) - fminf(top, 0.f)) / (1.f + expf(-fabsf(v))) : shifted_exp(v, top);
      const float total = part_sum<LANES>(q);
      const float share = total > 0.f ? q / total : 0.f;
      d = share * (g - part_sum<LANES>(g * share));
    } else {
      d = v > -INFINITY ? g / (1.f + expf(-v)) : 0.f;
    }
    if (a.sigmoid && v > -INFINITY) d *= 1.f / (1.f + expf(v));
  } else {
    float denom = 0.f;
    if (NI > 0) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < kChunk; ++j) m = fmaxf(m, s[i][j]);
      m = part_max<LANES>(m);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          s[i][j] = s[i][j] > -INFINITY ? shifted_exp(s[i][j], m) : 0.f;
          denom += s[i][j];
        }
    } else {
      for (int e = lane; live && e < a.E; e += LANES) m = fmaxf(m, clean_score(z[e]));
      m = part_max<LANES>(m);
      for (int e = lane; live && e < a.E; e += LANES) denom += shifted_exp(clean_score(z[e]), m);
    }
    const float mine = v > -INFINITY ? g * shifted_exp(v, m) : 0.f;
    denom = part_sum<LANES>(denom);
    const float base = part_sum<LANES>(mine);
    const float inv = m > -INFINITY ? 1.f / denom : 0.f;
    d = mine * inv;
    every = -base * inv * inv;  // an expert's gradient over exp(s - m), without its own slots
  }
  if (live) {
    if (NI > 0) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int e = (i * LANES + lane) * kChunk;
#pragma unroll
        for (int j = 0; j < kChunk; ++j) s[i][j] *= every;
        if (VEC) {
          if (e < a.E) store_chunk(dz + e, s[i]);
        } else {
#pragma unroll
          for (int j = 0; j < kChunk; ++j)
            if (e + j < a.E) dz[e + j] = Elem<T>::from(s[i][j]);
        }
      }
    } else if (softmax_all) {
      for (int e = lane; e < a.E; e += LANES)
        dz[e] = Elem<T>::from(m > -INFINITY ? every * shifted_exp(clean_score(z[e]), m) : 0.f);
    }
  }
  // slots of one expert are added by the first of them
  const int base_lane = (threadIdx.x & 31) - lane;
  bool first = id >= 0;
  uint32_t same = __match_any_sync(0xffffffffu, id < 0 ? -1 - (int)(threadIdx.x & 31) : id * 4 + (base_lane >> 3));
  if (__any_sync(0xffffffffu, same & (same - 1))) {
    float sum = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const float part = __shfl_sync(0xffffffffu, d, base_lane + j);
      if (same >> (base_lane + j) & 1u) sum += part;
    }
    if (first) d = sum;
    first = first && (int)(threadIdx.x & 31) == __ffs(same) - 1;
  }
  if (softmax_all && v > -INFINITY) d += every * shifted_exp(v, m);
  __syncwarp();
  if (first) dz[id] = Elem<T>::from(d);
}

// Four neighbouring scores move at once where every row allows it.
template <class T>
bool four_aligned(const void* p, int64_t ld, int E) {
  return E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0;
}

// From here on four tokens a warp are quicker than one (128 experts, k 8, bf16:
// 2048 tokens 3.0 and 3.3 us, 16384 tokens 5.4 and 10.0).
constexpr int kManyTokens = 2048;

struct SelectShape {
  int blocks, warps, smem;
};

// Two blocks an SM walk over the tokens, with as many warps each (at most
// kWarps and 96 KB of scratch) as give every warp the same number of tokens.
SelectShape select_shape(const SelectArgs& a, int sms) {
  const int row = a.E * (int)sizeof(uint64_t), blocks = 2 * sms;
  const int most = 96 * 1024 / row < kWarps ? 96 * 1024 / row : kWarps;
  const int turns = (a.Q + blocks * most - 1) / (blocks * most);
  const int warps = (a.Q + blocks * turns - 1) / (blocks * turns);
  const int need = (a.Q + warps - 1) / warps;
  return {need < blocks ? need : blocks, warps, warps * row + (a.counts ? a.E * (int)sizeof(int) : 0)};
}

template <class K>
cudaError_t start(K kernel, std::atomic<unsigned long long>& opted, const SelectArgs& a, const SelectShape& s,
                  cudaStream_t st) {
  int dev = 0;
  if (!device_flag_test(opted, &dev)) {
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    if (err != cudaSuccess) return err;
    device_flag_set(opted, dev);
  }
  return launch_early(kernel, s.blocks, 32 * s.warps, s.smem, st, a);
}

template <class T, int NI, bool VEC, bool BIAS, bool GROUPS>
cudaError_t start_select(const SelectArgs& a, const SelectShape& s, cudaStream_t st) {
  static std::atomic<unsigned long long> opted{0};
  return start(select_kernel<T, NI, VEC, BIAS, GROUPS>, opted, a, s, st);
}

template <class T, int NI, bool VEC>
cudaError_t pick_select(const SelectArgs& a, const SelectShape& s, cudaStream_t st) {
  if (a.groups > 1)
    return a.bias ? start_select<T, NI, VEC, true, true>(a, s, st) : start_select<T, NI, VEC, false, true>(a, s, st);
  return a.bias ? start_select<T, NI, VEC, true, false>(a, s, st) : start_select<T, NI, VEC, false, false>(a, s, st);
}

template <class T, int NI>
cudaError_t launch_select(const SelectArgs& a, const SelectShape& s, cudaStream_t st) {
  return four_aligned<T>(a.scores, a.ld, a.E) ? pick_select<T, NI, true>(a, s, st) : pick_select<T, NI, false>(a, s, st);
}

template <class T>
cudaError_t launch_many(const SelectArgs& a, int sms, cudaStream_t st) {
  SelectArgs quarter = a;  // a warp's turn is four tokens
  quarter.Q = (a.Q + 3) / 4;
  const SelectShape s = select_shape(quarter, sms);
  const bool vec = a.E % kChunk == 0 && rows_aligned(a.scores, a.ld, RAWINT4_TYPE_BF16);
  return launch_early(vec ? select_many_kernel<T, true> : select_many_kernel<T, false>, s.blocks, 32 * s.warps,
                      a.E * (int)sizeof(int), st, a);
}

template <class T>
cudaError_t select_type(const SelectArgs& a, int sms, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (!a.bias && a.E <= kManyExperts && a.k <= 8 && a.groups == 1 && a.Q >= kManyTokens) return launch_many<T>(a, sms, st);
  const SelectShape s = select_shape(a, sms);
  if (a.E <= 128) return launch_select<T, 1>(a, s, st);
  if (a.E <= 256) return launch_select<T, 2>(a, s, st);
  if (a.E <= 384) return launch_select<T, 3>(a, s, st);
  if (a.E <= 512) return launch_select<T, 4>(a, s, st);
  if (a.E <= 1024) return launch_select<T, 8>(a, s, st);
  static std::atomic<unsigned long long> opted{0};
  return start(select_wide_kernel<T>, opted, a, s, st);
}

template <class T, int LANES, int NI>
cudaError_t launch_bwd(const SelectArgs& a, cudaStream_t st) {
  const int tokens = kBwdThreads / LANES, blocks = (a.Q + tokens - 1) / tokens;
  const int type = sizeof(T) == 4 ? RAWINT4_TYPE_F32 : RAWINT4_TYPE_BF16;  // a size
  const bool vec = a.E % kChunk == 0 && rows_aligned(a.scores, a.ld, type) && rows_aligned(a.grad, a.E, type);
  return launch_early(vec ? select_bwd_kernel<T, LANES, NI, true> : select_bwd_kernel<T, LANES, NI, false>, blocks,
                      kBwdThreads, 0, st, a);
}

template <class T>
cudaError_t select_bwd_type(const SelectArgs& a, cudaStream_t st) {
  const bool all = !a.sigmoid && !a.renorm;
  // eight lanes a token (16384 x 128 fp32, k 8: 6.8 us, with 32 7.6), 32 where a row is longer (8192 x 384:
  // 6.4 us, with eight 8.5)
  if (a.k <= 8 && a.E <= 128) return all ? launch_bwd<T, 8, 2>(a, st) : launch_bwd<T, 8, 0>(a, st);
  if (!all || a.E > 1024) return launch_bwd<T, 32, 0>(a, st);
  if (a.E <= 256) return launch_bwd<T, 32, 1>(a, st);
  if (a.E <= 512) return launch_bwd<T, 32, 2>(a, st);
  return launch_bwd<T, 32, 4>(a, st);
}

}  // namespace
}  // namespace r4
