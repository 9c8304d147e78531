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
// the selection stands; the experts whose order is open (about one token in a
// hundred has some) are ordered again by their keys in double, and a token
// whose groups are open is selected again in double as a whole.
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
#include "prof.cuh"
#include "rows.cuh"

namespace r4 {
namespace {

constexpr int kWarps = 16;    // warps of a block at most, one token each at a time
constexpr int kBwdWarps = 4;

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
// Lane l holds experts 128 i + 4 l + j, j < 4, i < NI.
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
template <class T, int NI>
__device__ __forceinline__ void take_scores(const Four<T> (&r)[NI], int E, int lane, float (&s)[4 * NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[4 * i + j] = 128 * i + 4 * lane + j < E ? clean_score(r[i].v[j]) : -INFINITY;
}
__device__ __forceinline__ int expert_at(int slot, int lane) { return 128 * (slot >> 2) + 4 * lane + (slot & 3); }

// Keys further than this below the largest possible one share the lowest place.
constexpr float kSpread = 60.f;

// p by the fast exponential and division: with a relative error of the
// exponential below 2^-22 + 1.2 |s| 2^-23 (its documented bound), p (1 - p) |s|
// < 1/4, and the quotient's 2 ulp, the error of p is below 2^-21; a softmax adds
// its sum's E / 32 + 5 roundings (`key_error`).
__device__ __forceinline__ float fast_sigmoid(float s) { return __fdividef(1.f, 1.f + __expf(-s)); }

// A gap between two fp32 keys that their errors cannot close; p + bias rounds
// by 2^-24 of its size.
__device__ __forceinline__ bool apart(float hi, float lo, float err, float size) {
  return lo == -INFINITY || hi - lo > 2.f * err + 0x1p-22f * size;
}

template <class T, int NI, bool VEC>
__global__ void __launch_bounds__(32 * kWarps, NI <= 4 ? 2 : 1) select_kernel(const SelectArgs a) {
  constexpr int NP = 4 * NI;
  constexpr int kIndexBits = NI == 1 ? 7 : NI == 2 ? 8 : NI <= 4 ? 9 : 10;
  constexpr uint32_t kIndex = (1u << kIndexBits) - 1;
  constexpr int kShift = kIndexBits > 9 ? kIndexBits : 9;  // ten index bits cost the place its lowest bit
  extern __shared__ uint64_t keys[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* const scratch = keys + (size_t)warp * a.E;
  int* const tally = reinterpret_cast<int*>(keys + (size_t)warps * a.E);
  const int step = gridDim.x * warps;
  int t = blockIdx.x * warps + warp;
  const T* const all = static_cast<const T*>(a.scores);

  Four<T> ahead[NI];
  if (t < a.Q) fetch_scores<T, NI, VEC>(all + t * a.ld, a.E, lane, ahead);
  if (a.counts) {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) tally[e] = 0;
    __syncthreads();
  }
  // the bias of the lane's experts, and the range of finite keys p + bias
  float bias[NP], low = 0.f, range = 1.f;
  if (a.bias) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int e = expert_at(i, lane);
      const float b = e < a.E ? a.bias[e] : 0.f;
      bias[i] = b == b ? b : -INFINITY;
      if (e < a.E && fabsf(bias[i]) < INFINITY) {
        lo = fminf(lo, b);
        hi = fmaxf(hi, b);
      }
    }
    hi = warp_max_f(hi);
    low = fmaxf(-warp_max_f(-lo), hi - kSpread);
    range = hi + 1.f - low;
  }
  // 16-bit scores ranked as they are: all their bits, no rounding
  const bool whole = sizeof(T) == 2 && !a.bias;

  for (; t < a.Q; t += step) {
    float s[NP];
    take_scores<T, NI>(ahead, a.E, lane, s);
    const T* z = all + t * a.ld;
    if (t + step < a.Q) fetch_scores<T, NI, VEC>(all + (t + step) * a.ld, a.E, lane, ahead);

    float m = -INFINITY, denom = 1.f;
    if (!a.sigmoid || !(whole || a.bias)) {
#pragma unroll
      for (int i = 0; i < NP; ++i) m = fmaxf(m, s[i]);
      m = warp_max_f(m);
    }
    if (!a.sigmoid && (a.bias || !a.renorm)) {
      denom = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) denom += s[i] > -INFINITY ? shifted_exp(s[i], m) : 0.f;
      denom = row_warp_sum(denom);
    }
    const float key_error = a.sigmoid ? 0x1p-21f : 0x1p-21f + (NP + 16) * 0x1p-23f;
    auto prob = [&](float v) { return a.sigmoid ? fast_sigmoid(v) : shifted_exp(v, m) / denom; };
    // what is ranked, in fp32: the score, or the key (-inf where it ranks last)
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < NP; ++i) s[i] = s[i] > -INFINITY ? prob(s[i]) + bias[i] : -INFINITY;
    }

    bool sure = true;
    uint32_t open = 0xffffffffu;  // bit i: the lane's expert i lies in a kept group
    if (a.groups > 1) {
      float* const row = reinterpret_cast<float*>(scratch);
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
      const bool in = g < a.groups && better < a.kept;
      const uint32_t kept = __ballot_sync(0xffffffffu, in);
      if (a.kept < a.groups && (a.bias || a.group_top > 1)) {
        const float lo = -warp_max_f(in ? -b1 : -INFINITY), hi = warp_max_f(!in && g < a.groups ? b1 : -INFINITY);
        const float most = warp_max_f(g < a.groups && magnitude < INFINITY ? magnitude : 0.f);
        sure = apart(lo, hi, 2.f * key_error, 4.f * most);
      }
      const float inv_size = 1.f / (float)size;  // (e + 0.5) / size truncates to e / size for e < 4096
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int of = (int)(((float)expert_at(i, lane) + 0.5f) * inv_size);
        if (!((kept >> ((of << share) & 31)) & 1u)) open &= ~(1u << i);
      }
      __syncwarp();
    }

    // the numbers: 0 is no candidate, the index alone is -inf
    if (!whole && !a.bias) {
      float least = INFINITY;
#pragma unroll
      for (int i = 0; i < NP; ++i) least = s[i] > -INFINITY ? fminf(least, s[i]) : least;
      low = fmaxf(-warp_max_f(-least), m - kSpread);
      range = m - low;
    }
    // [low, low + range] to [1 + 2^-16, 2 - 2^-6); what lies below shares the lowest place, what lies above the
    // highest, and a slot that has one of the two is decided again
    const float scale = range > 0.f ? (1.f - 0x1p-5f) / range : 0.f, offset = fmaf(-low, scale, 1.f + 0x1p-16f);
    const float number_error = range * 0x1p-20f;  // of a number, as a key: rounding of the products and the cut
    auto number = [&](int i) -> uint32_t {
      const int e = expert_at(i, lane);
      if (e >= a.E || !(open >> i & 1u)) return 0u;
      uint32_t u = 0u;
      if (whole) u = ordered16<T>(s[i]) << 16;
      else if (s[i] > -INFINITY)
        u = __float_as_uint(fminf(fmaxf(fmaf(s[i], scale, offset), 1.f + 0x1p-17f), 2.f - 0x1p-23f)) << 9 & ~kIndex;
      return u | (kIndex - (uint32_t)e);
    };
    uint32_t b1 = 0u, b2 = 0u;
    auto look = [&](uint32_t below) {
      b1 = b2 = 0u;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint32_t u = number(i);
        u = u < below ? u : 0u;
        b2 = max(b2, min(b1, u));
        b1 = max(b1, u);
      }
    };
    look(0xffffffffu);
    auto round = [&]() {
      const uint32_t best = __reduce_max_sync(0xffffffffu, b1);
      const bool mine = b1 == best;
      if (__any_sync(0xffffffffu, mine && b2 == 0u)) {
        if (mine) look(best);
      } else if (mine) {
        b1 = b2;
        b2 = 0u;
      }
      return best;
    };
    uint32_t won = 0u;
    for (int j = 0; j < a.k; ++j) {
      const uint32_t best = round();
      if (lane == j) won = best;
    }
    int id = (int)(kIndex - (won & kIndex));
    if (!whole) {
      // as keys: the slot's, and the one behind it (the last slot's is the best that is left)
      const uint32_t rest = __reduce_max_sync(0xffffffffu, b1);
      const uint32_t behind = __shfl_down_sync(0xffffffffu, won, 1);
      const uint32_t next = lane + 1 < a.k ? behind : rest;
      // a gap of n steps is a gap of at least (n - 1) range 2^-23 of keys; both keys' errors have to fit
      const float steps = (float)((won >> kShift) - (next >> kShift)) * (1 << (kShift - 9));
      const float size = a.bias ? 2.f * (fabsf(low) + range) : 0.f;
      const float need = 2.f * ((a.bias ? key_error : 0.f) + number_error) + 0x1p-22f * size;
      const bool clear = next == 0u || (next >> kShift == 0u ? won >> kShift != 0u : steps * 0x1p-23f * range > need);
      const bool wild = lane < a.k && (won >> kShift == 0u || won >= ~kIndex);
      if (__any_sync(0xffffffffu, wild) || !(range < INFINITY)) {
        sure = false;
      } else if (__any_sync(0xffffffffu, lane < a.k && !clear)) {
        // all that may belong to the slots, one a lane, ordered by their keys in double
        const uint32_t last = __shfl_sync(0xffffffffu, won, a.k - 1);
        int n = a.k;
        while (n < 32) {
          const uint32_t top = __reduce_max_sync(0xffffffffu, b1);
          const float gap = (float)((last >> kShift) - (top >> kShift)) * (1 << (kShift - 9)) * 0x1p-23f * range;
          if (top >> kShift == 0u || gap > need) break;
          const uint32_t best = round();
          if (lane == n) won = best;
          ++n;
        }
        if (n == 32) {
          sure = false;
        } else {
          const int e = lane < n ? (int)(kIndex - (won & kIndex)) : 0;
          double exact = -INFINITY;
          if (lane < n) {
            const double v = clean_score(z[e]);
            exact = v;
            if (a.bias) {
              exact = a.sigmoid ? 1.0 / (1.0 + exp(-v)) : (v == (double)m ? 1.0 : exp(v - (double)m));
            }
          }
          if (a.bias && !a.sigmoid) {
            double sum = 0.0;
            for (int q = lane; q < a.E; q += 32) {
              const double v = clean_score(z[q]);
              sum += v == (double)m ? 1.0 : exp(v - (double)m);
            }
            sum = warp_sum_d(sum);
            exact = exact / sum;
          }
          if (a.bias && lane < n) exact += (double)a.bias[e];
          int rank = 0;
          for (int o = 0; o < n; ++o) {
            const double u = __shfl_sync(0xffffffffu, exact, o);
            const int eo = __shfl_sync(0xffffffffu, e, o);
            rank += u > exact || (u == exact && eo < e);
          }
          int* const place = reinterpret_cast<int*>(scratch);
          __syncwarp();
          if (lane < n && rank < a.k) place[rank] = e;
          __syncwarp();
          if (lane < a.k) id = place[lane];
          __syncwarp();
        }
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

// Rows of more than 1024 experts: the keys lie in shared memory, in double.
template <class T>
__global__ void __launch_bounds__(32 * kWarps) select_wide_kernel(const SelectArgs a) {
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
// NI > 0: the scores of a softmax over all experts lie in registers, as above;
// NI = 0: any number of experts, read again from cache.
template <class T, int NI, bool VEC>
__global__ void __launch_bounds__(32 * kBwdWarps) select_bwd_kernel(const SelectArgs a) {
  constexpr int NR = NI ? NI : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kBwdWarps + warp;
  if (t >= a.Q) return;
  const T* z = static_cast<const T*>(a.scores) + t * a.ld;
  T* dz = static_cast<T*>(a.grad) + (int64_t)t * a.E;
  const bool softmax_all = !a.sigmoid && !a.renorm;  // the gradient reaches every expert
  Four<T> raw[NR];
  if (NI > 0 && softmax_all) fetch_scores<T, NR, VEC>(z, a.E, lane, raw);

  int id = -1;
  float g = 0.f, v = -INFINITY;
  if (lane < a.k) {
    const int64_t wide = a.ids_in[(int64_t)t * a.k + lane];
    g = a.grad_route[(int64_t)t * a.k + lane] * a.scale;
    if (wide >= 0 && wide < a.E) {  // any other id contributes nothing
      id = (int)wide;
      v = clean_score(z[id]);
    } else {
      g = 0.f;
    }
  }
  float s[4 * NR];
  float d = 0.f, m = -INFINITY, every = 0.f;  // d: the slot's share of the gradient
  if (a.renorm) {
    float total;
    const float q = slot_share(v, a.sigmoid, &total);
    const float share = total > 0.f ? q / total : 0.f;
    const float mean = row_warp_sum(g * share);
    d = share * (g - mean);
  } else if (a.sigmoid) {
    d = v > -INFINITY ? g / (1.f + expf(-v)) : 0.f;
  } else {
    float denom = 0.f;
    if (NI > 0) {
      take_scores<T, NR>(raw, a.E, lane, s);
#pragma unroll
      for (int i = 0; i < 4 * NR; ++i) m = fmaxf(m, s[i]);
      m = warp_max_f(m);
#pragma unroll
      for (int i = 0; i < 4 * NR; ++i) {
        s[i] = s[i] > -INFINITY ? shifted_exp(s[i], m) : 0.f;
        denom += s[i];
      }
    } else {
      for (int e = lane; e < a.E; e += 32) m = fmaxf(m, clean_score(z[e]));
      m = warp_max_f(m);
      for (int e = lane; e < a.E; e += 32) denom += shifted_exp(clean_score(z[e]), m);
    }
    const float mine = v > -INFINITY ? g * shifted_exp(v, m) : 0.f;
    denom = row_warp_sum(denom);
    const float base = row_warp_sum(mine);
    const float inv = m > -INFINITY ? 1.f / denom : 0.f;
    d = mine * inv;
    every = -base * inv * inv;  // an expert's gradient over exp(s - m), without its own slots
  }
  if (a.sigmoid && v > -INFINITY) d *= 1.f / (1.f + expf(v));
  if (NI > 0) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int e = 128 * i + 4 * lane;
      Four<T> out;
#pragma unroll
      for (int j = 0; j < 4; ++j) out.v[j] = Elem<T>::from(softmax_all ? every * s[4 * i + j] : 0.f);
      if (VEC) {
        if (e < a.E) *reinterpret_cast<Four<T>*>(dz + e) = out;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e + j < a.E) dz[e + j] = out.v[j];
      }
    }
  } else {
    for (int e = lane; e < a.E; e += 32)
      dz[e] = Elem<T>::from(softmax_all && m > -INFINITY ? every * shifted_exp(clean_score(z[e]), m) : 0.f);
  }
  // slots of one expert are added by the first of them
  bool first = id >= 0;
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  if (__any_sync(0xffffffffu, id >= 0 && (same & (same - 1)))) {
    float sum = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const float part = __shfl_sync(0xffffffffu, d, j);
      if (same >> j & 1u) sum += part;
    }
    d = sum;
    first = first && lane == __ffs(same) - 1;
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

struct SelectShape {
  int blocks, warps, smem;
};

// As many warps a block as keep the SMs evenly busy, at most kWarps and 96 KB
// of scratch; two blocks an SM walk over the tokens.
SelectShape select_shape(const SelectArgs& a, int sms) {
  const int row = a.E * (int)sizeof(uint64_t);
  int warps = (a.Q + 2 * sms - 1) / (2 * sms);
  if (warps > 96 * 1024 / row) warps = 96 * 1024 / row;
  if (warps > kWarps) warps = kWarps;
  const int need = (a.Q + warps - 1) / warps;
  return {need < 2 * sms ? need : 2 * sms, warps, warps * row + (a.counts ? a.E * (int)sizeof(int) : 0)};
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
  kernel<<<s.blocks, 32 * s.warps, s.smem, st>>>(a);
  return cudaGetLastError();
}

template <class T, int NI, bool VEC>
cudaError_t start_select(const SelectArgs& a, const SelectShape& s, cudaStream_t st) {
  static std::atomic<unsigned long long> opted{0};
  return start(select_kernel<T, NI, VEC>, opted, a, s, st);
}

template <class T, int NI>
cudaError_t launch_select(const SelectArgs& a, const SelectShape& s, cudaStream_t st) {
  return four_aligned<T>(a.scores, a.ld, a.E) ? start_select<T, NI, true>(a, s, st) : start_select<T, NI, false>(a, s, st);
}

template <class T>
cudaError_t run_select(const SelectArgs& a, int sms, cudaStream_t st) {
  const SelectShape s = select_shape(a, sms);
  if (a.E <= 128) return launch_select<T, 1>(a, s, st);
  if (a.E <= 256) return launch_select<T, 2>(a, s, st);
  if (a.E <= 384) return launch_select<T, 3>(a, s, st);
  if (a.E <= 512) return launch_select<T, 4>(a, s, st);
  if (a.E <= 1024) return launch_select<T, 8>(a, s, st);
  static std::atomic<unsigned long long> opted{0};
  return start(select_wide_kernel<T>, opted, a, s, st);
}

template <class T, int NI>
void launch_bwd(const SelectArgs& a, cudaStream_t st) {
  const int blocks = (a.Q + kBwdWarps - 1) / kBwdWarps;
  if (four_aligned<T>(a.scores, a.ld, a.E) && four_aligned<T>(a.grad, a.E, a.E))
    select_bwd_kernel<T, NI, true><<<blocks, 32 * kBwdWarps, 0, st>>>(a);
  else
    select_bwd_kernel<T, NI, false><<<blocks, 32 * kBwdWarps, 0, st>>>(a);
}

template <class T>
cudaError_t run_bwd(const SelectArgs& a, cudaStream_t st) {
  if (a.E <= 128) launch_bwd<T, 1>(a, st);
  else if (a.E <= 256) launch_bwd<T, 2>(a, st);
  else if (a.E <= 384) launch_bwd<T, 3>(a, st);
  else if (a.E <= 512) launch_bwd<T, 4>(a, st);
  else if (a.E <= 1024) launch_bwd<T, 8>(a, st);
  else select_bwd_kernel<T, 0, false><<<(a.Q + kBwdWarps - 1) / kBwdWarps, 32 * kBwdWarps, 0, st>>>(a);
  return cudaGetLastError();
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
  return qlen >= 0 && ld >= c->experts && ld <= kMaxPitch && (qlen == 0 || scores);
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
  if (counts && cudaMemsetAsync(counts, 0, (size_t)a.E * sizeof(int32_t), st) != cudaSuccess) return RAWINT4_CUDA_ERROR;
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
  if (cfg->type == RAWINT4_TYPE_F32) err = run_bwd<float>(a, st);
  else if (cfg->type == RAWINT4_TYPE_BF16) err = run_bwd<__nv_bfloat16>(a, st);
  else err = run_bwd<__half>(a, st);
  return err == cudaSuccess ? RAWINT4_OK : RAWINT4_CUDA_ERROR;
}

}  // extern "C"
