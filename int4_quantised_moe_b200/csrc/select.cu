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
// rounds p + bias: the keys are compared in double. Without a bias p grows
// with s and the scores themselves are compared.
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

constexpr int kWarps = 4;  // tokens per block (one warp each) at most

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

__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
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

__device__ __forceinline__ double sigmoid_d(double s) { return 1.0 / (1.0 + exp(-s)); }

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

template <class T>
__global__ void __launch_bounds__(32 * kWarps) select_kernel(const SelectArgs a) {
  extern __shared__ uint64_t keys[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.Q) return;
  uint64_t* key = keys + (size_t)warp * a.E;
  const T* z = static_cast<const T*>(a.scores) + t * a.ld;

  // softmax: largest score and sum of exponents
  double m = 0.0, denom = 1.0;
  if (!a.sigmoid && (a.bias || !a.renorm || a.group_top > 1)) {
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
    return a.sigmoid ? sigmoid_d(s) : (s == m ? 1.0 : exp(s - m)) / denom;
  };
  for (int e = lane; e < a.E; e += 32) {
    const double s = clean_score(z[e]);
    double v = s;
    if (a.bias && s > -INFINITY) v = prob(s) + (double)a.bias[e];
    key[e] = ordered(v);
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

  const float s = lane < a.k ? clean_score(z[id]) : -INFINITY;
  float w;
  if (a.renorm) {
    float total;
    const float q = slot_share(s, a.sigmoid, &total);
    w = total > 0.f ? a.scale * (q / total) : 0.f;
  } else {
    w = a.scale * (float)prob((double)s);
  }
  if (lane < a.k) {
    a.ids[(int64_t)t * a.k + lane] = id;
    a.weights[(int64_t)t * a.k + lane] = w;
    if (a.counts) atomicAdd(a.counts + id, 1);
  }
}

template <class T>
__global__ void __launch_bounds__(32 * kWarps) select_bwd_kernel(const SelectArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= a.Q) return;
  const T* z = static_cast<const T*>(a.scores) + t * a.ld;
  T* dz = static_cast<T*>(a.grad) + (int64_t)t * a.E;
  int64_t id = -1;
  float g = 0.f, s = -INFINITY;
  if (lane < a.k) {
    id = a.ids_in[(int64_t)t * a.k + lane];
    if (id < 0 || id >= a.E) id = -1;  // that slot contributes nothing
    if (id >= 0) {
      g = a.grad_route[(int64_t)t * a.k + lane] * a.scale;
      s = clean_score(z[id]);
    }
  }
  float d = 0.f, base = 0.f, m = 0.f, denom = 1.f;  // the slot's share of the gradient
  if (a.renorm) {
    float total;
    const float q = slot_share(s, a.sigmoid, &total);
    const float share = total > 0.f ? q / total : 0.f;
    const float mean = row_warp_sum(g * share);
    d = share * (g - mean);
  } else if (a.sigmoid) {
    d = s > -INFINITY ? g / (1.f + expf(-s)) : 0.f;
  } else {
    m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, clean_score(z[e]));
    m = warp_max_f(m);
    denom = 0.f;
    for (int e = lane; e < a.E; e += 32) denom += shifted_exp(clean_score(z[e]), m);
    denom = row_warp_sum(denom);
    d = s > -INFINITY ? g * (shifted_exp(s, m) / denom) : 0.f;
    base = row_warp_sum(d);
  }
  if (a.sigmoid && s > -INFINITY) d *= 1.f / (1.f + expf(s));
  const bool dense = !a.sigmoid && !a.renorm && m > -INFINITY;
  for (int e = lane; e < a.E; e += 32)
    dz[e] = Elem<T>::from(dense ? -base * (shifted_exp(clean_score(z[e]), m) / denom) : 0.f);
  // slots of one expert are added by the first of them
  float sum = 0.f;
  bool first = id >= 0;
  for (int j = 0; j < a.k; ++j) {
    const int64_t other = __shfl_sync(0xffffffffu, id, j);
    const float v = __shfl_sync(0xffffffffu, d, j);
    if (other == id) {
      sum += v;
      if (j < lane) first = false;
    }
  }
  if (dense && id >= 0) sum -= base * (shifted_exp(s, m) / denom);
  __syncwarp();
  if (first && lane < a.k) dz[id] = Elem<T>::from(sum);
}

template <class T>
cudaError_t run_select(const SelectArgs& a, cudaStream_t st) {
  int warps = (int)(48 * 1024 / (sizeof(uint64_t) * a.E));
  warps = warps < 1 ? 1 : warps > kWarps ? kWarps : warps;
  select_kernel<T><<<(a.Q + warps - 1) / warps, 32 * warps, warps * a.E * sizeof(uint64_t), st>>>(a);
  return cudaGetLastError();
}

template <class T>
cudaError_t run_bwd(const SelectArgs& a, cudaStream_t st) {
  select_bwd_kernel<T><<<(a.Q + kWarps - 1) / kWarps, 32 * kWarps, 0, st>>>(a);
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
  if (cfg->type == RAWINT4_TYPE_F32) err = run_select<float>(a, st);
  else if (cfg->type == RAWINT4_TYPE_BF16) err = run_select<__nv_bfloat16>(a, st);
  else err = run_select<__half>(a, st);
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
