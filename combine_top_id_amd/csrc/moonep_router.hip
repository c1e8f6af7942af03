// The router in front of the plan: scores of the experts, the K chosen ones and their weights,
// and the gradient of the logits.
//
//   s = softmax(l) or sigmoid(l);  key = s + bias;  ids = the K largest keys of the best groups
//   w = scale * s[ids], or scale * s[ids] / sum(s[ids])
//
// L lanes of a wave hold a token's logits, expert v * L + lane in register v, and everything between
// them is moves between lanes.
#include <cmath>

#include "moonep_internal.h"

namespace moonep {
namespace {

constexpr int kMaxGroups = MOONEP_MAX_GROUPS;

struct RouterArgs {
  const void* logits;
  const float* bias;
  int64_t T;
  int E, K, groups, top_groups;
  float scale;
  const int32_t* ids_in;
  const float* g_w;
  int32_t* ids;
  float* w;
  void* g;
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}

// The value of a partner lane in step STEP of a reduction over 2, 4, 8 ... 64 lanes: every lane of a
// group that already agrees has a lane of the other half as its partner.
template <int STEP>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
#ifdef __HIP_DEVICE_COMPILE__
  if constexpr (STEP == 0) return dpp<0xB1>(v);       // lane ^ 1
  if constexpr (STEP == 1) return dpp<0x4E>(v);       // lane ^ 2
  if constexpr (STEP == 2) return dpp<0x141>(v);      // mirrored in 8
  if constexpr (STEP == 3) return dpp<0x140>(v);      // mirrored in 16
  const bool odd = STEP == 4 ? threadIdx.x & 16 : threadIdx.x & 32;
  const auto p = STEP == 4 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return odd ? p[0] : p[1];
#else
  return v;
#endif
}
template <int STEP>
__device__ __forceinline__ float partner(float v) { return __uint_as_float(partner<STEP>(__float_as_uint(v))); }
template <int STEP>
__device__ __forceinline__ int partner(int v) { return (int)partner<STEP>((uint32_t)v); }
template <int STEP>
__device__ __forceinline__ uint64_t partner(uint64_t v) {
  return (uint64_t)partner<STEP>((uint32_t)(v >> 32)) << 32 | partner<STEP>((uint32_t)v);
}

// op over the L lanes of a token, in each of them; the order is fixed and the same in all.
template <int L, int STEP = 0, class T, class F>
__device__ __forceinline__ T over(T v, F op) {
  if constexpr ((1 << STEP) < L) return over<L, STEP + 1>(op(v, partner<STEP>(v)), op);
  return v;
}
template <int L, class T>
__device__ __forceinline__ T most(T v) { return over<L>(v, [](T a, T b) { return a > b ? a : b; }); }
template <int L, class T>
__device__ __forceinline__ T least(T v) { return over<L>(v, [](T a, T b) { return a < b ? a : b; }); }
template <int L>
__device__ __forceinline__ float sum(float v) { return over<L>(v, [](float a, float b) { return a + b; }); }

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// A logit as it counts: NaN as -inf (an expert that is masked), +inf as the largest number.
__device__ __forceinline__ float clean(float l) {
  return l != l ? -INFINITY : fminf(l, 3.402823466e38f);
}

// Integers in the order of the numbers.  0 is for experts that cannot be chosen (any more), 1 for those
// that are masked, which come after all others.
__device__ __forceinline__ uint64_t order(double v) {
  if (!(v > -INFINITY)) return 1;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);         // -0 is 0
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double number(uint64_t k) {
  if (k <= 1) return -INFINITY;
  return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k));
}

constexpr int kSoftmax = MOONEP_SCORE_SOFTMAX, kSigmoid = MOONEP_SCORE_SIGMOID;

template <class T, int SCORE, bool NORM, int L, int V>
__global__ __launch_bounds__(256) void router_kernel(const RouterArgs a) {
  constexpr int kTokens = 256 / L;             // of a workgroup
  constexpr int kGV = kMaxGroups / L > 0 ? (kMaxGroups + L - 1) / L : 1;
  constexpr int kKV = (MOONEP_MAX_K + L - 1) / L;
  __shared__ uint64_t held[kTokens][V * L];    // the keys, for the groups' sake
  const int sub = threadIdx.x % L, mine = threadIdx.x / L;
  for (int64_t first = (int64_t)blockIdx.x * kTokens; first < a.T; first += (int64_t)gridDim.x * kTokens) {
    const int64_t t = min(first + mine, a.T - 1);          // the last token again, where there is none
    const bool there = first + mine < a.T;
    const T* row = static_cast<const T*>(a.logits) + t * a.E;
    float l[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + sub;
      l[v] = e < a.E ? clean(load_logit(row + e)) : -INFINITY;
    }
    float top = 0.f, total = 1.f;                          // softmax: of the whole row
    if constexpr (SCORE == kSoftmax) {
      top = l[0];
#pragma unroll
      for (int v = 1; v < V; ++v) top = fmaxf(top, l[v]);
      top = most<L>(top);
      if constexpr (!NORM) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) s += l[v] > -INFINITY ? expf(l[v] - top) : 0.f;
        total = sum<L>(s);
      }
    }
    uint64_t key[V];
    const bool plain = !a.bias && a.groups == 1;           // the logits' order is the scores'
    if (plain) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = v * L + sub < a.E ? order((double)l[v]) : 0;
    } else {
      // scores that differ little are told apart in 64 bits
      double whole = 1.0;
      if constexpr (SCORE == kSoftmax) {
        double s = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) s += l[v] > -INFINITY ? exp((double)l[v] - (double)top) : 0.0;
        whole = __longlong_as_double((long long)over<L>((uint64_t)__double_as_longlong(s), [](uint64_t x, uint64_t y) {
          return (uint64_t)__double_as_longlong(__longlong_as_double((long long)x) + __longlong_as_double((long long)y));
        }));
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * L + sub;
        double s = SCORE == kSoftmax ? exp((double)l[v] - (double)top) / whole : 1.0 / (1.0 + exp(-(double)l[v]));
        if (a.bias) s += (double)(e < a.E ? a.bias[e] : 0.f);
        key[v] = e < a.E ? order(l[v] > -INFINITY ? s : -INFINITY) : 0;
      }
    }
    if (a.groups > 1) {
      const int gs = a.E / a.groups;
      const uint32_t magic = ((1u << 20) + gs - 1) / gs;   // e / gs for e < 1024 and gs <= 512
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) held[mine][v * L + sub] = key[v];
      __syncthreads();
      uint64_t score[kGV];
#pragma unroll
      for (int j = 0; j < kGV; ++j) {
        const int g = j * L + sub;
        uint64_t m1 = 1, m2 = 1;
        for (int i = 0; g < a.groups && i < gs; ++i) {
          const uint64_t k = held[mine][g * gs + i];
          m2 = max(m2, min(m1, k));
          m1 = max(m1, k);
        }
        // two keys that are not masked, or as many as there are
        score[j] = g < a.groups ? order(number(m1) + (m2 > 1 ? number(m2) : 0.0)) : 0;
      }
      uint64_t chosen = 0;
      for (int n = 0; n < a.top_groups; ++n) {
        uint64_t m = 0;
#pragma unroll
        for (int j = 0; j < kGV; ++j) m = max(m, score[j]);
        m = most<L>(m);
        int g = 1 << 20;
#pragma unroll
        for (int j = kGV - 1; j >= 0; --j) g = score[j] == m ? j * L + sub : g;
        g = least<L>(g);
        chosen |= 1ull << g;
#pragma unroll
        for (int j = 0; j < kGV; ++j) score[j] = g == j * L + sub ? 0 : score[j];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * L + sub;
        if (!(chosen >> (e * magic >> 20 & 63) & 1)) key[v] = 0;
      }
    }
    int id[kKV];
#pragma unroll
    for (int j = 0; j < kKV; ++j) id[j] = 0;
    for (int k = 0; k < a.K; ++k) {
      uint64_t m = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = max(m, key[v]);
      m = most<L>(m);
      int e = 1 << 20;
#pragma unroll
      for (int v = V - 1; v >= 0; --v) e = key[v] == m ? v * L + sub : e;
      e = least<L>(e);
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = e == v * L + sub ? 0 : key[v];
#pragma unroll
      for (int j = 0; j < kKV; ++j) id[j] = k == j * L + sub ? e : id[j];
    }
    // lane k has the k-th
    float x[kKV], m = -INFINITY, w[kKV], s = 0.f;
#pragma unroll
    for (int j = 0; j < kKV; ++j) {
      x[j] = j * L + sub < a.K ? clean(load_logit(row + id[j])) : -INFINITY;
      m = fmaxf(m, SCORE == kSigmoid ? fminf(x[j], 0.f) : x[j]);
    }
    // normalised: of the scores' ratios, so that scores too small for fp32 still have them
    m = NORM ? most<L>(m) : SCORE == kSigmoid ? 0.f : top;
#pragma unroll
    for (int j = 0; j < kKV; ++j) {
      if constexpr (SCORE == kSigmoid) w[j] = expf(fminf(x[j], 0.f) - m) / (1.f + expf(-fabsf(x[j])));
      else w[j] = expf(x[j] - m) / total;
      w[j] = x[j] > -INFINITY ? w[j] : 0.f;
      s += w[j];
    }
    if constexpr (NORM) {
      s = sum<L>(s);
      s = s > 0.f ? a.scale / s : 0.f;
    } else {
      s = a.scale;
    }
#pragma unroll
    for (int j = 0; j < kKV; ++j)
      if (there && j * L + sub < a.K) {
        a.ids[t * a.K + j * L + sub] = id[j];
        a.w[t * a.K + j * L + sub] = w[j] * s;
      }
  }
}

// The chosen logits' gradients, from the weights':
//   normalised, p = s / sum(s):  scale p (g - sum(g p)), times 1 - s for the sigmoid;
//   else sigmoid: scale g s (1 - s);  softmax: scale s (g - sum(g s)), and -scale s sum(g s) for
//   every logit that was not chosen.
template <class T, int SCORE, bool NORM, int L, int V>
__global__ __launch_bounds__(256) void router_bwd_kernel(const RouterArgs a) {
  constexpr int kTokens = 256 / L;
  constexpr int kKV = (MOONEP_MAX_K + L - 1) / L;
  constexpr bool kDense = SCORE == kSoftmax && !NORM;
  __shared__ float held[kTokens][V * L];       // of each expert, what its choice brings
  const int sub = threadIdx.x % L, mine = threadIdx.x / L;
  for (int64_t first = (int64_t)blockIdx.x * kTokens; first < a.T; first += (int64_t)gridDim.x * kTokens) {
    const int64_t t = min(first + mine, a.T - 1);
    const bool there = first + mine < a.T;
    const T* row = static_cast<const T*>(a.logits) + t * a.E;
    float l[kDense ? V : 1], top = -INFINITY, total = 1.f;
    if constexpr (kDense) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * L + sub;
        l[v] = e < a.E ? clean(load_logit(row + e)) : -INFINITY;
        top = fmaxf(top, l[v]);
      }
      top = most<L>(top);
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        l[v] = l[v] > -INFINITY ? expf(l[v] - top) : 0.f;
        s += l[v];
      }
      total = sum<L>(s);
    }
    int id[kKV];
    float x[kKV], g[kKV], m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kKV; ++j) {
      const int k = j * L + sub;
      id[j] = k < a.K ? a.ids_in[t * a.K + k] : -1;
      const bool in = (unsigned)id[j] < (unsigned)a.E;
      if (!in) id[j] = -1;
      g[j] = in ? a.g_w[t * a.K + k] * a.scale : 0.f;
      x[j] = in ? clean(load_logit(row + id[j])) : -INFINITY;
      if (x[j] == -INFINITY) g[j] = 0.f;                   // masked: a score of zero, whatever its logit
      m = fmaxf(m, SCORE == kSigmoid ? fminf(x[j], 0.f) : x[j]);
    }
    m = NORM ? most<L>(m) : SCORE == kSigmoid ? 0.f : top;
    float p[kKV], rest[kKV], s = 0.f;
#pragma unroll
    for (int j = 0; j < kKV; ++j) {
      const float z = 1.f / (1.f + expf(-fabsf(x[j])));    // sigmoid of |x|
      if constexpr (SCORE == kSigmoid) p[j] = expf(fminf(x[j], 0.f) - m) * z;
      else p[j] = expf(x[j] - m) / total;
      p[j] = x[j] > -INFINITY ? p[j] : 0.f;
      // 1 - s, without the difference where s is near one
      rest[j] = SCORE == kSoftmax ? 1.f : x[j] > 0.f ? expf(-x[j]) * z : z;
      s += p[j];
    }
    if constexpr (NORM) {
      s = sum<L>(s);
      s = s > 0.f ? 1.f / s : 0.f;
    } else {
      s = 1.f;
    }
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < kKV; ++j) {
      p[j] *= s;
      dot += g[j] * p[j];
    }
    dot = SCORE == kSigmoid && !NORM ? 0.f : sum<L>(dot);
    float d[kKV];
#pragma unroll
    for (int j = 0; j < kKV; ++j) d[j] = kDense ? p[j] * g[j] : p[j] * (g[j] - dot) * rest[j];
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) held[mine][v * L + sub] = 0.f;
    __syncthreads();
    for (int k = 0; k < a.K; ++k) {                        // in turn: an expert may be named twice
#pragma unroll
      for (int j = 0; j < kKV; ++j)
        if (k == j * L + sub && id[j] >= 0) held[mine][id[j]] += d[j];
    }
    __syncthreads();
    T* out = static_cast<T*>(a.g) + t * a.E;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + sub;
      float r = held[mine][e];
      if constexpr (kDense) r -= total > 0.f ? l[v] / total * dot : 0.f;
      if (there && e < a.E) store_logit(out + e, r);
    }
  }
}

template <class T, int SCORE, bool NORM, bool BWD, int L, int V>
void launch_as(const RouterArgs& a, hipStream_t st) {
  constexpr int kTokens = 256 / L;
  const unsigned grid = (unsigned)std::min<int64_t>((a.T + kTokens - 1) / kTokens, 1 << 23);
  if constexpr (BWD) hipLaunchKernelGGL((router_bwd_kernel<T, SCORE, NORM, L, V>), dim3(grid), dim3(256), 0, st, a);
  else hipLaunchKernelGGL((router_kernel<T, SCORE, NORM, L, V>), dim3(grid), dim3(256), 0, st, a);
}

template <class T, int SCORE, bool NORM, bool BWD>
void launch_sized(const RouterArgs& a, hipStream_t st) {
  if (a.E <= 64) launch_as<T, SCORE, NORM, BWD, 16, 4>(a, st);
  else if (a.E <= 256) launch_as<T, SCORE, NORM, BWD, 16, 16>(a, st);
  else if (a.E <= 384) launch_as<T, SCORE, NORM, BWD, 16, 24>(a, st);
  else launch_as<T, SCORE, NORM, BWD, 64, 16>(a, st);
}

template <bool BWD>
int launch(const RouterArgs& a, int dtype, int score, bool norm, hipStream_t st) {
  (void)hipGetLastError();
  auto of = [&](auto t) {
    using T = decltype(t);
    if (score == kSoftmax) norm ? launch_sized<T, kSoftmax, true, BWD>(a, st) : launch_sized<T, kSoftmax, false, BWD>(a, st);
    else norm ? launch_sized<T, kSigmoid, true, BWD>(a, st) : launch_sized<T, kSigmoid, false, BWD>(a, st);
  };
  if (dtype == MOONEP_F32) of(float{}); else of(uint16_t{});
  return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check_router(int dtype, int64_t T, int E, int K, int score, int normalize, float scale) {
  if ((dtype != MOONEP_F32 && dtype != MOONEP_BF16) || (score != kSoftmax && score != kSigmoid) ||
      (normalize != 0 && normalize != 1) || T < 0 || E < 1 || K < 1 || K > E || !std::isfinite(scale))
    return MOONEP_EINVAL;
  if (E > MOONEP_MAX_E || K > MOONEP_MAX_K || T > INT32_MAX) return MOONEP_ELIMIT;
  return MOONEP_OK;
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" {

int moonep_router(const void* logits, int dtype, const float* bias, int64_t T, int E, int K, int score, int groups,
                  int top_groups, int normalize, float scale, int32_t* topk_ids, float* topk_w, hipStream_t stream) {
  const int rc = check_router(dtype, T, E, K, score, normalize, scale);
  if (rc != MOONEP_OK) return rc;
  if (groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups ||
      (int64_t)top_groups * (E / groups) < K)
    return MOONEP_EINVAL;
  if (groups > kMaxGroups) return MOONEP_ELIMIT;
  if (T == 0) return MOONEP_OK;
  if (!logits || !topk_ids || !topk_w) return MOONEP_EINVAL;
  const int size = dtype == MOONEP_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4)) return MOONEP_EALIGN;
  const Span ls = span(logits, T, (int64_t)E * size), bs = span(bias, 1, 4ll * E), is = span(topk_ids, T, 4ll * K),
             ws = span(topk_w, T, 4ll * K);
  if (overlap(is, {ls, bs, ws}) || overlap(ws, {ls, bs})) return MOONEP_EINVAL;
  RouterArgs a{};
  a.logits = logits; a.bias = bias;
  a.T = T; a.E = E; a.K = K; a.scale = scale;
  a.groups = top_groups == groups ? 1 : groups;        // all groups: no choice of them
  a.top_groups = top_groups;
  a.ids = topk_ids; a.w = topk_w;
  return launch<false>(a, dtype, score, normalize, stream);
}

int moonep_router_bwd(const void* logits, int dtype, const int32_t* topk_ids, const float* g_w, int64_t T, int E, int K,
                      int score, int normalize, float scale, void* g_logits, hipStream_t stream) {
  const int rc = check_router(dtype, T, E, K, score, normalize, scale);
  if (rc != MOONEP_OK) return rc;
  if (T == 0) return MOONEP_OK;
  if (!logits || !topk_ids || !g_w || !g_logits) return MOONEP_EINVAL;
  const int size = dtype == MOONEP_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(topk_ids, 4) || !aligned(g_w, 4) || !aligned(g_logits, size)) return MOONEP_EALIGN;
  const Span ls = span(logits, T, (int64_t)E * size), is = span(topk_ids, T, 4ll * K), ws = span(g_w, T, 4ll * K),
             os = span(g_logits, T, (int64_t)E * size);
  if (overlap(os, {ls, is, ws})) return MOONEP_EINVAL;
  RouterArgs a{};
  a.logits = logits;
  a.T = T; a.E = E; a.K = K; a.scale = scale;
  a.ids_in = topk_ids; a.g_w = g_w; a.g = g_logits;
  return launch<true>(a, dtype, score, normalize, stream);
}

}  // extern "C"
