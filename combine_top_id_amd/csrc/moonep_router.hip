// The router in front of the plan: scores of the experts, the K chosen ones and their weights,
// and the gradient of the logits.
//
//   s = softmax(l) or sigmoid(l);  key = s + bias;  ids = the K largest keys of the best groups
//   w = scale * s[ids], or scale * s[ids] / sum(s[ids])
//
// L lanes of a wave hold a token's logits, expert v * L + lane in register v, and everything between
// them is moves between lanes.
#include <cmath>
#include <type_traits>

#include "moonep_internal.h"

namespace moonep {
namespace {

constexpr int kMaxGroups = MOONEP_MAX_GROUPS;
constexpr int64_t kWgs = 1 << 23;          // of a grid, at most

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

constexpr float kLargest = 3.402823466e38f;      // number in fp32

// A logit as it counts: NaN as -inf (an expert that is masked), +inf as the largest number, -0 as 0.
__device__ __forceinline__ float clean(float l) {
  l += 0.f;
  return l == l ? fminf(l, kLargest) : -INFINITY;
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

// The same of a float.  -inf, which masked experts have, is the smallest, and none is 0.
__device__ __forceinline__ uint32_t order(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (uint32_t)((int)b >> 31 | (int)0x80000000);
}
__device__ __forceinline__ float number(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); }
// Without its last five bits, where register v stands instead: 31 - v, so that the order of equal numbers
// is that of the experts of a lane.
__device__ __forceinline__ uint32_t short_key(float x, int v) { return (order(x) & ~31u) | (uint32_t)(31 - v); }
constexpr uint32_t kMasked32 = 0x007FFFFFu;      // of -inf, and the largest short key of one

__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t c) {
  return max(min(a, b), min(max(a, b), c));
}

// What the choice goes by: logits alone, scores and biases, or these in groups.
enum Mode { kPlain, kBiased, kGrouped };

constexpr int kSoftmax = MOONEP_SCORE_SOFTMAX, kSigmoid = MOONEP_SCORE_SIGMOID;

// Sum over the L lanes, of doubles.
template <int L>
__device__ __forceinline__ double sum64(double v) {
  return __longlong_as_double((long long)over<L>((uint64_t)__double_as_longlong(v), [](uint64_t x, uint64_t y) {
    return (uint64_t)__double_as_longlong(__longlong_as_double((long long)x) + __longlong_as_double((long long)y));
  }));
}

// The best groups, as bits.  `held` has a token's keys; top two of each group, then the groups in turn.  `close` is set
// where two scores that the choice depends on are no further apart than gap(score).
template <int L, class K, class Number, class Order, class Gap>
__device__ __forceinline__ uint64_t best_groups(const K* held, int sub, int E, int groups, int top_groups, K masked, Number number,
                                                Order order, Gap gap, bool& close) {
  constexpr int kGV = (kMaxGroups + L - 1) / L;
  const int gs = E / groups;
  // lanes to a group: a power of two, more than one where there are few groups
  int shift = 0;
  while ((2 << shift) * groups <= L) ++shift;
  const int part = sub & ((1 << shift) - 1);
  K score[kGV];
#pragma unroll
  for (int j = 0; j < kGV; ++j) {
    const int g = (j * L + sub) >> shift;
    K m1 = masked, m2 = masked;
    if (g < groups) {
      const int n = (gs - part + (1 << shift) - 1) >> shift;          // of this lane's, from a place of its own on
      int i = n ? sub % n : 0;
      for (int c = 0; c < n; ++c) {
        const K k = held[g * gs + part + (i << shift)];
        m2 = max(m2, min(m1, k));
        m1 = max(m1, k);
        if (++i == n) i = 0;
      }
    }
    auto merge = [&](K o1, K o2) {
      m2 = max(max(m2, o2), min(m1, o1));
      m1 = max(m1, o1);
    };
    if (j == 0) {                                  // more than one lane to a group: all groups are in j = 0
      if (shift > 0) merge(partner<0>(m1), partner<0>(m2));
      if (shift > 1) merge(partner<1>(m1), partner<1>(m2));
      if (shift > 2) merge(partner<2>(m1), partner<2>(m2));
      if (shift > 3) merge(partner<3>(m1), partner<3>(m2));
      if constexpr (L > 16) {
        if (shift > 4) merge(partner<4>(m1), partner<4>(m2));
      }
    }
    // two keys that are not masked, or as many as there are
    const K two = m1 > masked ? order(number(m1) + (m2 > masked ? number(m2) : 0)) : masked;
    score[j] = g < groups && part == 0 && (j == 0 || shift == 0) ? two : 0;
  }
  uint64_t chosen = 0;
  K last = 0;
  for (int n = 0; n <= top_groups && n < groups; ++n) {
    K m = 0;
#pragma unroll
    for (int j = 0; j < kGV; ++j) m = max(m, score[j]);
    m = most<L>(m);
    // the last that is kept and the first that is not
    if (n == top_groups) {
      close = m > masked && !(number(last) - number(m) > gap(number(last)));
      break;
    }
    last = m;
    int g = 1 << 20;
#pragma unroll
    for (int j = kGV - 1; j >= 0; --j) g = score[j] == m ? (j * L + sub) >> shift : g;
    g = least<L>(g);
    chosen |= 1ull << g;
#pragma unroll
    for (int j = 0; j < kGV; ++j) score[j] = g == (j * L + sub) >> shift ? 0 : score[j];
  }
  return chosen;
}

// LDS of a wave: its tokens' short keys, where there are groups, or one token's keys in 64 bits.
__host__ __device__ constexpr int held_bytes(int E, int L, int groups) {
  const int tokens = groups > 1 ? 64 / L : 1;
  return (E * (tokens > 1 ? tokens * 4 : 8) + 15) / 16 * 16;
}

// A token's choice by keys in 64 bits, by a whole wave: lane k has the k-th.  Its loops are not unrolled: with ordinary
// fp32 logits it is needed so rarely that a wave waits for each line of its code to come from memory.
template <class T, int SCORE, int MODE>
__device__ __forceinline__ int exact_choice(const RouterArgs& a, int64_t t, uint64_t* held) {
  constexpr bool plain = MODE == kPlain;
  const int lane = threadIdx.x & 63;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  double top = 0.0, whole = 1.0;
  if (SCORE == kSoftmax && !plain) {
    float m = -INFINITY;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) m = fmaxf(m, clean(load_logit(row + e)));
    top = (double)most<64>(m);
    whole = 0.0;
  }
  wave_sync();
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const double l = (double)clean(load_logit(row + e));
    double s = l;
    if (!plain) {
      s = exp(SCORE == kSoftmax ? l - top : -l);
      if (SCORE == kSoftmax) whole += l > -INFINITY ? s : 0.0;
      else s = 1.0 / (1.0 + s);
    }
    held[e] = (uint64_t)__double_as_longlong(s);
  }
  if (SCORE == kSoftmax && !plain) whole = sum64<64>(whole);
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    double s = __longlong_as_double((long long)held[e]);
    if (SCORE == kSoftmax && !plain) s /= whole;
    if (a.bias) s += (double)a.bias[e];
    held[e] = order(clean(load_logit(row + e)) > -INFINITY ? s : -INFINITY);
  }
  wave_sync();
  if constexpr (MODE == kGrouped) {
    bool none;
    const uint64_t chosen = best_groups<64>(held, lane, a.E, a.groups, a.top_groups, (uint64_t)1,
                                            [](uint64_t k) { return number(k); }, [](double v) { return order(v); },
                                            [](double) { return -1.0; }, none);
    const int size = a.E / a.groups;
    wave_sync();
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64)
      if (!(chosen >> (e / size & 63) & 1)) held[e] = 0;
    wave_sync();
  }
  int id = 0;
#pragma unroll 1
  for (int k = 0; k < a.K; ++k) {
    uint64_t m = 0;
    int e = 1 << 20;
#pragma unroll 1
    for (int i = lane; i < a.E; i += 64) {
      const uint64_t x = held[i];
      e = x > m ? i : e;
      m = max(m, x);
    }
    const uint64_t best = most<64>(m);
    e = least<64>(m == best ? e : 1 << 20);
    if (lane == (e & 63)) held[e] = 0;
    wave_sync();
    if (k == lane) id = e;
  }
  return id;
}

// The choice is made in two ways.  First by keys in fp32 less five bits, of which each lane holds its best four in
// order, so that a round is a reduction over the lanes and one move; then the K chosen and the next one are looked
// at, and only where the order of two is too close for fp32 to tell, or the last one and the next are equal, the wave
// chooses again by keys in 64 bits, one token after another.  Logits in bf16 without biases and groups are exact in
// the short keys.
// These are few with normal fp32 logits of spread 1.5 (of 384 experts with biases 3 tokens in 1000 by sigmoids, 1 by
// softmax), and many where keys tie or lie close together (131072 tokens, K 8):
//   fp32 logits that hold bf16 values: a tenth of the tokens of 384 experts; 85 us where others of fp32 take 49
//   groups whose scores differ by less than what is allowed for their errors, 2^-14 with softmax, 2^-18 with sigmoids: 256
//     experts in 8 groups without biases, softmax of logits of spread 0.1: 320 us, 0.02: 481, where 1.5 is 136; sigmoids of
//     logits below -14: 430 for 89
//
// 16 lanes a token rather than 64: a reduction is four moves in place of six, and a wave's four tokens share each
// instruction.  Measured on MI355X: 131072 tokens of 384 fp32 experts with biases, K 8: 60 us, of which the vector
// instructions are 45 (the logits' bytes would take 32); with all keys in 64 bits 386.  The same by softmax: 85.  8 tokens
// of 256 experts in 8 groups with biases: 8.8, and 7.6 a launch in a graph, where the same without groups and biases are 4.0
// (64 lanes were no faster).
template <class T, int SCORE, bool NORM, int L, int MODE>
__global__ __launch_bounds__(256, 4) void router_kernel(const RouterArgs a) {
  constexpr bool plain = MODE == kPlain;       // the logits' order is the scores'
  constexpr bool grouped = MODE == kGrouped;
  constexpr int kTokens = 256 / L;             // of a workgroup
  constexpr int kBatch = 8;                    // logits of a lane that are loaded at once
  // the biases, then for each wave what its tokens' groups are found from: short keys, or a token's in 64 bits
  extern __shared__ __align__(16) char smem[];
  float* const bias = reinterpret_cast<float*>(smem);
  const int lane = threadIdx.x & 63, sub = lane % L, mine = threadIdx.x / L;
  const int nv = (a.E + L - 1) / L;            // 32 at most: v is five bits of a key
  uint64_t* const held64 = reinterpret_cast<uint64_t*>(smem + (plain ? 0 : (a.E + 3) / 4 * 16) + (threadIdx.x >> 6) * held_bytes(a.E, L, a.groups));
  uint32_t* const held = reinterpret_cast<uint32_t*>(held64) + lane / L * a.E;
  // softmax: the least bias of a wave's experts that are not masked, and of all
  __shared__ float lows[4];
  float low = INFINITY;
  const uint32_t magic = grouped ? ((1u << 20) + a.E / a.groups - 1) / (a.E / a.groups) : 0;   // e / size for e < 1024, size <= 512
  if constexpr (!plain) {
    for (int e = threadIdx.x; e < a.E; e += 256) {
      const float b = a.bias ? a.bias[e] : 0.f;
      bias[e] = b == b ? fminf(b, kLargest) : -INFINITY;   // +inf would be no number among the short keys
      low = fminf(low, b > -INFINITY ? b : INFINITY);
    }
    if constexpr (SCORE == kSoftmax) {
      low = least<64>(low);
      if (lane == 0) lows[threadIdx.x >> 6] = low;
    }
    __syncthreads();
    if constexpr (SCORE == kSoftmax) low = fminf(fminf(lows[0], lows[1]), fminf(lows[2], lows[3]));
  }
  for (int64_t first = (int64_t)blockIdx.x * kTokens; first < a.T; first += (int64_t)gridDim.x * kTokens) {
    const int64_t t = min(first + mine, a.T - 1);          // the last token again, where there is none
    const bool there = first + mine < a.T;
    const T* row = static_cast<const T*>(a.logits) + t * a.E;
    // f(v, logit) for this lane's logits in turn, a batch ahead; where there is no expert any more, the logit is
    // NaN and v -1
    auto each = [&](auto f) {
      const T* at = row + sub;
      float now[kBatch], then[kBatch];
      int v0 = 0;
      auto fetch = [&](float (&to)[kBatch], int v, auto whole) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          to[u] = load_logit(whole ? at + u * L : row + min((v + u) * L + sub, a.E - 1));
        at += kBatch * L;
      };
      const int full = a.E / (kBatch * L);                 // batches that every lane has all of
      if (full > 0) {
        fetch(now, 0, std::true_type{});
#pragma unroll 1
        for (int i = 1; i <= full; ++i, v0 += kBatch) {
          if (i < full) fetch(then, v0 + kBatch, std::true_type{});
#pragma unroll
          for (int u = 0; u < kBatch; ++u) f(v0 + u, now[u]);
#pragma unroll
          for (int u = 0; u < kBatch; ++u) now[u] = then[u];
        }
      }
      if (v0 < nv) {
        fetch(now, v0, std::false_type{});
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if ((v0 + u) * L + sub < a.E) f(v0 + u, now[u]);
      }
    };
    float top = 0.f, total = 1.f;                          // softmax: of the whole row
    if (SCORE == kSoftmax && (!NORM || !plain)) {
      top = -INFINITY;
      each([&](int, float l) { top = fmaxf(top, clean(l)); });
      top = most<L>(top);
      total = 0.f;
      each([&](int, float l) { total += l > -INFINITY ? expf(clean(l) - top) : 0.f; });
      total = sum<L>(total);
    }
    const float over_total = 1.f / total;
    // an expert's score in fp32: off by 3 * 2^-23 (sigmoid), by 2^-17 of itself and 2^-63 (softmax, x away from the
    // largest logit: 52 + 2.25 x roundings, of the sum and of the argument's size, are 128 up to x = 33, and beyond
    // it, down to where the exponential underflows, the score is below 2^-47)
    auto score32 = [&](float x) -> float {
      return SCORE == kSoftmax ? __expf(x - top) * over_total : __builtin_amdgcn_rcpf(1.f + __expf(-x));
    };
    // a score underflows to +0, so that no sum is -0
    auto key_of = [&](int v, float l) -> uint32_t {
      if constexpr (plain) return short_key(clean(l), v);
      float x = score32(SCORE == kSoftmax ? fminf(l, kLargest) : l);
      x += bias[v * L + sub];
      return short_key(l > -INFINITY ? x : -INFINITY, v);
    };
    bool close = false;                                    // fp32 cannot tell
    uint64_t chosen = ~0ull;
    if constexpr (grouped) {
      float largest = 0.f;                                 // magnitude of a key
      wave_sync();
      each([&](int v, float l) {
        const uint32_t k = key_of(v, l);
        held[v * L + sub] = k;
        largest = fmaxf(largest, k > kMasked32 ? fabsf(number(k)) : 0.f);
      });
      largest = most<L>(largest) * 0x1.0001p0f;
      wave_sync();
      chosen = best_groups<L>(
          held, sub, a.E, a.groups, a.top_groups, kMasked32, [](uint32_t k) { return k > kMasked32 ? number(k) : -INFINITY; },
          [](float x) { return order(fmaxf(x, -kLargest) + 0.f); },
          // two keys of each, off by their errors and five bits; sums that may be out of range say nothing
          [&](float) { return largest < 0x1p126f ? (SCORE == kSoftmax ? 0x1p-14f : 0x1p-18f) + largest * 0x1p-15f : INFINITY; }, close);
    }
    uint32_t k0 = 0, k1 = 0, k2 = 0, k3 = 0;               // the lane's best four
    auto take = [&](uint32_t x) {
      k3 = med3(k2, k3, x);
      k2 = med3(k1, k2, x);
      k1 = med3(k0, k1, x);
      k0 = max(k0, x);
    };
    // of all keys, or those below `limit`
    auto fill = [&](auto all, uint32_t limit) {
      k0 = k1 = k2 = k3 = 0;
      if constexpr (grouped) {
#pragma unroll 4
        for (int v = 0; v < nv; ++v) {
          const int e = v * L + sub;
          const uint32_t x = e < a.E ? held[e] : 0;
          take((all || x < limit) && (chosen >> (e * magic >> 20 & 63) & 1) ? x : 0);
        }
      } else {
        each([&](int v, float l) {
          const uint32_t x = key_of(v, l);
          take(all || x < limit ? x : 0);
        });
      }
    };
    int id = 0, left = 4;                                  // lane k has the k-th, lane K the next
    fill(std::true_type{}, 0);
#pragma unroll 1
    for (int k = 0;;) {
      const uint32_t m = most<L>(k0);
      const int from = least<L>(k0 == m ? sub : L);
      if (k == sub) id = m ? (int)(31 - (m & 31)) * L + from : -1;       // -1: there is no next one
      if (k == a.K) break;
      ++k;
      if (from == sub) {
        k0 = k1;
        k1 = k2;
        k2 = k3;
        k3 = 0;
        --left;
      }
      if (__any(left == 0)) {                              // a lane whose four are gone may have more
        const uint32_t o0 = k0, o1 = k1, o2 = k2, o3 = k3;
        fill(std::false_type{}, m);
        if (left != 0) {
          k0 = o0; k1 = o1; k2 = o2; k3 = o3;
        } else {
          left = 4;
        }
      }
    }
    // lane k's logit, and whether k and k + 1 can be told apart
    auto chosen_logit = [&](int e) -> float { return (unsigned)e < (unsigned)a.E ? clean(load_logit(row + e)) : -INFINITY; };
    float x = sub <= a.K ? chosen_logit(id) : -INFINITY;
    if (!(plain && sizeof(T) == 2)) {
      const float b = !plain && sub <= a.K && id >= 0 ? bias[id] : 0.f;
      float f = x, s = 0.f;
      if (!plain) {
        s = x > -INFINITY ? score32(x) : 0.f;
        f = x > -INFINITY ? s + b : -INFINITY;
      }
      auto next = [](float v) {
        if constexpr (L == 16) return __uint_as_float(dpp<0x101>(__float_as_uint(v)));
        return __uint_as_float(dpp<0x130>(__float_as_uint(v)));
      };
      const float fn = next(f), xn = next(x), bn = next(b), sn = next(s);
      const int idn = (int)__float_as_uint(next(__uint_as_float((uint32_t)id)));
      const bool last = sub == a.K - 1;
      // both keys are off, each by its own score's error.  Behind the last one others may be hidden, by the five bits or
      // by their errors: their scores are not larger than the largest, nor than what the least bias leaves of a key
      const float hidden = fminf(over_total, f - low + (fabsf(f) + fabsf(low)) * 0x1p-16f);
      float gap = plain ? 0.f : fabsf(f) * 0x1p-22f + (SCORE == kSoftmax ? (s + (last ? hidden : sn)) * 0x1p-17f + 0x1p-62f : 0x1p-20f);
      if (last) gap += fabsf(f) * 0x1p-17f + 0x1p-144f;    // the five bits, of subnormal numbers too
      // masked ones are in order, and so are equal ones, but for biases that may be +inf; what is beyond the last is not known to be
      const bool apart = f - fn > gap || (f > -INFINITY && fn == -INFINITY) || (f == -INFINITY && fn == -INFINITY && x == -INFINITY) ||
                         (!last && x == xn && b == bn && b < kLargest && id < idn);
      if (sub < a.K && idn >= 0 && !apart) close = true;
    }
    // one token after another, by all lanes
    uint64_t again = __ballot(close);
    while (again) {
      const int at = (__ffsll((unsigned long long)again) - 1) / L;           // its lanes' place
      again &= ~(((L == 64 ? 0ull : 1ull << (L & 63)) - 1) << at * L);
      const int e = exact_choice<T, SCORE, MODE>(a, min(first + mine - lane / L + at, a.T - 1), held64);
      const int got = __shfl(e, sub);
      if (lane / L == at) id = got;
      x = sub < a.K ? chosen_logit(id) : -INFINITY;
    }
    if (sub >= a.K) x = -INFINITY;
    // normalised: of the scores' ratios, so that scores too small for fp32 still have them
    float m = SCORE == kSigmoid ? fminf(x, 0.f) : x, w;
    m = NORM ? most<L>(m) : SCORE == kSigmoid ? 0.f : top;
    if constexpr (SCORE == kSigmoid) w = expf(fminf(x, 0.f) - m) / (1.f + expf(-fabsf(x)));
    else w = NORM ? expf(x - m) : expf(x - m) / total;
    w = x > -INFINITY ? w : 0.f;
    if constexpr (NORM) {
      const float s = sum<L>(w);
      w = s > 0.f ? w / s : 0.f;
    }
    if (there && sub < a.K) {
      a.ids[t * a.K + sub] = id;
      a.w[t * a.K + sub] = w * a.scale;
    }
  }
}

// The chosen logits' gradients, from the weights':
//   normalised, p = s / sum(s):  scale p (g - sum(g p)), times 1 - s for the sigmoid;
//   else sigmoid: scale g s (1 - s);  softmax: scale s (g - sum(g s)), and -scale s sum(g s) for
//   every logit that was not chosen.
// A wave's rows come together in LDS and leave in whole lines, since lines of which parts are written cost their
// reading: zeros first and the chosen ones over them took 32 us where this takes 27, and 37 where the caches hold nothing of
// it (131072 tokens of 384 bf16 logits, K 8, normalised: 100 MB to write, and the K logits of a row are in nearly
// all its lines, so all are read).
template <class T, int SCORE, bool NORM, int L, int V>
__global__ __launch_bounds__(256) void router_bwd_kernel(const RouterArgs a) {
  constexpr int kTokens = 64 / L;              // of a wave
  constexpr bool kDense = SCORE == kSoftmax && !NORM;
  constexpr int kVec = 16 / sizeof(T);
  __shared__ __align__(16) float rows[4][kTokens * V * L];
  const int lane = threadIdx.x & 63, sub = lane % L, mine = lane / L;
  float* const held = rows[threadIdx.x >> 6];  // E to a token
  const int64_t step = (int64_t)gridDim.x * 4 * kTokens;
  for (int64_t first = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * kTokens; first < a.T; first += step) {
    const int64_t t = min(first + mine, a.T - 1);
    const T* row = static_cast<const T*>(a.logits) + t * a.E;
    int id = sub < a.K ? a.ids_in[t * a.K + sub] : -1;
    if ((unsigned)id >= (unsigned)a.E) id = -1;
    float g = id >= 0 ? a.g_w[t * a.K + sub] * a.scale : 0.f;
    const float x = id >= 0 ? clean(load_logit(row + id)) : -INFINITY;
    if (x == -INFINITY) g = 0.f;               // masked: a score of zero, whatever its logit
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
    float m = SCORE == kSigmoid ? fminf(x, 0.f) : x;
    m = NORM ? most<L>(m) : SCORE == kSigmoid ? 0.f : top;
    const float z = 1.f / (1.f + expf(-fabsf(x)));         // sigmoid of |x|
    float p = SCORE == kSigmoid ? expf(fminf(x, 0.f) - m) * z : NORM ? expf(x - m) : expf(x - m) / total;
    p = x > -INFINITY ? p : 0.f;
    // 1 - s, without the difference where s is near one
    const float rest = SCORE == kSoftmax ? 1.f : x > 0.f ? expf(-x) * z : z;
    if constexpr (NORM) {
      const float s = sum<L>(p);
      p = s > 0.f ? p / s : 0.f;
    }
    const float dot = SCORE == kSigmoid && !NORM ? 0.f : sum<L>(g * p);
    const float d = kDense ? p * g : p * (g - dot) * rest;
    // whether an expert is named twice: then one of the lanes does not find itself there
    wave_sync();
    if (id >= 0) held[mine * a.E + id] = (float)sub;
    wave_sync();
    const bool twice = id >= 0 && held[mine * a.E + id] != (float)sub;
    wave_sync();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + sub;
      if (e < a.E) held[mine * a.E + e] = kDense && total > 0.f ? l[kDense ? v : 0] / total * -dot : 0.f;
    }
    wave_sync();
    if (__any(twice)) {                        // the lanes take turns
      for (int k = 0; k < a.K; ++k) {
        if (k == sub && id >= 0) held[mine * a.E + id] += d;
        wave_sync();
      }
    } else if (id >= 0) {
      held[mine * a.E + id] += d;
    }
    wave_sync();
    const int n = (int)min((int64_t)kTokens, a.T - first) * a.E;
    T* const out = static_cast<T*>(a.g) + first * a.E;
    const int whole = reinterpret_cast<uintptr_t>(out) % 16 == 0 ? n / kVec : 0;      // vectors
    for (int i = lane; i < whole; i += 64) {
      T o[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) store_logit(o + j, held[i * kVec + j]);
      *reinterpret_cast<u32x4*>(out + i * kVec) = __builtin_bit_cast(u32x4, o);
    }
    for (int i = whole * kVec + lane; i < n; i += 64) store_logit(out + i, held[i]);
  }
}

template <class T, int SCORE, bool NORM, int L>
void launch_fwd(const RouterArgs& a, hipStream_t st) {
  constexpr int kTokens = 256 / L;               // of a workgroup
  const int lds = (a.bias || a.groups > 1 ? (a.E + 3) / 4 * 16 : 0) + 4 * held_bytes(a.E, L, a.groups);
  const unsigned grid = (unsigned)std::min<int64_t>((a.T + kTokens - 1) / kTokens, kWgs);
  if (a.groups > 1) hipLaunchKernelGGL((router_kernel<T, SCORE, NORM, L, kGrouped>), dim3(grid), dim3(256), lds, st, a);
  else if (a.bias) hipLaunchKernelGGL((router_kernel<T, SCORE, NORM, L, kBiased>), dim3(grid), dim3(256), lds, st, a);
  else hipLaunchKernelGGL((router_kernel<T, SCORE, NORM, L, kPlain>), dim3(grid), dim3(256), lds, st, a);
}

template <class T, int SCORE, bool NORM, int L, int V>
void launch_bwd(const RouterArgs& a, hipStream_t st) {
  constexpr int kTokens = 256 / L;
  const unsigned grid = (unsigned)std::min<int64_t>((a.T + kTokens - 1) / kTokens, kWgs);
  hipLaunchKernelGGL((router_bwd_kernel<T, SCORE, NORM, L, V>), dim3(grid), dim3(256), 0, st, a);
}

template <class T, int SCORE, bool NORM, bool BWD>
void launch_sized(const RouterArgs& a, hipStream_t st) {
  if constexpr (!BWD) {
    // lane K of a token has the first that is not chosen
    if (a.K >= 16 || a.E > 512) launch_fwd<T, SCORE, NORM, 64>(a, st);
    else launch_fwd<T, SCORE, NORM, 16>(a, st);
  } else {
    if (a.K > 16 || a.E > 384) launch_bwd<T, SCORE, NORM, 64, 16>(a, st);
    else if (a.E <= 64) launch_bwd<T, SCORE, NORM, 16, 4>(a, st);
    else launch_bwd<T, SCORE, NORM, 16, 24>(a, st);
  }
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
