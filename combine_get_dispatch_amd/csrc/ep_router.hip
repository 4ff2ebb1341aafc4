// The router's kernels for gfx950: top-k selection, the load-balance loss,
// and the gradient of both for the logits.  Contracts in include/ep_moe.h.
//
// A token's row of E logits belongs to LPT lanes of one wave, V values each
// (four consecutive ones at a time, so a row is read in 16-byte pieces):
// element i of lane l is expert (i / 4) * 4 * LPT + 4 * l + i % 4.  Rows
// stay in registers from the load to the result.
#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <type_traits>
#include <stdint.h>

#include "ep.h"
#include "ep_host.h"
#include "ep_moe.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kQuad = 4;  // consecutive experts per piece of a row

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}

// Nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

__device__ __forceinline__ float logit_of(float v) { return v; }
__device__ __forceinline__ float logit_of(uint16_t v) { return bf16_to_f32(v); }

// LDS written by some lanes of a wave and read by others of the same wave: a
// wave's LDS accesses complete in order, so only the compiler is held.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int LPT, int V>
__device__ __forceinline__ int expert_of(int l, int i) {
  return (i / kQuad) * (kQuad * LPT) + l * kQuad + i % kQuad;
}

// One lane's part of a row; elements past E are -inf.  vec: rows are aligned
// to a piece (E % 4 == 0 and an aligned base).  Past the end a lane reads the
// row's last elements, so that no load is under a branch.
template <int LPT, int V, typename L>
__device__ __forceinline__ void load_row(const L *row, int E, int l, bool vec, float (&x)[V]) {
  typedef L Piece __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int q = 0; q < V / kQuad; ++q) {
    const int e = expert_of<LPT, V>(l, q * kQuad);
    Piece v;
    if (vec) {
      v = *reinterpret_cast<const Piece *>(row + (e < E ? e : E - kQuad));
    } else {
      // worked out here, not held through a caller's loop
      int at = e;
      asm volatile("" : "+v"(at));
#pragma unroll
      for (int i = 0; i < kQuad; ++i) v[i] = row[at + i < E ? at + i : E - 1];
    }
#pragma unroll
    for (int i = 0; i < kQuad; ++i)
      x[q * kQuad + i] = e + i < E ? logit_of(v[i]) : -INFINITY;
  }
}

template <int LPT, int V>
__device__ __forceinline__ void store_row(float *row, int E, int l, bool vec,
                                          const float (&x)[V]) {
#pragma unroll
  for (int q = 0; q < V / kQuad; ++q) {
    const int e = expert_of<LPT, V>(l, q * kQuad);
    if (vec) {
      const f32x4 v = {x[q * kQuad], x[q * kQuad + 1], x[q * kQuad + 2], x[q * kQuad + 3]};
      if (e < E) *reinterpret_cast<f32x4 *>(row + e) = v;
    } else {
#pragma unroll
      for (int i = 0; i < kQuad; ++i)
        if (e + i < E) row[e + i] = x[q * kQuad + i];
    }
  }
}

template <int LPT, int V>
__device__ __forceinline__ void store_row(uint16_t *row, int E, int l, bool vec,
                                          const float (&x)[V]) {
#pragma unroll
  for (int q = 0; q < V / kQuad; ++q) {
    const int e = expert_of<LPT, V>(l, q * kQuad);
    if (vec) {
      const u16x4 v = {f32_to_bf16(x[q * kQuad]), f32_to_bf16(x[q * kQuad + 1]),
                       f32_to_bf16(x[q * kQuad + 2]), f32_to_bf16(x[q * kQuad + 3])};
      if (e < E) *reinterpret_cast<u16x4 *>(row + e) = v;
    } else {
#pragma unroll
      for (int i = 0; i < kQuad; ++i)
        if (e + i < E) row[e + i] = f32_to_bf16(x[q * kQuad + i]);
    }
  }
}

// A value of another lane.  Step s of a reduction over LPT lanes pairs lanes
// whose groups of 2^s lanes are still apart: inside 16 lanes by data-parallel
// moves (neighbours, pairs, and mirrors of 8 and of 16 lanes: after the steps
// before, all lanes of a half hold the same), beyond by a shuffle.
template <int kStep>
__device__ __forceinline__ int other_lane(int v) {
  if constexpr (kStep == 0)
    return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);
  else if constexpr (kStep == 1)
    return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);
  else if constexpr (kStep == 2)
    return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);
  else if constexpr (kStep == 3)
    return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);
  else
    return __shfl_xor(v, 1 << kStep);
}

template <int kStep>
__device__ __forceinline__ float other_lane(float v) {
  return __int_as_float(other_lane<kStep>(__float_as_int(v)));
}

template <int kStep>
__device__ __forceinline__ uint32_t other_lane(uint32_t v) {
  return (uint32_t)other_lane<kStep>((int)v);
}

template <int kStep>
__device__ __forceinline__ double other_lane(double v) {
  return __hiloint2double(other_lane<kStep>(__double2hiint(v)),
                          other_lane<kStep>(__double2loint(v)));
}

// Calls f with steps 0, 1, ... of a reduction over LPT lanes.
template <int LPT, int kStep = 0, typename F>
__device__ __forceinline__ void each_step(F f) {
  if constexpr ((1 << kStep) < LPT) {
    f(std::integral_constant<int, kStep>{});
    each_step<LPT, kStep + 1>(f);
  }
}

// Reductions over the LPT lanes of a token: every lane gets the same result,
// in a fixed order.
template <int LPT, typename T>
__device__ __forceinline__ T token_max(T v) {
  each_step<LPT>([&](auto s) {
    const T o = other_lane<s.value>(v);
    v = o > v ? o : v;
  });
  return v;
}

template <int LPT>
__device__ __forceinline__ float token_max(float v) {
  each_step<LPT>([&](auto s) { v = fmaxf(v, other_lane<s.value>(v)); });
  return v;
}

template <int LPT, typename T>
__device__ __forceinline__ T token_sum(T v) {
  each_step<LPT>([&](auto s) { v += other_lane<s.value>(v); });
  return v;
}

template <int LPT>
__device__ __forceinline__ int token_or(int v) {
  each_step<LPT>([&](auto s) { v |= other_lane<s.value>(v); });
  return v;
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// exp of every score of a row: the hardware's exp2 of x log2(e), off by
// (1.23 |x| + 3) 2^-24 of it: the product's rounding 1 |x|, its fp32 constant
// 0.22 |x|, the exp2 2.  (A second fma for the constant's rest would be two
// instructions more on a path that instructions bound, for scores whose own
// steps are far larger.)
__device__ __forceinline__ float exp_fast(float v) {
  return __builtin_amdgcn_exp2f(v * 0x1.715476p+0f);
}

// sigmoid(x) / exp(m) with m = min(0, the largest x in play), so that scores
// whose largest would underflow keep their ratios: for x <= 0,
// exp(x - m) / (1 + exp(x)).
__device__ __forceinline__ float sigmoid_over(float x, float m) {
  const float t = exp_of(-fabsf(x));
  const float num = x > 0.0f ? 1.0f : (m == 0.0f ? t : exp_of(x - m));
  return num / (1.0f + t);
}

// The sigmoid for every score of a row: exp overflows to inf and the quotient
// to 0 below -88.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x));
}

template <typename K>
__device__ __forceinline__ K sigmoid_of(K x) {
  const K t = exp_of(x > K(0) ? -x : x);
  return (x > K(0) ? K(1) : t) / (K(1) + t);
}

struct RouteArgs {
  const void *logits;
  const float *bias;
  const uint8_t *token_mask;
  int32_t *topk_idx;
  float *topk_weights;
  int32_t *status;
  int64_t T;
  int32_t E, k, G, group_size, topk_groups, group_topn;
  int32_t group_steps;  // log2(group_size / 4) for keep_even_groups, -1: keep_groups
  uint32_t group_inv;  // ceil(2^22 / group_size): e / group_size = e * group_inv >> 22
  bool softmax, normalize, vec;
  float scale;
};

// The two best of a set, as the set grows.
template <typename K>
struct Best2 {
  K first, second;
  __device__ __forceinline__ void add(K v) {
    second = v > first ? first : (v > second ? v : second);
    first = v > first ? v : first;
  }
  template <int kStep>
  __device__ __forceinline__ void join() {
    const K a = other_lane<kStep>(first), b = other_lane<kStep>(second);
    const K low = a < first ? a : first, high = b > second ? b : second;
    first = a > first ? a : first;
    second = low > high ? low : high;
  }
  __device__ __forceinline__ K key(int topn) const {
    return topn == 2 && second > K(-INFINITY) ? first + second : first;
  }
};

// In 32 bits by the median of three (no NaN gets here).
template <>
struct Best2<float> {
  float first, second;
  __device__ __forceinline__ void add(float v) {
    second = __builtin_amdgcn_fmed3f(first, second, v);
    first = fmaxf(first, v);
  }
  template <int kStep>
  __device__ __forceinline__ void join() {
    const float a = other_lane<kStep>(first), b = other_lane<kStep>(second);
    second = fmaxf(fminf(first, a), fmaxf(second, b));
    first = fmaxf(first, a);
  }
  // two keys near the type's lowest add to -inf, which would mean no key
  __device__ __forceinline__ float key(int topn) const {
    return topn == 2 && second > -INFINITY ? fmaxf(first + second, -FLT_MAX) : first;
  }
  // what its rounding goes by: the two may cancel
  __device__ __forceinline__ float size(int topn) const {
    return topn == 2 && second > -INFINITY ? fmaxf(fabsf(first), fabsf(second)) : fabsf(first);
  }
};

// How far a key in 32 bits may be off by the rounding of its own bias and sum:
// of one key 2^-24 of itself, of a group's sum of two 2^-22 of the larger.  Two
// neighbours are compared by the lower one: a higher one of more than twice its
// size is far enough away.
constexpr float kKeyStep = 0x1p-20f;
constexpr float kGroupStep = 0x1p-21f;

// The groups kept, as 64 bits, from the group keys in LDS (written by lanes of
// this token, and read here after the wave has met; behind them, if near is
// given, their sizes).  Lane l ranks groups l, l + LPT, ...; near: a kept and a
// dropped group are within `margin` and what their own roundings add.
template <int LPT>
__device__ __forceinline__ uint64_t kept_of(const RouteArgs &a, int l, float *group_key,
                                            float margin, bool *near) {
  const float none = -INFINITY;
  if (l < (-a.G & 3)) group_key[a.G + l] = none;
  wave_sync();
  uint32_t kept[2] = {0, 0};
  float low = INFINITY, high = none;  // the lowest a kept one can be, the highest a dropped one
  for (int g = l; g < a.G; g += LPT) {
    const float v = group_key[g];
    if (!(v > none)) continue;
    const float off = near != nullptr ? kGroupStep * group_key[EP_MAX_GROUPS + g] : 0.0f;
    int before = 0;
    for (int h = 0; h < a.G; h += 4) {  // the keys are filled up to fours
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float o = group_key[h + i];
        before += o > v || (o == v && h + i < g);
      }
    }
    if (before < a.topk_groups) {
      kept[g / 32] |= 1u << (g % 32);
      low = fminf(low, v - off);
    } else {
      high = fmaxf(high, v + off);
    }
  }
  if (near != nullptr) {
    low = -token_max<LPT>(-low);
    high = token_max<LPT>(high);
    if (high > none && !(low - high > margin)) *near = true;
  }
  const uint32_t lo = token_or<LPT>((int)kept[0]);
  const uint32_t hi = a.G > 32 ? token_or<LPT>((int)kept[1]) : 0;
  return (uint64_t)hi << 32 | lo;
}

// Drops the keys of the groups that are not kept.  Groups of any size: each is
// gathered from the lanes by itself.
template <int LPT, int V>
__device__ __forceinline__ void keep_groups(const RouteArgs &a, float (&key)[V], int l,
                                            float *group_key, float margin, bool *near) {
  const float none = -INFINITY;
  for (int g = 0; g < a.G; ++g) {
    Best2<float> best = {none, none};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = expert_of<LPT, V>(l, i) - g * a.group_size;
      best.add(e >= 0 && e < a.group_size ? key[i] : none);
    }
    each_step<LPT>([&](auto s) { best.template join<s.value>(); });
    if (l == 0) group_key[g] = best.key(a.group_topn);
    if (l == 0 && near != nullptr) group_key[EP_MAX_GROUPS + g] = best.size(a.group_topn);
  }
  const uint64_t kept = kept_of<LPT>(a, l, group_key, margin, near);
  wave_sync();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int g = (int)(((uint32_t)expert_of<LPT, V>(l, i) * a.group_inv) >> 22);
    if (g >= 64 || !((kept >> g) & 1)) key[i] = none;
  }
}

// The same for groups of 2^n pieces of four experts that lie within one piece
// per lane (a.group_steps = n): all groups of a piece at once, by n steps
// between lanes.  256 experts in 8 groups: 100 instructions instead of 800.
template <int LPT, int V>
__device__ __forceinline__ void keep_even_groups(const RouteArgs &a, float (&key)[V], int l,
                                                 float *group_key, float margin, bool *near) {
  const float none = -INFINITY;
  Best2<float> best[V / kQuad];
#pragma unroll
  for (int q = 0; q < V / kQuad; ++q) {
    best[q] = {key[q * kQuad], none};
#pragma unroll
    for (int i = 1; i < kQuad; ++i) best[q].add(key[q * kQuad + i]);
  }
  each_step<LPT>([&](auto s) {
    if (s.value < a.group_steps) {
#pragma unroll
      for (int q = 0; q < V / kQuad; ++q) best[q].template join<s.value>();
    }
  });
  const bool leader = (l & ((1 << a.group_steps) - 1)) == 0;
#pragma unroll
  for (int q = 0; q < V / kQuad; ++q) {
    const int g = (q * LPT + l) >> a.group_steps;
    if (leader && g < a.G) {
      group_key[g] = best[q].key(a.group_topn);
      if (near != nullptr) group_key[EP_MAX_GROUPS + g] = best[q].size(a.group_topn);
    }
  }
  const uint64_t kept = kept_of<LPT>(a, l, group_key, margin, near);
  wave_sync();
#pragma unroll
  for (int q = 0; q < V / kQuad; ++q) {
    const int g = (q * LPT + l) >> a.group_steps;
    if (g >= 64 || !((kept >> g) & 1)) {
#pragma unroll
      for (int i = 0; i < kQuad; ++i) key[q * kQuad + i] = none;
    }
  }
}

// The k best of one token's keys, in order, by k rounds of a search; slot j is
// given to lane j % LPT as its mine[j / LPT].  A key of -inf is never selected.
// near (kCheck): two neighbours in the order, the first one not selected
// among them, are within `margin` and what their own roundings add.
template <int LPT, int V, bool kCheck>
__device__ __forceinline__ void best_by_rounds(const RouteArgs &a, float (&key)[V], int l,
                                               int (&mine)[32 / (LPT < 32 ? LPT : 32)],
                                               float margin, bool *near) {
  const float none = -INFINITY;
#pragma unroll
  for (int s = 0; s < 32 / (LPT < 32 ? LPT : 32); ++s) mine[s] = -1;
  float last = INFINITY;
#pragma unroll 1
  for (int j = 0; j < (kCheck ? a.k + 1 : a.k); ++j) {
    float best = none;
    int at = 1 << 20;
#pragma unroll
    for (int i = 0; i < V; ++i) {  // experts ascend with i: the first of equals stays
      at = key[i] > best ? expert_of<LPT, V>(l, i) : at;
      best = key[i] > best ? key[i] : best;
    }
    each_step<LPT>([&](auto s) {
      const float o = other_lane<s.value>(best);
      const int oat = other_lane<s.value>(at);
      const bool take = o > best || (o == best && oat < at);
      best = take ? o : best;
      at = take ? oat : at;
    });
    if (!(best > none)) break;
    if (kCheck && !(last - best > margin + kKeyStep * fabsf(best))) *near = true;
    last = best;
#pragma unroll
    for (int s = 0; s < 32 / (LPT < 32 ? LPT : 32); ++s)
      if (j < a.k && j == s * LPT + l) mine[s] = at;
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = expert_of<LPT, V>(l, i) == at ? none : key[i];
  }
}

// The front bits of a fp32 key, ordered as whole numbers, and its expert in the
// last bits, so that one maximum moves both and the lowest expert is the
// greatest of equals.  0: a key of -inf.
template <int kBits>
__device__ __forceinline__ uint32_t pack_key(float key, int e) {
  constexpr uint32_t kMask = (1u << kBits) - 1;
  const uint32_t u = __float_as_uint(key + 0.0f);  // -0 as +0
  const uint32_t ordered = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  const uint32_t p = (ordered & ~kMask) | ((uint32_t)e ^ kMask);
  return key > -INFINITY ? p : 0u;
}

template <int kBits>
__device__ __forceinline__ int expert_in(uint32_t p) {
  constexpr uint32_t kMask = (1u << kBits) - 1;
  return p == 0 ? -1 : (int)((p & kMask) ^ kMask);
}

// The least (low) or the greatest key with these front bits.
template <int kBits>
__device__ __forceinline__ float key_in(uint32_t p, bool low) {
  constexpr uint32_t kMask = (1u << kBits) - 1;
  const uint32_t o = low ? p & ~kMask : p | kMask;
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

__device__ __forceinline__ void order(uint32_t &a, uint32_t &b) {
  const uint32_t high = umax(a, b);
  b = umin(a, b);
  a = high;
}

constexpr int kList = 8;

// Sorts a list that first rises or falls and then does the other; descending.
__device__ __forceinline__ void sort_bitonic(uint32_t (&v)[kList]) {
#pragma unroll
  for (int d = kList / 2; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < kList; ++i)
      if ((i & d) == 0) order(v[i], v[i + d]);
}

__device__ __forceinline__ void sort4(uint32_t *v) {
  order(v[0], v[1]);
  order(v[2], v[3]);
  order(v[0], v[2]);
  order(v[1], v[3]);
  order(v[1], v[2]);
}

// 19 comparisons, the fewest for eight values.
__device__ __forceinline__ void sort8(uint32_t *v) {
  order(v[0], v[2]); order(v[1], v[3]); order(v[4], v[6]); order(v[5], v[7]);
  order(v[0], v[4]); order(v[1], v[5]); order(v[2], v[6]); order(v[3], v[7]);
  order(v[0], v[1]); order(v[2], v[3]); order(v[4], v[5]); order(v[6], v[7]);
  order(v[2], v[4]); order(v[3], v[5]);
  order(v[1], v[4]); order(v[3], v[6]);
  order(v[1], v[2]); order(v[3], v[4]); order(v[5], v[6]);
}

// The eight best of one token's packed keys, in order, in every lane.  Each
// lane sorts its own; joining two sorted lists of eight keeps the greater of
// a[i] and b[7 - i], which are the eight best and rise and fall once.
template <int LPT, int V>
__device__ __forceinline__ void best_eight(uint32_t (&v)[V], uint32_t (&list)[kList]) {
  if constexpr (V == 4) {
    sort4(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      list[i] = v[i];
      list[7 - i] = other_lane<0>(v[i]);
    }
    sort_bitonic(list);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += kList) sort8(v + i);
#pragma unroll
    for (int i = 0; i < kList; ++i) list[i] = v[i];
#pragma unroll
    for (int n = kList; n < V; n += kList) {
#pragma unroll
      for (int i = 0; i < kList; ++i) list[i] = umax(list[i], v[n + 7 - i]);
      sort_bitonic(list);
    }
  }
  each_step<LPT>([&](auto s) {
    if constexpr (V > 4 || s.value > 0) {  // V == 4: step 0 is done above
      uint32_t joined[kList];
#pragma unroll
      for (int i = 0; i < kList; ++i) joined[i] = umax(list[i], other_lane<s.value>(list[7 - i]));
#pragma unroll
      for (int i = 0; i < kList; ++i) list[i] = joined[i];
      sort_bitonic(list);
    }
  });
}

// What a route kernel's keys are.
constexpr int kByLogit = 0, kBySigmoid = 1, kBySoftmax = 2;

// Keys s + b of one lane's experts (key of a logit of -inf: -inf), and the
// best score there can be: 1, or a softmax's.
template <int LPT, int V, int kMode>
__device__ __forceinline__ float score_keys(const float (&x)[V], float xmax, const float *bias,
                                            int l, float (&key)[V]) {
  float best = 1.0f;
  if (kMode == kBySoftmax) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = exp_fast(x[i] - xmax);
      sum += key[i];
    }
    best = 1.0f / token_sum<LPT>(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] *= best;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = sigmoid_fast(x[i]);
  }
#pragma unroll
  for (int q = 0; q < V; q += kQuad) {
    const f32x4 b = *reinterpret_cast<const f32x4 *>(bias + expert_of<LPT, V>(l, q));
#pragma unroll
    for (int i = q; i < q + kQuad; ++i) key[i] = x[i] > -INFINITY ? key[i] + b[i % kQuad] : -INFINITY;
  }
  return best;
}

// The selection of one token with keys in 64 bits, by the whole wave: the path
// of the few tokens whose groups (or more than 32 keys) are within the margin.
// keys: LDS of E doubles, group_key of 64; expert j of the selection is given
// to lane j as the result, -1 if there is none.  One token alone would leave
// most of its wave idle for 20 us, which a short launch then waits for; by the
// whole wave it is 3.
template <typename L, int kMode>
__device__ __forceinline__ int select_exactly(const RouteArgs &a, const L *row, float xmax,
                                              double *keys, double *group_key) {
  const double none = -INFINITY;
  const int lane = threadIdx.x % 64;
  double sum = 0.0;
  if constexpr (kMode == kBySoftmax) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) sum += exp((double)logit_of(row[e]) - (double)xmax);
    sum = token_sum<64>(sum);
  }
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    double v = logit_of(row[e]);
    if (v > none) {
      v = kMode == kBySoftmax ? exp(v - (double)xmax) / sum : sigmoid_of(v);
      if (a.bias != nullptr) v += (double)a.bias[e];
    }
    keys[e] = v;
  }
  wave_sync();
  uint64_t kept = ~uint64_t{0};
  if (a.G > 1) {
    Best2<double> best = {none, none};
    if (lane < a.G) {
#pragma unroll 1
      for (int i = 0; i < a.group_size; ++i) best.add(keys[lane * a.group_size + i]);
    }
    const double own = best.key(a.group_topn);
    group_key[lane] = own;
    wave_sync();
    int before = 0;
#pragma unroll 1
    for (int h = 0; h < a.G; ++h)
      before += group_key[h] > own || (group_key[h] == own && h < lane);
    kept = __ballot(lane < a.G && own > none && before < a.topk_groups);
  }
  int mine = -1;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    double best = none;
    int at = 1 << 20;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {  // ascending: the first of equals stays
      const int g = a.G > 1 ? (int)(((uint32_t)e * a.group_inv) >> 22) : 0;
      const double v = (kept >> g) & 1 ? keys[e] : none;
      at = v > best ? e : at;
      best = v > best ? v : best;
    }
    each_step<64>([&](auto s) {
      const double o = other_lane<s.value>(best);
      const int oat = other_lane<s.value>(at);
      const bool take = o > best || (o == best && oat < at);
      best = take ? o : best;
      at = take ? oat : at;
    });
    if (!(best > none)) break;
    if (lane == j) mine = at;
    if (lane == at % 64) keys[at] = none;
    wave_sync();
  }
  wave_sync();
  return mine;
}

// The order of the keys at or above `least`, in 64 bits: at most 32 of them,
// a lane works out one or a few and ranks it among the others.  `own` is the
// token's LDS: 32 doubles, then 2 x 32 integers.  False: there are more.
// Written for few instructions (loops stay loops): a path that is taken now
// and then waits for its own code to be fetched, which measured several times
// what the code then takes.
template <typename L, int LPT, int V, int kMode>
__device__ __forceinline__ bool order_exactly(const RouteArgs &a, const L *row,
                                              const float (&key)[V], int l, float xmax,
                                              float least, double *own,
                                              int (&mine)[32 / (LPT < 32 ? LPT : 32)]) {
  constexpr int kMost = 32;
  int *expert = reinterpret_cast<int *>(own + kMost), *slot = expert + kMost;
  uint32_t in = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) in |= key[i] >= least ? 1u << i : 0u;
  const int count = __popc(in);
  int at = count;  // of this lane's among the token's: the lanes' counts before it
#pragma unroll 1
  for (int d = 1; d < LPT; d *= 2) {
    const int before = __shfl_up(at, d, LPT);
    at += l >= d ? before : 0;
  }
  const int n = __shfl(at, LPT - 1, LPT);
  if (n > kMost) return false;
  at -= count;
#pragma unroll 1
  for (; in != 0; in &= in - 1) expert[at++] = expert_of<LPT, V>(l, __ffs(in) - 1);
  double sum = 0.0;
  if constexpr (kMode == kBySoftmax) {
#pragma unroll 1
    for (int e = l; e < a.E; e += LPT) sum += exp((double)logit_of(row[e]) - (double)xmax);
    sum = token_sum<LPT>(sum);
  }
  wave_sync();
#pragma unroll 1
  for (int c = l; c < kMost; c += LPT) {
    slot[c] = -1;
    if (c >= n) continue;
    const int e = expert[c];
    double v = logit_of(row[e]);
    if constexpr (kMode == kBySoftmax) v = exp(v - (double)xmax) / sum;
    if constexpr (kMode == kBySigmoid) v = sigmoid_of(v);
    if (kMode != kByLogit && a.bias != nullptr) v += (double)a.bias[e];
    own[c] = v;
  }
  wave_sync();
#pragma unroll 1
  for (int c = l; c < n; c += LPT) {
    const double v = own[c];
    const int e = expert[c];
    int before = 0;
#pragma unroll 1
    for (int h = 0; h < n; ++h) before += own[h] > v || (own[h] == v && expert[h] < e);
    slot[before] = e;
  }
  wave_sync();
#pragma unroll
  for (int s = 0; s < 32 / (LPT < 32 ? LPT : 32); ++s) {
    const int c = s * LPT + l;
    mine[s] = c < a.k && c < kMost ? slot[c] : -1;
  }
  wave_sync();
  return true;
}

// One token per LPT lanes, several tokens in turn: the next row is loaded
// before the present one is worked on.  Bound by the instructions of the
// search, not by the logits it reads, so it goes in steps, each for what the
// one before left open:
//   kShort (k <= 8): sorted lists of eight keys cut to their front bits.
//     Neighbours that the cut bits (or, for keys that are scores, the margin
//     below) cannot tell apart leave the token open, about three in a hundred;
//     the few keys in question are then ordered in 64 bits (order_exactly).
//   k > 8 (and more than 32 keys in question): k rounds of a search over the
//     32-bit keys.
//   Groups, or neighbours of that search, within the margin: all of the token's
//     keys and groups in 64 bits (select_exactly).
// The margin is 2^-18 of the best score there can be, 2^-17 for a softmax.  In
// steps of 2^-24 of the best: a score is off by 4 by its exponential and quotient
// (s (1 - s) (1.23 |x| + 3) + 3 s of a sigmoid, e^-t (1.23 t + 3) + 1 of a
// softmax), the scores of a softmax, all alike, by 31 of themselves by the sum of
// the row (15 additions in a lane, 6 between lanes, 3 + 1.23 t w / (w + 1) <= 8.5
// for the terms with w = 1023 e^-t, a quotient).  A difference of two sums of two
// keys is off by 4 x 4 + 2 x 31 = 78 at most.  What the biases
// add goes by the keys compared (kKeyStep, kGroupStep), not by the largest bias,
// so that experts put last by a large finite one leave the others' order to 32
// bits.  bf16 logits are whole within the front bits: equal means equal.
// 4096 x 256 fp32, groups: 8 us; 131072 x 64 bf16: 15 (1.5 TB/s); 65536 x 256
// fp32, sigmoid, bias, groups: 50 (1.4 TB/s), of which scores and lists are 28,
// groups 9 and the 64-bit orders 14; a softmax there 53; 16384 x 256, k = 20: 24
// by logit, 61 by sigmoid and bias.  All keys in 64 bits: 152; k rounds of a
// search for k = 8: 128.  A batch whose keys are all equal is ordered in 64 bits
// token by token: 260.
template <typename L, int LPT, int V, int kMode, bool kShort>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
  constexpr int kTokens = kThreads / LPT;
  constexpr int kSlots = 32 / (LPT < 32 ? LPT : 32);
  constexpr int kBits = LPT * V <= 32 ? 5 : LPT * V <= 64 ? 6 : LPT * V <= 128 ? 7
                      : LPT * V <= 256 ? 8 : LPT * V <= 512 ? 9 : 10;
  constexpr bool kScores = kMode != kByLogit;
  __shared__ double group_keys[kTokens][EP_MAX_GROUPS];
  __shared__ double rows[kScores ? kThreads / 64 : 1][kScores ? LPT * V : 1];
  __shared__ float biases[kScores ? LPT * V : 1];
  int l = threadIdx.x % LPT;
  const int slot = threadIdx.x / LPT;
  double *group_key = group_keys[slot];
  const int64_t stride = (int64_t)gridDim.x * kTokens;
  int bias_bad = 0;
  if constexpr (kScores) {
    for (int e = threadIdx.x; e < LPT * V; e += kThreads)
      biases[e] = a.bias != nullptr && e < a.E ? a.bias[e] : 0.0f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float b = biases[expert_of<LPT, V>(l, i)];
      bias_bad |= !(b < INFINITY);
    }
    bias_bad = token_or<LPT>(bias_bad);
  }
  const L *logits = static_cast<const L *>(a.logits);
  // the first token of the wave, and this lane's: the whole wave stays in the
  // loop until none of its tokens is left
  int64_t first = (int64_t)blockIdx.x * kTokens + threadIdx.x / 64 * (64 / LPT);
  const int in_wave = (int)(threadIdx.x % 64) / LPT;
  float next[V];
  bool next_on = false;
  const auto load = [&](int64_t n) {
    next_on = n < a.T && (a.token_mask == nullptr || a.token_mask[n] != 0);
    load_row<LPT, V>(logits + (n < a.T ? n : a.T - 1) * a.E, a.E, l, a.vec, next);
  };
  load(first + in_wave);
  for (; first < a.T; first += stride) {
    const int64_t t = first + in_wave;
    // the experts of a lane are a few additions: worked out before the loop,
    // their numbers would fill the registers through it
    asm volatile("" : "+v"(l));
    const L *row = logits + (t < a.T ? t : a.T - 1) * a.E;
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = next_on ? next[i] : -INFINITY;
    load(t + stride);
    float xmax = -INFINITY;
    int bad = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bad |= !(x[i] < INFINITY);
      xmax = fmaxf(xmax, x[i]);
    }
    xmax = token_max<LPT>(xmax);
    float key[V], margin = 0.0f;
    if constexpr (kScores) {
      // a row of -inf has no scores: any finite value for its maximum
      const float best =
          score_keys<LPT, V, kMode>(x, xmax > -INFINITY ? xmax : 0.0f, biases, l, key);
      margin = (kMode == kBySoftmax ? 0x1p-17f : 0x1p-18f) * best;
      if (bias_bad) {
#pragma unroll
        for (int i = 0; i < V; ++i) bad |= !(key[i] < INFINITY);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = x[i];
    }
    bad = token_or<LPT>(bad);
    if (bad) {  // no expert can be selected
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = -INFINITY;
    }
    // the weights' denominator where it is not that of the slots; the row's
    // registers end here
    float row_sum = 0.0f;
    if (kMode != kBySigmoid && a.softmax && !a.normalize) {
#pragma unroll
      for (int i = 0; i < V; ++i) row_sum += exp_fast(x[i] - xmax);
      row_sum = token_sum<LPT>(row_sum);
    }
    bool open = false, near = false;
    if (a.G > 1) {
      float *gk = reinterpret_cast<float *>(group_key);
      if (a.group_steps >= 0)
        keep_even_groups<LPT, V>(a, key, l, gk, margin, kScores ? &near : nullptr);
      else
        keep_groups<LPT, V>(a, key, l, gk, margin, kScores ? &near : nullptr);
    }
    int mine[kSlots];
    if constexpr (kShort) {
      uint32_t packed[V], list[kList], after = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) packed[i] = pack_key<kBits>(key[i], expert_of<LPT, V>(l, i));
      best_eight<LPT, V>(packed, list);
      uint32_t own = 0;
#pragma unroll
      for (int j = 0; j < kList; ++j) {
        own = l == j ? list[j] : own;
        if (j + 1 < kList) after = l == j ? list[j + 1] : after;
      }
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
        mine[s] = s == 0 && l < a.k ? expert_in<kBits>(own) : -1;
      if constexpr (kScores || sizeof(L) == 4) {
        // own against the next in the order; after the eighth, any other key that
        // is not clearly below it
        if (l < a.k && l + 1 < kList && own != 0 && after != 0) {
          const float next_key = key_in<kBits>(after, false);
          open = !(key_in<kBits>(own, true) - next_key >
                   (kScores ? margin + kKeyStep * fabsf(next_key) : 0.0f));
        }
        uint32_t kth = list[0];
#pragma unroll
        for (int j = 1; j < kList; ++j) kth = j < a.k ? list[j] : kth;
        const float kth_key = key_in<kBits>(kth, true);
        const float below = kScores ? margin + kKeyStep * fabsf(kth_key) : 0.0f;
        const float least =  // never -inf: keys of -inf are not among them
            kth != 0 ? fmaxf(kth_key - below, -FLT_MAX) : -FLT_MAX;
        if (a.k == kList) {
          int above = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) above += key[i] >= least ? 1 : 0;
          if (kth != 0 && token_sum<LPT>(above) > kList) open = true;
        }
        open = token_or<LPT>(open) != 0;
        if (open)
          open = !order_exactly<L, LPT, V, kMode>(a, row, key, l, xmax, least, group_key, mine);
      }
    }
    if constexpr (kShort && kScores)
      near = near || open;
    else if (!kShort || open)
      best_by_rounds<LPT, V, kScores>(a, key, l, mine, margin, &near);
    if constexpr (kScores) {
      for (uint64_t todo = __ballot(near && l == 0 && !bad); todo != 0; todo &= todo - 1) {
        const int from = __ffsll((unsigned long long)todo) - 1;
        const int64_t n = first + from / LPT;
        const int e = select_exactly<L, kMode>(a, logits + n * a.E, __shfl(xmax, from),
                                               rows[threadIdx.x / 64],
                                               group_keys[threadIdx.x / 64 * (64 / LPT)]);
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
          const int got = __shfl(e, s * LPT + l);
          if (in_wave == from / LPT) mine[s] = got;
        }
      }
    }
    if (bad && l == 0) atomicOr(a.status, EP_STATUS_BIT_NONFINITE);
    // Weights from the selected logits, relative to the largest in play.
    float sx[kSlots], w[kSlots], smax = -INFINITY, total = 1.0f;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      sx[s] = mine[s] >= 0 ? logit_of(row[mine[s] >= 0 ? mine[s] : 0]) : -INFINITY;
      smax = fmaxf(smax, sx[s]);
    }
    if (a.softmax) {
      const float top = a.normalize ? token_max<LPT>(smax) : xmax;
      float sum = 0.0f;
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        w[s] = mine[s] >= 0 ? exp_of(sx[s] - top) : 0.0f;
        sum += w[s];
      }
      total = a.normalize ? token_sum<LPT>(sum) : row_sum;
    } else {
      const float m = a.normalize ? fminf(token_max<LPT>(smax), 0.0f) : 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        w[s] = mine[s] >= 0 ? sigmoid_over(sx[s], m) : 0.0f;
        sum += w[s];
      }
      if (a.normalize) total = token_sum<LPT>(sum);
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const int at = s * LPT + l;
      if (at < a.k && t < a.T) {
        a.topk_idx[t * a.k + at] = mine[s];
        a.topk_weights[t * a.k + at] = mine[s] >= 0 ? a.scale * (w[s] / total) : 0.0f;
      }
    }
  }
}

// --------------------------------------------------------------------------
// Balance loss
// --------------------------------------------------------------------------

struct BalanceArgs {
  const void *logits;
  const int32_t *topk_idx;
  const int32_t *seq_offsets;
  int64_t T;
  int32_t E, k, S, tile;
  bool softmax, vec;
  float coef;
  float *part_p;     // [tiles + S, E] probability sums of a tile's part of a sequence
  int32_t *part_c;   // [tiles + S, E] counts, likewise
  int32_t *part_n;   // [tiles + S] tokens that count
  double *seq_loss;  // [S, seq_blocks] sum of f P over 64 experts
  int32_t seq_blocks;
  int32_t *counts, *seq_tokens;
  float *mean_probs, *prob_grad, *loss;
  int32_t *status;
};

__device__ __forceinline__ int64_t seq_bound(const int32_t *offsets, int32_t s, int64_t T) {
  if (offsets == nullptr) return s == 0 ? 0 : T;
  const int64_t o = offsets[s];
  return o < 0 ? 0 : (o > T ? T : o);
}

// The last sequence that starts at or before token t (the same for the whole
// wave): 64 starts are looked at side by side, so that 64 sequences take one
// load and 4096 two.
__device__ __forceinline__ int seq_of(const int32_t *offsets, int S, int64_t t) {
  if (offsets == nullptr) return 0;
  const int lane = threadIdx.x % 64;
  int lo = 0, n = S;  // it is one of [lo, lo + n)
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int at = lane * step;
    const uint64_t in = __ballot(at < n && offsets[lo + (at < n ? at : 0)] <= t);
    // starts ascend; if they do not (which is reported), any of them will do
    const int last = in != 0 ? 63 - __clzll(in) : 0;
    lo += last * step;
    n = n - last * step < step ? n - last * step : step;
  }
  return lo;
}

// Scores of one token's row over exp(m) and the inverse of their sum: p[i] *
// the result are its probabilities (0 if nothing has a score).
template <int LPT, int V, bool kSoftmax>
__device__ __forceinline__ float row_scores(const float (&x)[V], float (&p)[V]) {
  float xmax = x[0], sum = 0.0f;
#pragma unroll
  for (int i = 1; i < V; ++i) xmax = fmaxf(xmax, x[i]);
  xmax = token_max<LPT>(xmax);
  if (kSoftmax) {
    xmax = xmax > -INFINITY ? xmax : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = exp_fast(x[i] - xmax);
  } else if (xmax > -60.0f) {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = sigmoid_fast(x[i]);
  } else {  // the scores underflow or nearly: relative to the largest
    const float m = xmax > -INFINITY ? xmax : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = exp_fast(x[i] - m);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sum += p[i];
  sum = token_sum<LPT>(sum);
  return sum > 0.0f ? 1.0f / sum : 0.0f;
}

// One workgroup per tile of tokens.  A tile's part of sequence s goes to row
// tile + s of the partial sums: along the tokens one of the two grows, so
// every part has a row of its own.  The next token's row and ids are loaded
// before the present one's are worked on.  65536 x 256 bf16, sigmoid: 16 us, 2.2
// TB/s.  Of these the exponentials are 3 and the LDS counts none (timing copies
// without them 13.4 and 16.3); what is left is a workgroup's chain of a few
// loads, its sums in LDS and its partial row.  Longer tiles: 128 tokens 17, 256
// tokens (one workgroup per compute unit) 23.
template <typename L, int LPT, int V, bool kSoftmax>
__global__ __launch_bounds__(kThreads) void balance_tile_kernel(BalanceArgs a) {
  constexpr int kTokens = kThreads / LPT;
  constexpr int kSlots = 32 / (LPT < 32 ? LPT : 32);
  __shared__ float sums[kTokens * LPT * V];
  __shared__ int32_t cnt[EP_MAX_EXPERTS];
  __shared__ int32_t ntok;
  int l = threadIdx.x % LPT;
  const int slot = threadIdx.x / LPT;
  const int64_t first = (int64_t)blockIdx.x * a.tile;
  const int64_t end = first + a.tile < a.T ? first + a.tile : a.T;
  float next[V];
  int ids[kSlots];
  const auto load = [&](int64_t t) {
    t = t < end ? t : end - 1;
    load_row<LPT, V>(static_cast<const L *>(a.logits) + t * a.E, a.E, l, a.vec, next);
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const int at = s * LPT + l;
      ids[s] = at < a.k ? a.topk_idx[t * a.k + (at < a.k ? at : 0)] : -1;
    }
  };
  for (int64_t lo = first; lo < end;) {
    const int s = seq_of(a.seq_offsets, a.S, lo);
    int64_t hi = seq_bound(a.seq_offsets, s + 1, a.T);
    hi = hi < end ? hi : end;
    if (hi <= lo) break;  // the offsets do not ascend to T: reported by the next kernel
    load(lo + slot);
    for (int e = threadIdx.x; e < a.E; e += kThreads) cnt[e] = 0;
    if (threadIdx.x == 0) ntok = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    int mine = 0;
    for (int64_t t = lo + slot; t < hi; t += kTokens) {
      asm volatile("" : "+v"(l));  // the experts' numbers are not held through the loop
      float x[V], p[V];
      int any = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = next[i];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        const int e = ids[j];
        if (e >= 0 && e < a.E) {
          any = 1;
          atomicAdd(&cnt[e], 1);
        } else if (e != -1) {
          atomicOr(a.status, EP_STATUS_BIT_ROUTE);
        }
      }
      any = token_or<LPT>(any);
      load(t + kTokens);
      const float inv = row_scores<LPT, V, kSoftmax>(x, p);
      mine += any;
      if (any) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(p[i], inv, acc[i]);
      }
    }
    if (l == 0 && mine > 0) atomicAdd(&ntok, mine);
#pragma unroll
    for (int i = 0; i < V; ++i) sums[slot * LPT * V + expert_of<LPT, V>(l, i)] = acc[i];
    __syncthreads();
    const int64_t out = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      float v = 0.0f;
#pragma unroll 8
      for (int g = 0; g < kTokens; ++g) v += sums[g * LPT * V + e];
      a.part_p[out * a.E + e] = v;
      a.part_c[out * a.E + e] = cnt[e];
    }
    if (threadIdx.x == 0) a.part_n[out] = ntok;
    __syncthreads();
    lo = hi;
  }
}

constexpr int kSeqThreads = 1024;
constexpr int kSeqCols = 64;  // experts of a workgroup

// One workgroup per sequence and 64 experts: adds the sequence's parts in 64
// bits, 16 slices of them side by side and then those in order.  A chain of
// loads and barriers: 6 us for 1 x 64 of 256 parts as for 37 x 256 of 1061, 12
// for 1 x 64 of 1024 parts (131072 tokens in one sequence), which one workgroup
// adds.
__global__ __launch_bounds__(kSeqThreads) void balance_seq_kernel(BalanceArgs a) {
  constexpr int kSlices = kSeqThreads / kSeqCols;
  __shared__ double sum_p[kSlices][kSeqCols];
  __shared__ int32_t sum_c[kSlices][kSeqCols];
  __shared__ int32_t tokens;
  const int s = blockIdx.x;
  const int64_t lo = seq_bound(a.seq_offsets, s, a.T);
  const int64_t hi = seq_bound(a.seq_offsets, s + 1, a.T);
  if (threadIdx.x == 0) tokens = 0;
  if (threadIdx.x == 0 && a.seq_offsets != nullptr) {
    const int64_t o0 = a.seq_offsets[s], o1 = a.seq_offsets[s + 1];
    if (o0 > o1 || o0 < 0 || o1 > a.T || (s == 0 && o0 != 0) || (s == a.S - 1 && o1 != a.T))
      atomicOr(a.status, EP_STATUS_BIT_SEQS);
  }
  const int64_t first = lo / a.tile + s;
  const int64_t last = lo < hi ? (hi - 1) / a.tile + s : first - 1;
  const int col = threadIdx.x % kSeqCols, slice = threadIdx.x / kSeqCols;
  const int e = blockIdx.y * kSeqCols + col;
  double p = 0.0;
  int c = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int64_t r = first + slice; r <= last; r += kSlices) {
      p += (double)a.part_p[r * a.E + e];
      c += a.part_c[r * a.E + e];
    }
  }
  sum_p[slice][col] = p;
  sum_c[slice][col] = c;
  __syncthreads();
  int n = 0;
  for (int64_t r = first + threadIdx.x; r <= last; r += kSeqThreads) n += a.part_n[r];
  if (n > 0) atomicAdd(&tokens, n);
  __syncthreads();
  if (slice != 0) return;
  n = tokens;
#pragma unroll
  for (int g = 1; g < kSlices; ++g) {
    p += sum_p[g][col];
    c += sum_c[g][col];
  }
  const double mean = n > 0 ? p / n : 0.0;
  double dot = n > 0 ? (double)a.E * c / ((double)a.k * n) * mean : 0.0;
  if (e < a.E) {
    a.counts[(int64_t)s * a.E + e] = c;
    a.mean_probs[(int64_t)s * a.E + e] = (float)mean;
  }
  dot = token_sum<kSeqCols>(dot);
  if (col == 0) {
    a.seq_loss[(int64_t)s * gridDim.y + blockIdx.y] = dot;
    if (blockIdx.y == 0) a.seq_tokens[s] = n;
  }
}

// Workgroups of the last launch: sequences in turn.  Each counts those with
// tokens, which would grow with the square of a workgroup per sequence.
constexpr int kLossGrid = 512;

// prob_grad, and by workgroup 0 the loss.
__global__ __launch_bounds__(kThreads) void balance_loss_kernel(BalanceArgs a) {
  __shared__ double red[kThreads];
  __shared__ int32_t live;
  if (threadIdx.x == 0) live = 0;
  __syncthreads();
  double part = 0.0;
  int mine = 0;
  for (int s = threadIdx.x; s < a.S; s += kThreads) {
    mine += a.seq_tokens[s] > 0;
    for (int b = 0; b < a.seq_blocks; ++b) part += a.seq_loss[(int64_t)s * a.seq_blocks + b];
  }
  if (mine > 0) atomicAdd(&live, mine);
  red[threadIdx.x] = part;
  __syncthreads();
  const double scale = live > 0 ? (double)a.coef / live : 0.0;
  if (blockIdx.x == 0) {
    for (int m = kThreads / 2; m > 0; m /= 2) {
      if ((int)threadIdx.x < m) red[threadIdx.x] += red[threadIdx.x + m];
      __syncthreads();
    }
    if (threadIdx.x == 0) *a.loss = (float)(scale * red[0]);
  }
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    const int n = a.seq_tokens[s];
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      const double c = a.counts[(int64_t)s * a.E + e];
      a.prob_grad[(int64_t)s * a.E + e] =
          n > 0 ? (float)(scale * ((double)a.E * c / ((double)a.k * n)) / n) : 0.0f;
    }
  }
}

// --------------------------------------------------------------------------
// Gradient for the logits
// --------------------------------------------------------------------------

struct GradArgs {
  const void *logits;
  const int32_t *topk_idx;
  const float *grad_weights, *prob_grad;
  const int32_t *seq_offsets;
  const float *grad_loss;
  void *grad_logits;
  int32_t *status;
  int64_t T;
  int32_t E, k, S, passes;
  bool normalize, vec, vec_q;
  float scale;
};

// Tokens of a workgroup, in passes of one per LPT lanes: it looks for its
// sequence once.  Fewer workgroups than two per compute unit take one pass
// (333 tokens of 60 experts: 5 us, with four passes 10).
constexpr int kGradPasses = 4;
constexpr int kGradFew = 512;

// With p the probabilities, q the loss's gradient for them and g its own,
// d x_e = g p_e (q_e - sum q p), times (1 - s_e) for sigmoid scores.  The gates'
// part concerns the selected experts (and, for a softmax that is not
// normalised over them, -s_e sum s u for all): it reaches its place in the row
// through LDS, where only the places written are cleared again.  Bound by
// reading the logits and writing the gradient: the next row is loaded before
// the present one is worked on.  65536 x 256 fp32, both gradients: 37 us, 3.7
// TB/s of the 5.1 that a copy reaches.  kLoss: prob_grad is given.
template <typename L, int LPT, int V, bool kSoftmax, bool kLoss>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(GradArgs a) {
  constexpr int kTokens = kThreads / LPT;
  constexpr int kSlots = 32 / (LPT < 32 ? LPT : 32);
  __shared__ __align__(16) float lds[kTokens * LPT * V];
  int l = threadIdx.x % LPT;
  const int slot = threadIdx.x / LPT;
  float *own = lds + slot * LPT * V;
  const L *logits = static_cast<const L *>(a.logits);
  const float g = kLoss ? (a.grad_loss != nullptr ? *a.grad_loss : 1.0f) : 0.0f;
  const bool dense = kLoss || (kSoftmax && !a.normalize && a.grad_weights != nullptr);
#pragma unroll
  for (int i = 0; i < V; ++i) own[l * V + i] = 0.0f;
  const int64_t first = (int64_t)blockIdx.x * kTokens * a.passes;
  int64_t t = first + slot;
  int seq = kLoss ? seq_of(a.seq_offsets, a.S, first) : 0;
  float next[V], next_u[kSlots];
  int next_id[kSlots];
  const auto load = [&](int64_t n) {
    n = n < a.T ? n : a.T - 1;
    load_row<LPT, V>(logits + n * a.E, a.E, l, a.vec, next);
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const int at = s * LPT + l;
      next_id[s] = at < a.k ? a.topk_idx[n * a.k + at] : -1;
      next_u[s] = at < a.k && a.grad_weights != nullptr ? a.grad_weights[n * a.k + at] : 0.0f;
    }
  };
  if (t >= a.T) return;
  load(t);
  for (int pass = 0; pass < a.passes && t < a.T; ++pass, t += kTokens) {
    asm volatile("" : "+v"(l));  // the experts' numbers are not held through the loop
    const L *row = logits + t * a.E;
    float x[V], d[V], q[V], u[kSlots], sx[kSlots];
    int mine[kSlots], any = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = next[i];
    bool inside = false;
    if constexpr (kLoss) {
      if (t >= seq_bound(a.seq_offsets, seq + 1, a.T)) {
        int high = a.S - 1;  // the last sequence that starts at or before t
        while (seq < high) {
          const int mid = seq + (high - seq + 1) / 2;
          if (seq_bound(a.seq_offsets, mid, a.T) <= t)
            seq = mid;
          else
            high = mid - 1;
        }
      }
      inside = t >= seq_bound(a.seq_offsets, seq, a.T) &&
               t < seq_bound(a.seq_offsets, seq + 1, a.T);
      load_row<LPT, V>(a.prob_grad + (int64_t)seq * a.E, a.E, l, a.vec_q, q);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      int e = next_id[j];
      if (e < -1 || e >= a.E) {
        atomicOr(a.status, EP_STATUS_BIT_ROUTE);
        e = -1;
      }
      mine[j] = e;
      any |= e >= 0;
      u[j] = e >= 0 ? next_u[j] : 0.0f;
      sx[j] = e >= 0 ? logit_of(row[e >= 0 ? e : 0]) : -INFINITY;
    }
    any = token_or<LPT>(any);
    load(t + kTokens);
    float inv = 0.0f;
    if (dense) inv = row_scores<LPT, V, kSoftmax>(x, d);
    float dot = 0.0f, share = 0.0f;  // sum q p;  scale sum s u of a plain softmax
    if constexpr (kLoss) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        dot = __builtin_fmaf(expert_of<LPT, V>(l, i) < a.E ? q[i] : 0.0f, d[i], dot);
      dot = token_sum<LPT>(dot) * inv;
    }
    // the gates' part, per slot
    if (a.grad_weights != nullptr) {
      float w[kSlots], smax = sx[0], total = 0.0f, sum = 0.0f;
#pragma unroll
      for (int j = 1; j < kSlots; ++j) smax = fmaxf(smax, sx[j]);
      smax = token_max<LPT>(smax);
      if (a.normalize) {
        const float sm = fminf(smax, 0.0f);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          w[j] = sx[j] > -INFINITY
                     ? (kSoftmax ? exp_of(sx[j] - smax) : sigmoid_over(sx[j], sm))
                     : 0.0f;
          total += w[j];
        }
        total = token_sum<LPT>(total);
        total = total > 0.0f ? total : 1.0f;  // slots of -inf logits only: no gradient
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          w[j] /= total;
          sum += w[j] * u[j];
        }
        sum = token_sum<LPT>(sum);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          w[j] = a.scale * w[j] * (u[j] - sum);
          if (!kSoftmax) w[j] *= sigmoid_of(-sx[j]);
        }
      } else if (kSoftmax) {
        // the scores' own maximum, as row_scores takes it
        float xmax = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) xmax = fmaxf(xmax, x[i]);
        xmax = token_max<LPT>(xmax);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          w[j] = sx[j] > -INFINITY ? exp_of(sx[j] - xmax) * inv * u[j] : 0.0f;
          sum += w[j];
          w[j] *= a.scale;
        }
        share = a.scale * token_sum<LPT>(sum);
      } else {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          w[j] = mine[j] >= 0 ? a.scale * sigmoid_of(sx[j]) * sigmoid_of(-sx[j]) * u[j] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (mine[j] >= 0) atomicAdd(&own[mine[j]], w[j]);
      wave_sync();
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v = 0.0f;
      if (dense) {
        const float p = d[i] * inv;
        v = -p * share;
        if (kLoss) {
          float c = inside ? g * p * (q[i] - dot) : 0.0f;
          if (!kSoftmax) c *= sigmoid_fast(-x[i]);
          v += expert_of<LPT, V>(l, i) < a.E ? c : 0.0f;
        }
      }
      d[i] = v;
    }
    if (a.grad_weights != nullptr) {
#pragma unroll
      for (int i = 0; i < V; i += kQuad) {
        const f32x4 at = *reinterpret_cast<const f32x4 *>(own + expert_of<LPT, V>(l, i));
#pragma unroll
        for (int n = 0; n < kQuad; ++n) d[i + n] += at[n];
      }
      wave_sync();
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (mine[j] >= 0) own[mine[j]] = 0.0f;
      wave_sync();
    }
    if (!any) {  // padding, whatever its logits are
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = 0.0f;
    }
    store_row<LPT, V>(static_cast<L *>(a.grad_logits) + t * a.E, a.E, l, a.vec, d);
  }
}

// --------------------------------------------------------------------------
// Host side
// --------------------------------------------------------------------------

// Calls f with the lanes per token and values per lane that cover E experts.
template <typename F>
void with_row_shape(int32_t E, F f) {
  using std::integral_constant;
  if (E <= 32)
    f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
  else if (E <= 64)
    f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
  else if (E <= 128)
    f(integral_constant<int, 8>{}, integral_constant<int, 16>{});
  else if (E <= 256)
    f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else if (E <= 512)
    f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
  else
    f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

int lanes_per_token(int32_t E) { return E <= 128 ? 8 : E <= 256 ? 16 : E <= 512 ? 32 : 64; }

// Workgroups of a route launch: eight per compute unit, tokens in turn.
constexpr int64_t kRouteGrid = 2048;

// Tokens of a balance tile: about 1024 tiles (four workgroups per compute
// unit) of 32 to 256 tokens.
int balance_tile(int64_t T) {
  int tile = 32;
  while (tile < 256 && T / tile > 1024) tile *= 2;
  return tile;
}

ep_status_t check_router(const ep_router_t *r) {
  if (r == nullptr) return failf(EP_ERR_INVALID_ARG, "router is NULL");
  if (r->num_tokens < 0) return failf(EP_ERR_INVALID_ARG, "num_tokens %d < 0", r->num_tokens);
  if (r->num_experts < 1 || r->num_experts > EP_MAX_EXPERTS)
    return failf(EP_ERR_INVALID_ARG, "num_experts %d outside [1, %d]", r->num_experts,
                 EP_MAX_EXPERTS);
  if (r->num_topk < 1 || r->num_topk > EP_MAX_TOPK || r->num_topk > r->num_experts)
    return failf(EP_ERR_INVALID_ARG, "num_topk %d outside [1, min(num_experts, %d)]",
                 r->num_topk, EP_MAX_TOPK);
  if (r->score != EP_SCORE_SOFTMAX && r->score != EP_SCORE_SIGMOID)
    return failf(EP_ERR_INVALID_ARG, "unknown score %d", r->score);
  if (r->num_groups < 1 || r->num_groups > EP_MAX_GROUPS ||
      r->num_experts % r->num_groups != 0)
    return failf(EP_ERR_INVALID_ARG, "num_groups %d must be in [1, %d] and divide num_experts %d",
                 r->num_groups, EP_MAX_GROUPS, r->num_experts);
  if (r->topk_groups < 1 || r->topk_groups > r->num_groups)
    return failf(EP_ERR_INVALID_ARG, "topk_groups %d outside [1, num_groups %d]", r->topk_groups,
                 r->num_groups);
  if (r->topk_groups * (r->num_experts / r->num_groups) < r->num_topk)
    return failf(EP_ERR_INVALID_ARG, "%d groups of %d experts hold fewer than num_topk %d",
                 r->topk_groups, r->num_experts / r->num_groups, r->num_topk);
  if (r->group_topn != 1 && r->group_topn != 2)
    return failf(EP_ERR_INVALID_ARG, "group_topn %d must be 1 or 2", r->group_topn);
  if (!isfinite(r->scale)) return failf(EP_ERR_INVALID_ARG, "scale is not finite");
  // one workgroup per few tokens of 256 lanes, and fewer than 2^32 lanes
  const int64_t lanes = (int64_t)r->num_tokens * lanes_per_token(r->num_experts);
  if (lanes > (int64_t{1} << 32) - 2 * kThreads)
    return failf(EP_ERR_INVALID_ARG, "num_tokens %d too large: at most 2^32 lanes fit one launch",
                 r->num_tokens);
  return EP_OK;
}

ep_status_t check_logits(const ep_router_t *r, ep_dtype_t dtype, const void *logits,
                         const char *name) {
  if (dtype != EP_DTYPE_F32 && dtype != EP_DTYPE_BF16)
    return failf(EP_ERR_INVALID_ARG, "logits dtype %d must be fp32 or bf16", (int)dtype);
  if (r->num_tokens > 0 && logits == nullptr)
    return failf(EP_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned_to(logits, dtype == EP_DTYPE_F32 ? 4 : 2))
    return failf(EP_ERR_INVALID_ARG, "%s is not aligned to its type", name);
  return EP_OK;
}

bool vector_rows(const ep_router_t *r, ep_dtype_t dtype, const void *p) {
  return r->num_experts % kQuad == 0 && aligned_to(p, dtype == EP_DTYPE_F32 ? 16 : 8);
}

struct BalanceLayout {
  int64_t tiles, rows, blocks;
  size_t part_p, part_c, part_n, seq_loss, total;
};

BalanceLayout balance_layout(int64_t T, int64_t E, int64_t S) {
  BalanceLayout w;
  const auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  const int tile = balance_tile(T);
  w.tiles = (T + tile - 1) / tile;
  w.blocks = (E + kSeqCols - 1) / kSeqCols;
  w.rows = w.tiles + S;
  w.part_p = 0;
  w.part_c = up(w.part_p + sizeof(float) * w.rows * E);
  w.part_n = up(w.part_c + sizeof(int32_t) * w.rows * E);
  w.seq_loss = up(w.part_n + sizeof(int32_t) * w.rows);
  w.total = up(w.seq_loss + sizeof(double) * S * w.blocks);
  return w;
}

ep_status_t check_seqs(int32_t num_seqs) {
  if (num_seqs < 1 || num_seqs >= (1 << 21))
    return failf(EP_ERR_INVALID_ARG, "num_seqs %d outside [1, 2^21)", num_seqs);
  return EP_OK;
}

}  // namespace
}  // namespace ep

extern "C" {

ep_status_t ep_route(const ep_router_t *router, ep_dtype_t logits_dtype, const void *logits,
                     const float *bias, const uint8_t *token_mask, int32_t *topk_idx,
                     float *topk_weights, int32_t *status, hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_router(router));
  EP_TRY(check_logits(router, logits_dtype, logits, "logits"));
  if (router->num_tokens == 0) return EP_OK;
  if (topk_idx == nullptr || topk_weights == nullptr || status == nullptr)
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.token_mask = token_mask;
  a.topk_idx = topk_idx;
  a.topk_weights = topk_weights;
  a.status = status;
  a.T = router->num_tokens;
  a.E = router->num_experts;
  a.k = router->num_topk;
  a.G = router->num_groups;
  a.group_size = router->num_experts / router->num_groups;
  a.topk_groups = router->topk_groups;
  a.group_topn = router->group_topn;
  a.group_inv = ((1u << 22) + a.group_size - 1) / a.group_size;
  a.softmax = router->score == EP_SCORE_SOFTMAX;
  a.normalize = router->normalize != 0;
  const bool by_logit = bias == nullptr && (a.G == 1 || a.group_topn == 1);
  a.vec = vector_rows(router, logits_dtype, logits);
  a.scale = router->scale;
  a.group_steps = -1;
  const int lanes = lanes_per_token(a.E);
  for (int s = 0; (1 << s) <= lanes && a.G > 1; ++s)
    if (a.group_size == kQuad << s) a.group_steps = s;
  with_row_shape(a.E, [&](auto lpt, auto v) {
    const int64_t need = (a.T + kThreads / lpt.value - 1) / (kThreads / lpt.value);
    const dim3 grid((unsigned)(need < kRouteGrid ? need : kRouteGrid));
    const auto launch = [&](auto type, auto mode) {
      if (a.k <= kList)
        hipLaunchKernelGGL(
            (route_kernel<decltype(type), lpt.value, v.value, mode.value, true>), grid,
            dim3(kThreads), 0, stream, a);
      else
        hipLaunchKernelGGL(
            (route_kernel<decltype(type), lpt.value, v.value, mode.value, false>), grid,
            dim3(kThreads), 0, stream, a);
    };
    const auto by_mode = [&](auto type) {
      if (by_logit)
        launch(type, std::integral_constant<int, kByLogit>{});
      else if (a.softmax)
        launch(type, std::integral_constant<int, kBySoftmax>{});
      else
        launch(type, std::integral_constant<int, kBySigmoid>{});
    };
    if (logits_dtype == EP_DTYPE_F32)
      by_mode(float{});
    else
      by_mode(uint16_t{});
  });
  return launched("route launch");
}

ep_status_t ep_balance_workspace_bytes(const ep_router_t *router, int32_t num_seqs,
                                       size_t *bytes_host) {
  using namespace ep;
  EP_TRY(check_router(router));
  EP_TRY(check_seqs(num_seqs));
  if (bytes_host == nullptr) return failf(EP_ERR_INVALID_ARG, "bytes_host is NULL");
  *bytes_host = balance_layout(router->num_tokens, router->num_experts, num_seqs).total;
  return EP_OK;
}

ep_status_t ep_balance_loss(const ep_router_t *router, ep_dtype_t logits_dtype,
                            const void *logits, const int32_t *topk_idx,
                            const int32_t *seq_offsets, int32_t num_seqs, float coef,
                            void *workspace, size_t workspace_bytes, int32_t *counts,
                            int32_t *seq_tokens, float *mean_probs, float *prob_grad, float *loss,
                            int32_t *status, hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_router(router));
  EP_TRY(check_logits(router, logits_dtype, logits, "logits"));
  EP_TRY(check_seqs(num_seqs));
  if (seq_offsets == nullptr && num_seqs != 1)
    return failf(EP_ERR_INVALID_ARG, "num_seqs %d needs seq_offsets", num_seqs);
  if (!isfinite(coef)) return failf(EP_ERR_INVALID_ARG, "coef is not finite");
  if ((router->num_tokens > 0 && topk_idx == nullptr) || workspace == nullptr ||
      counts == nullptr || seq_tokens == nullptr || mean_probs == nullptr ||
      prob_grad == nullptr || loss == nullptr || status == nullptr)
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  const BalanceLayout w = balance_layout(router->num_tokens, router->num_experts, num_seqs);
  if (workspace_bytes < w.total)
    return failf(EP_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", workspace_bytes,
                 w.total);
  if (!aligned_to(workspace, 256))
    return failf(EP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  char *ws = static_cast<char *>(workspace);
  BalanceArgs a;
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.seq_offsets = seq_offsets;
  a.T = router->num_tokens;
  a.E = router->num_experts;
  a.k = router->num_topk;
  a.S = num_seqs;
  a.tile = balance_tile(a.T);
  a.seq_blocks = (int32_t)w.blocks;
  a.softmax = router->score == EP_SCORE_SOFTMAX;
  a.vec = vector_rows(router, logits_dtype, logits);
  a.coef = coef;
  a.part_p = reinterpret_cast<float *>(ws + w.part_p);
  a.part_c = reinterpret_cast<int32_t *>(ws + w.part_c);
  a.part_n = reinterpret_cast<int32_t *>(ws + w.part_n);
  a.seq_loss = reinterpret_cast<double *>(ws + w.seq_loss);
  a.counts = counts;
  a.seq_tokens = seq_tokens;
  a.mean_probs = mean_probs;
  a.prob_grad = prob_grad;
  a.loss = loss;
  a.status = status;
  if (w.tiles > 0)
    with_row_shape(a.E, [&](auto lpt, auto v) {
      const dim3 grid((unsigned)w.tiles);
      const auto launch = [&](auto type, auto softmax) {
        hipLaunchKernelGGL(
            (balance_tile_kernel<decltype(type), lpt.value, v.value, softmax.value>), grid,
            dim3(kThreads), 0, stream, a);
      };
      if (logits_dtype == EP_DTYPE_F32 && a.softmax)
        launch(float{}, std::true_type{});
      else if (logits_dtype == EP_DTYPE_F32)
        launch(float{}, std::false_type{});
      else if (a.softmax)
        launch(uint16_t{}, std::true_type{});
      else
        launch(uint16_t{}, std::false_type{});
    });
  hipLaunchKernelGGL(balance_seq_kernel, dim3((unsigned)num_seqs, (unsigned)w.blocks),
                     dim3(kSeqThreads), 0, stream, a);
  hipLaunchKernelGGL(balance_loss_kernel,
                     dim3((unsigned)(num_seqs < kLossGrid ? num_seqs : kLossGrid)),
                     dim3(kThreads), 0, stream, a);
  return launched("balance loss launch");
}

ep_status_t ep_route_backward(const ep_router_t *router, ep_dtype_t logits_dtype,
                              const void *logits, const int32_t *topk_idx,
                              const float *grad_weights, const float *prob_grad,
                              const int32_t *seq_offsets, int32_t num_seqs,
                              const float *grad_loss, void *grad_logits, int32_t *status,
                              hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_router(router));
  EP_TRY(check_logits(router, logits_dtype, logits, "logits"));
  EP_TRY(check_logits(router, logits_dtype, grad_logits, "grad_logits"));
  if (prob_grad != nullptr) {
    EP_TRY(check_seqs(num_seqs));
    if (seq_offsets == nullptr && num_seqs != 1)
      return failf(EP_ERR_INVALID_ARG, "num_seqs %d needs seq_offsets", num_seqs);
  }
  if (router->num_tokens == 0) return EP_OK;
  if (topk_idx == nullptr || status == nullptr)
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  GradArgs a;
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.grad_weights = grad_weights;
  a.prob_grad = prob_grad;
  a.seq_offsets = seq_offsets;
  a.grad_loss = grad_loss;
  a.grad_logits = grad_logits;
  a.status = status;
  a.T = router->num_tokens;
  a.E = router->num_experts;
  a.k = router->num_topk;
  a.S = num_seqs;
  a.normalize = router->normalize != 0;
  a.vec = vector_rows(router, logits_dtype, logits) &&
          vector_rows(router, logits_dtype, grad_logits);
  a.vec_q = vector_rows(router, EP_DTYPE_F32, prob_grad);
  a.scale = router->scale;
  const bool softmax = router->score == EP_SCORE_SOFTMAX;
  with_row_shape(a.E, [&](auto lpt, auto v) {
    const int64_t once = kThreads / lpt.value;
    a.passes = a.T > once * kGradPasses * kGradFew ? kGradPasses : 1;
    const int64_t tokens = once * a.passes;
    const dim3 grid((unsigned)((a.T + tokens - 1) / tokens));
    const auto launch = [&](auto type, auto soft) {
      if (prob_grad != nullptr)
        hipLaunchKernelGGL(
            (route_backward_kernel<decltype(type), lpt.value, v.value, soft.value, true>), grid,
            dim3(kThreads), 0, stream, a);
      else
        hipLaunchKernelGGL(
            (route_backward_kernel<decltype(type), lpt.value, v.value, soft.value, false>), grid,
            dim3(kThreads), 0, stream, a);
    };
    if (logits_dtype == EP_DTYPE_F32 && softmax)
      launch(float{}, std::true_type{});
    else if (logits_dtype == EP_DTYPE_F32)
      launch(float{}, std::false_type{});
    else if (softmax)
      launch(uint16_t{}, std::true_type{});
    else
      launch(uint16_t{}, std::false_type{});
  });
  return launched("route backward launch");
}

}  // extern "C"
