// The router's kernels for gfx950: top-k selection, the load-balance loss,
// and the gradient of both for the logits.  Contracts in include/ep_moe.h.
//
// A token's row of E logits belongs to LPT lanes of one wave, V values each
// (four consecutive ones at a time, so a row is read in 16-byte pieces):
// element i of lane l is expert (i / 4) * 4 * LPT + 4 * l + i % 4.  Rows
// stay in registers from the load to the result.
#include <hip/hip_runtime.h>
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
// to a piece (E % 4 == 0 and an aligned base).
template <int LPT, int V>
__device__ __forceinline__ void load_row(const float *row, int E, int l, bool vec, float (&x)[V]) {
#pragma unroll
  for (int q = 0; q < V / kQuad; ++q) {
    const int e = expert_of<LPT, V>(l, q * kQuad);
    if (vec) {
      f32x4 v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (e < E) v = *reinterpret_cast<const f32x4 *>(row + e);
#pragma unroll
      for (int i = 0; i < kQuad; ++i) x[q * kQuad + i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < kQuad; ++i) x[q * kQuad + i] = e + i < E ? row[e + i] : -INFINITY;
    }
  }
}

template <int LPT, int V>
__device__ __forceinline__ void load_row(const uint16_t *row, int E, int l, bool vec,
                                         float (&x)[V]) {
#pragma unroll
  for (int q = 0; q < V / kQuad; ++q) {
    const int e = expert_of<LPT, V>(l, q * kQuad);
    if (vec) {
      u16x4 v = {0xFF80, 0xFF80, 0xFF80, 0xFF80};
      if (e < E) v = *reinterpret_cast<const u16x4 *>(row + e);
#pragma unroll
      for (int i = 0; i < kQuad; ++i) x[q * kQuad + i] = bf16_to_f32(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kQuad; ++i)
        x[q * kQuad + i] = e + i < E ? bf16_to_f32(row[e + i]) : -INFINITY;
    }
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

__device__ __forceinline__ float logit_at(const float *row, int e) { return row[e]; }
__device__ __forceinline__ float logit_at(const uint16_t *row, int e) {
  return bf16_to_f32(row[e]);
}

// Reductions over the LPT lanes of a token: every lane gets the same result,
// in a fixed order.
template <int LPT, typename T>
__device__ __forceinline__ T token_max(T v) {
#pragma unroll
  for (int m = 1; m < LPT; m *= 2) {
    const T o = __shfl_xor(v, m);
    v = o > v ? o : v;
  }
  return v;
}

template <int LPT, typename T>
__device__ __forceinline__ T token_sum(T v) {
#pragma unroll
  for (int m = 1; m < LPT; m *= 2) v += __shfl_xor(v, m);
  return v;
}

template <int LPT>
__device__ __forceinline__ int token_or(int v) {
#pragma unroll
  for (int m = 1; m < LPT; m *= 2) v |= __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// sigmoid(x) / exp(m) with m = min(0, the largest x in play), so that scores
// whose largest would underflow keep their ratios: for x <= 0,
// exp(x - m) / (1 + exp(x)).
__device__ __forceinline__ float sigmoid_over(float x, float m) {
  const float t = exp_of(-fabsf(x));
  const float num = x > 0.0f ? 1.0f : (m == 0.0f ? t : exp_of(x - m));
  return num / (1.0f + t);
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
  uint32_t group_inv;  // ceil(2^22 / group_size): e / group_size = e * group_inv >> 22
  bool softmax, normalize, by_logit, vec;
  float scale;
};

// Groups of one token kept by its keys, as 64 bits.  Lane l reads the keys
// of groups l, l + LPT, ... from LDS.  near: a kept and a dropped group are
// within `margin` of each other.
template <typename K, int LPT, int V>
__device__ __forceinline__ uint64_t kept_groups(const RouteArgs &a, const K (&key)[V], int l,
                                                K *row, K *group_key, K margin, bool *near) {
  const K none = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert_of<LPT, V>(l, i);
    if (e < a.E) row[e] = key[i];
  }
  wave_sync();
  for (int g = l; g < a.G; g += LPT) {
    K best = none, second = none;
    for (int i = 0; i < a.group_size; ++i) {
      const K v = row[g * a.group_size + i];
      second = v > best ? best : (v > second ? v : second);
      best = v > best ? v : best;
    }
    group_key[g] = a.group_topn == 2 && second > none ? best + second : best;
  }
  wave_sync();
  uint64_t kept = 0;
  K low = INFINITY, high = none;  // worst kept, best dropped
  for (int g = 0; g < a.G; ++g) {
    const K v = group_key[g];
    int before = 0;
    for (int h = 0; h < a.G; ++h) {
      const K o = group_key[h];
      before += o > v || (o == v && h < g);
    }
    if (!(v > none)) continue;
    if (before < a.topk_groups) {
      kept |= uint64_t{1} << g;
      low = v < low ? v : low;
    } else {
      high = v > high ? v : high;
    }
  }
  wave_sync();
  if (near != nullptr && high > none && !(low - high > margin)) *near = true;
  return kept;
}

// The k best of one token's keys, in order; slot j is given to lane j % LPT
// as its mine[j / LPT].  A key of -inf is never selected.  near: two
// neighbours in the order, the first one not selected among them, are within
// `margin`.
template <typename K, int LPT, int V>
__device__ __forceinline__ void best_experts(const RouteArgs &a, K (&key)[V], int l,
                                             int (&mine)[2], K margin, bool *near) {
  const K none = -INFINITY;
  mine[0] = mine[1] = -1;
  K last = INFINITY;
  const int rounds = near != nullptr ? a.k + 1 : a.k;
  for (int j = 0; j < rounds; ++j) {
    K best = none;
    int at = 1 << 20;
#pragma unroll
    for (int i = 0; i < V; ++i)  // experts ascend with i: the first of equals stays
      if (key[i] > best) {
        best = key[i];
        at = expert_of<LPT, V>(l, i);
      }
#pragma unroll
    for (int m = 1; m < LPT; m *= 2) {
      const K o = __shfl_xor(best, m);
      const int oat = __shfl_xor(at, m);
      if (o > best || (o == best && oat < at)) {
        best = o;
        at = oat;
      }
    }
    if (!(best > none)) break;
    if (near != nullptr && !(last - best > margin)) *near = true;
    last = best;
    if (j < a.k && j % LPT == l) mine[j / LPT] = at;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (expert_of<LPT, V>(l, i) == at) key[i] = none;
  }
}

// Selection by keys of type K.
template <typename K, int LPT, int V>
__device__ __forceinline__ void select(const RouteArgs &a, K (&key)[V], int l, char *lds_row,
                                       int (&mine)[2], K margin, bool *near) {
  if (a.G > 1) {
    K *row = reinterpret_cast<K *>(lds_row);
    const uint64_t kept = kept_groups<K, LPT, V>(a, key, l, row, row + LPT * V, margin, near);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int g = (int)(((uint32_t)expert_of<LPT, V>(l, i) * a.group_inv) >> 22);
      if (g >= 64 || !((kept >> g) & 1)) key[i] = -INFINITY;
    }
  }
  best_experts<K, LPT, V>(a, key, l, mine, margin, near);
}

// Keys s + b of one lane's experts (key of a logit of -inf: -inf).
template <typename K, int LPT, int V>
__device__ __forceinline__ void score_keys(const RouteArgs &a, const float (&x)[V], int l,
                                           float xmax, K (&key)[V], K *best_score) {
  K sum = 0;
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = exp_of(K(x[i]) - K(xmax));
      sum += key[i];
    }
    sum = token_sum<LPT>(sum);
    *best_score = K(1) / sum;
  } else {
    *best_score = sigmoid_of(K(xmax));
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert_of<LPT, V>(l, i);
    K s = a.softmax ? key[i] / sum : sigmoid_of(K(x[i]));
    if (a.bias != nullptr && e < a.E) s += K(a.bias[e]);
    key[i] = x[i] > -INFINITY ? s : K(-INFINITY);
  }
}

// One token per LPT lanes.  Bound by the k rounds of the search, not by the
// logits it reads.  Keys other than logits are computed in 32 bits first;
// where neighbours in the order are within 2^-19 of the best score and key the
// token's keys and order are computed again in 64.  (A score is off by at most
// 2^-21.5 of the best, its sum with the bias by 2^-24 of the key; two sums of
// two keys by four times that.)
template <typename L, int LPT, int V>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
  constexpr int kTokens = kThreads / LPT;
  __shared__ __align__(16) char lds[kTokens * (LPT * V + EP_MAX_GROUPS) * sizeof(double)];
  const int l = threadIdx.x % LPT;
  const int slot = threadIdx.x / LPT;
  const int64_t t = (int64_t)blockIdx.x * kTokens + slot;
  char *lds_row = lds + slot * (LPT * V + EP_MAX_GROUPS) * sizeof(double);
  const bool live = t < a.T;
  const bool on = live && (a.token_mask == nullptr || a.token_mask[t] != 0);
  const L *row = static_cast<const L *>(a.logits) + (live ? t : 0) * a.E;
  float x[V];
  if (on) {
    load_row<LPT, V>(row, a.E, l, a.vec, x);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = -INFINITY;
  }
  float xmax = -INFINITY;
  int bad = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bad |= !(x[i] < INFINITY);
    xmax = fmaxf(xmax, x[i]);
  }
  bad = token_or<LPT>(bad);
  xmax = token_max<LPT>(xmax);
  int mine[2] = {-1, -1};
  if (!bad && xmax > -INFINITY) {
    float key[V];
    if (a.by_logit) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = x[i];
      select<float, LPT, V>(a, key, l, lds_row, mine, 0.0f, nullptr);
    } else {
      float best_score;
      score_keys<float, LPT, V>(a, x, l, xmax, key, &best_score);
      float size = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        bad |= !(key[i] < INFINITY);
        if (key[i] > -INFINITY) size = fmaxf(size, fabsf(key[i]));
      }
      bad = token_or<LPT>(bad);
      if (!bad) {
        size = token_max<LPT>(size);
        bool near = false;
        const float margin = 0x1p-19f * (best_score + size);
        select<float, LPT, V>(a, key, l, lds_row, mine, margin, &near);
        if (near) {
          double exact[V], best;
          score_keys<double, LPT, V>(a, x, l, xmax, exact, &best);
          select<double, LPT, V>(a, exact, l, lds_row, mine, 0.0, nullptr);
        }
      }
    }
  }
  if (!live) return;
  if (bad) {
    mine[0] = mine[1] = -1;
    if (l == 0) atomicOr(a.status, EP_STATUS_BIT_NONFINITE);
  }
  // Weights from the selected logits, relative to the largest in play.
  float sx[2];
  float smax = -INFINITY;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    sx[j] = mine[j] >= 0 ? logit_at(row, mine[j]) : -INFINITY;
    smax = fmaxf(smax, sx[j]);
  }
  smax = token_max<LPT>(smax);
  float w[2], total;
  if (a.softmax) {
    const float top = a.normalize ? smax : xmax;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[j] = mine[j] >= 0 ? exp_of(sx[j] - top) : 0.0f;
      sum += w[j];
    }
    if (!a.normalize) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += xmax > -INFINITY ? exp_of(x[i] - xmax) : 0.0f;
    }
    total = token_sum<LPT>(sum);
  } else {
    const float m = a.normalize ? fminf(smax, 0.0f) : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[j] = mine[j] >= 0 ? sigmoid_over(sx[j], m) : 0.0f;
      sum += w[j];
    }
    total = a.normalize ? token_sum<LPT>(sum) : 1.0f;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = j * LPT + l;
    if (at < a.k) {
      a.topk_idx[t * a.k + at] = mine[j];
      a.topk_weights[t * a.k + at] = mine[j] >= 0 ? a.scale * (w[j] / total) : 0.0f;
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
  double *seq_loss;  // [S] sum_e f P
  int32_t *counts, *seq_tokens;
  float *mean_probs, *prob_grad, *loss;
  int32_t *status;
};

__device__ __forceinline__ int64_t seq_bound(const int32_t *offsets, int32_t s, int64_t T) {
  if (offsets == nullptr) return s == 0 ? 0 : T;
  const int64_t o = offsets[s];
  return o < 0 ? 0 : (o > T ? T : o);
}

// The last sequence that starts at or before token t.
__device__ __forceinline__ int seq_of(const int32_t *offsets, int S, int64_t t) {
  if (offsets == nullptr) return 0;
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (offsets[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Probabilities of one token's row; false (p zero) if nothing has a score.
template <int LPT, int V>
__device__ __forceinline__ void probabilities(const float (&x)[V], bool softmax, float (&p)[V]) {
  float xmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) xmax = fmaxf(xmax, x[i]);
  xmax = token_max<LPT>(xmax);
  if (xmax == -INFINITY) {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = 0.0f;
    return;
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    p[i] = softmax ? exp_of(x[i] - xmax) : sigmoid_over(x[i], fminf(xmax, 0.0f));
    sum += p[i];
  }
  const float inv = 1.0f / token_sum<LPT>(sum);
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] *= inv;
}

// One workgroup per tile of tokens.  A tile's part of sequence s goes to row
// tile + s of the partial sums: along the tokens one of the two grows, so
// every part has a row of its own.
template <typename L, int LPT, int V>
__global__ __launch_bounds__(kThreads) void balance_tile_kernel(BalanceArgs a) {
  constexpr int kTokens = kThreads / LPT;
  __shared__ float sums[kTokens * LPT * V];
  __shared__ int32_t cnt[EP_MAX_EXPERTS];
  __shared__ int32_t ntok;
  const int l = threadIdx.x % LPT;
  const int slot = threadIdx.x / LPT;
  const int64_t first = (int64_t)blockIdx.x * a.tile;
  const int64_t end = first + a.tile < a.T ? first + a.tile : a.T;
  int s = seq_of(a.seq_offsets, a.S, first);
  for (int64_t lo = first; lo < end && s < a.S; ++s) {
    int64_t hi = seq_bound(a.seq_offsets, s + 1, a.T);
    hi = hi < end ? hi : end;
    if (hi <= lo) continue;
    for (int e = threadIdx.x; e < a.E; e += kThreads) cnt[e] = 0;
    if (threadIdx.x == 0) ntok = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    int mine = 0;
    for (int64_t t = lo + slot; t < hi; t += kTokens) {
      int any = 0;
      for (int j = l; j < a.k; j += LPT) {
        const int e = a.topk_idx[t * a.k + j];
        if (e >= 0 && e < a.E) {
          any = 1;
          atomicAdd(&cnt[e], 1);
        } else if (e != -1) {
          atomicOr(a.status, EP_STATUS_BIT_ROUTE);
        }
      }
      if (!token_or<LPT>(any)) continue;
      mine += 1;
      float x[V], p[V];
      load_row<LPT, V>(static_cast<const L *>(a.logits) + t * a.E, a.E, l, a.vec, x);
      probabilities<LPT, V>(x, a.softmax, p);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += p[i];
    }
    if (l == 0 && mine > 0) atomicAdd(&ntok, mine);
#pragma unroll
    for (int i = 0; i < V; ++i) sums[slot * LPT * V + expert_of<LPT, V>(l, i)] = acc[i];
    __syncthreads();
    const int64_t out = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      float v = 0.0f;
      for (int g = 0; g < kTokens; ++g) v += sums[g * LPT * V + e];
      a.part_p[out * a.E + e] = v;
      a.part_c[out * a.E + e] = cnt[e];
    }
    if (threadIdx.x == 0) a.part_n[out] = ntok;
    __syncthreads();
    lo = hi;
  }
}

// One workgroup per sequence: adds its parts in order, in 64 bits.
__global__ __launch_bounds__(kThreads) void balance_seq_kernel(BalanceArgs a) {
  __shared__ double red[kThreads];
  const int s = blockIdx.x;
  const int64_t lo = seq_bound(a.seq_offsets, s, a.T);
  const int64_t hi = seq_bound(a.seq_offsets, s + 1, a.T);
  if (threadIdx.x == 0 && a.seq_offsets != nullptr) {
    const int64_t o0 = a.seq_offsets[s], o1 = a.seq_offsets[s + 1];
    if (o0 > o1 || o0 < 0 || o1 > a.T || (s == 0 && o0 != 0) || (s == a.S - 1 && o1 != a.T))
      atomicOr(a.status, EP_STATUS_BIT_SEQS);
  }
  const int64_t first = lo / a.tile + s;
  const int64_t last = lo < hi ? (hi - 1) / a.tile + s : first - 1;
  int n = 0;
  for (int64_t r = first; r <= last; ++r) n += a.part_n[r];
  double dot = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    double p = 0.0;
    int c = 0;
    for (int64_t r = first; r <= last; ++r) {
      p += (double)a.part_p[r * a.E + e];
      c += a.part_c[r * a.E + e];
    }
    const double mean = n > 0 ? p / n : 0.0;
    const double f = n > 0 ? (double)a.E * c / ((double)a.k * n) : 0.0;
    a.counts[(int64_t)s * a.E + e] = c;
    a.mean_probs[(int64_t)s * a.E + e] = (float)mean;
    dot += f * mean;
  }
  red[threadIdx.x] = dot;
  __syncthreads();
  for (int m = kThreads / 2; m > 0; m /= 2) {
    if ((int)threadIdx.x < m) red[threadIdx.x] += red[threadIdx.x + m];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    a.seq_loss[s] = red[0];
    a.seq_tokens[s] = n;
  }
}

// Workgroup s: prob_grad of sequence s; workgroup 0 the loss too.
__global__ __launch_bounds__(kThreads) void balance_loss_kernel(BalanceArgs a) {
  __shared__ double red[kThreads];
  __shared__ int32_t live;
  if (threadIdx.x == 0) live = 0;
  __syncthreads();
  double part = 0.0;
  int mine = 0;
  for (int s = threadIdx.x; s < a.S; s += kThreads) {
    mine += a.seq_tokens[s] > 0;
    part += a.seq_loss[s];
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
  const int s = blockIdx.x;
  const int n = a.seq_tokens[s];
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    const double c = a.counts[(int64_t)s * a.E + e];
    a.prob_grad[(int64_t)s * a.E + e] =
        n > 0 ? (float)(scale * ((double)a.E * c / ((double)a.k * n)) / n) : 0.0f;
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
  int32_t E, k, S;
  bool softmax, normalize, vec;
  float scale;
};

// One token per LPT lanes.  With p the probabilities, q the loss's gradient
// for them and g its own:  d x_e = g p_e (q_e - sum q p), times (1 - s_e) for
// sigmoid scores; the gates' part concerns the selected experts only (and,
// for a softmax that is not normalised over them, -s_e sum s u for all): it
// is spread over the row through LDS.
template <typename L, int LPT, int V>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(GradArgs a) {
  constexpr int kTokens = kThreads / LPT;
  __shared__ float lds[kTokens * LPT * V];
  const int l = threadIdx.x % LPT;
  const int slot = threadIdx.x / LPT;
  const int64_t t = (int64_t)blockIdx.x * kTokens + slot;
  if (t >= a.T) return;
  float *own = lds + slot * LPT * V;
  const L *row = static_cast<const L *>(a.logits) + t * a.E;
  float u[2], sx[2];
  int mine[2], any = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = j * LPT + l;
    int e = at < a.k ? a.topk_idx[t * a.k + at] : -1;
    if (e < -1 || e >= a.E) {
      atomicOr(a.status, EP_STATUS_BIT_ROUTE);
      e = -1;
    }
    mine[j] = e;
    any |= e >= 0;
    u[j] = e >= 0 && a.grad_weights != nullptr ? a.grad_weights[t * a.k + at] : 0.0f;
    sx[j] = e >= 0 ? logit_at(row, e) : -INFINITY;
  }
  any = token_or<LPT>(any);
  float x[V], d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    d[i] = 0.0f;
    own[expert_of<LPT, V>(l, i)] = 0.0f;
  }
  wave_sync();
  if (any) {
    load_row<LPT, V>(row, a.E, l, a.vec, x);
    float xmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) xmax = fmaxf(xmax, x[i]);
    xmax = token_max<LPT>(xmax);
    const float m = fminf(xmax, 0.0f);
    const bool loss = a.prob_grad != nullptr;
    float p[V], sum = 0.0f;
    const bool dense = loss || (a.softmax && !a.normalize);
    if (dense) {
      if (xmax == -INFINITY) xmax = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] = a.softmax ? exp_of(x[i] - xmax) : sigmoid_over(x[i], m);
        sum += p[i];
      }
      sum = token_sum<LPT>(sum);
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= inv;
    }
    // the gates' part, per slot
    if (a.grad_weights != nullptr) {
      float g[2];
      if (a.normalize) {
        float smax = token_max<LPT>(fmaxf(sx[0], sx[1]));
        const float sm = fminf(smax, 0.0f);
        float w[2], tot = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[j] = sx[j] > -INFINITY
                     ? (a.softmax ? exp_of(sx[j] - smax) : sigmoid_over(sx[j], sm))
                     : 0.0f;
          tot += w[j];
        }
        tot = token_sum<LPT>(tot);
        if (!(tot > 0.0f)) tot = 1.0f;  // slots of -inf logits only: no gradient
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[j] /= tot;
          dot += w[j] * u[j];
        }
        dot = token_sum<LPT>(dot);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          g[j] = a.scale * w[j] * (u[j] - dot);
          if (!a.softmax) g[j] *= sigmoid_of(-sx[j]);
        }
      } else if (a.softmax) {
        float s[2], dot = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[j] = sx[j] > -INFINITY ? exp_of(sx[j] - xmax) / sum : 0.0f;
          dot += s[j] * u[j];
        }
        dot = token_sum<LPT>(dot);
#pragma unroll
        for (int j = 0; j < 2; ++j) g[j] = a.scale * s[j] * u[j];
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = -p[i] * (a.scale * dot);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          g[j] = mine[j] < 0 ? 0.0f : a.scale * sigmoid_of(sx[j]) * sigmoid_of(-sx[j]) * u[j];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (mine[j] >= 0) atomicAdd(&own[mine[j]], g[j]);
    }
    wave_sync();
    if (loss) {
      const int s = seq_of(a.seq_offsets, a.S, t);
      const bool inside = t >= seq_bound(a.seq_offsets, s, a.T) &&
                          t < seq_bound(a.seq_offsets, s + 1, a.T);
      if (inside) {
        const float g = a.grad_loss != nullptr ? *a.grad_loss : 1.0f;
        float q[V], dot = 0.0f;
        load_row<LPT, V>(a.prob_grad + (int64_t)s * a.E, a.E, l,
                         a.E % kQuad == 0 && ((uintptr_t)a.prob_grad & 15) == 0, q);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (expert_of<LPT, V>(l, i) < a.E) dot = __builtin_fmaf(q[i], p[i], dot);
        dot = token_sum<LPT>(dot);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (expert_of<LPT, V>(l, i) >= a.E) continue;
          float v = g * p[i] * (q[i] - dot);
          if (!a.softmax) v *= sigmoid_of(-x[i]);
          d[i] += v;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] += own[expert_of<LPT, V>(l, i)];
  }
  store_row<LPT, V>(static_cast<L *>(a.grad_logits) + t * a.E, a.E, l, a.vec, d);
}

// --------------------------------------------------------------------------
// Host side
// --------------------------------------------------------------------------

// Calls f with the lanes per token and values per lane that cover E experts.
template <typename F>
void with_row_shape(int32_t E, F f) {
  using std::integral_constant;
  if (E <= 64)
    f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (E <= 128)
    f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (E <= 256)
    f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else if (E <= 512)
    f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
  else
    f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

int lanes_per_token(int32_t E) { return E <= 256 ? 16 : (E <= 512 ? 32 : 64); }

// Tokens of a balance tile.
constexpr int kBalanceTile = 64;

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
  int64_t tiles, rows;
  size_t part_p, part_c, part_n, seq_loss, total;
};

BalanceLayout balance_layout(int64_t T, int64_t E, int64_t S) {
  BalanceLayout w;
  const auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  w.tiles = (T + kBalanceTile - 1) / kBalanceTile;
  w.rows = w.tiles + S;
  w.part_p = 0;
  w.part_c = up(w.part_p + sizeof(float) * w.rows * E);
  w.part_n = up(w.part_c + sizeof(int32_t) * w.rows * E);
  w.seq_loss = up(w.part_n + sizeof(int32_t) * w.rows);
  w.total = up(w.seq_loss + sizeof(double) * S);
  return w;
}

ep_status_t check_seqs(int32_t num_seqs) {
  if (num_seqs < 1 || num_seqs >= (1 << 24))
    return failf(EP_ERR_INVALID_ARG, "num_seqs %d outside [1, 2^24)", num_seqs);
  return EP_OK;
}

#define EP_TRY(expr)                \
  do {                              \
    const ep_status_t st_ = (expr); \
    if (st_ != EP_OK) return st_;   \
  } while (0)

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
  a.by_logit = bias == nullptr && (a.G == 1 || a.group_topn == 1);
  a.vec = vector_rows(router, logits_dtype, logits);
  a.scale = router->scale;
  with_row_shape(a.E, [&](auto lpt, auto v) {
    const dim3 grid((unsigned)((a.T + kThreads / lpt.value - 1) / (kThreads / lpt.value)));
    if (logits_dtype == EP_DTYPE_F32)
      hipLaunchKernelGGL((route_kernel<float, lpt.value, v.value>), grid, dim3(kThreads), 0,
                         stream, a);
    else
      hipLaunchKernelGGL((route_kernel<uint16_t, lpt.value, v.value>), grid, dim3(kThreads), 0,
                         stream, a);
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
  a.tile = kBalanceTile;
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
      if (logits_dtype == EP_DTYPE_F32)
        hipLaunchKernelGGL((balance_tile_kernel<float, lpt.value, v.value>), grid,
                           dim3(kThreads), 0, stream, a);
      else
        hipLaunchKernelGGL((balance_tile_kernel<uint16_t, lpt.value, v.value>), grid,
                           dim3(kThreads), 0, stream, a);
    });
  hipLaunchKernelGGL(balance_seq_kernel, dim3((unsigned)num_seqs), dim3(kThreads), 0, stream, a);
  hipLaunchKernelGGL(balance_loss_kernel, dim3((unsigned)num_seqs), dim3(kThreads), 0, stream, a);
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
  a.softmax = router->score == EP_SCORE_SOFTMAX;
  a.normalize = router->normalize != 0;
  a.vec = vector_rows(router, logits_dtype, logits) &&
          vector_rows(router, logits_dtype, grad_logits);
  a.scale = router->scale;
  with_row_shape(a.E, [&](auto lpt, auto v) {
    const dim3 grid((unsigned)((a.T + kThreads / lpt.value - 1) / (kThreads / lpt.value)));
    if (logits_dtype == EP_DTYPE_F32)
      hipLaunchKernelGGL((route_backward_kernel<float, lpt.value, v.value>), grid,
                         dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((route_backward_kernel<uint16_t, lpt.value, v.value>), grid,
                         dim3(kThreads), 0, stream, a);
  });
  return launched("route backward launch");
}

}  // extern "C"
