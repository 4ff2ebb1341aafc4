// The experts' products with bf16 weights for gfx950, and their gradients for
// the rows and for the weights.  Contracts in include/ep_moe.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ep.h"
#include "ep_host.h"
#include "ep_moe.h"
#include "ep_rows.h"

namespace ep {
namespace {

// What a product multiplies.  A matrix is named by its place in
// c[m, n] = sum_l a[m, l] b[n, l]:
//   product         a = x [rows, K],        b = w [N, K],          l = K
//   rows' gradient  a = grad_out [rows, N], b = w, read [l, n],    l = N
//   weights'        a = grad_out, [l, m],   b = x, [l, n],         l = rows
enum Kind { kProduct = 0, kRowsGrad = 1, kWeightsGrad = 2 };

struct ProductArgs {
  ExpertRows rows;
  const void *x;          // product and weights' gradient
  const float *x_scales;  // of FP8 rows
  const uint16_t *w;      // product and rows' gradient
  const uint16_t *grad;   // gradients: of the product's output
  const void *add;        // weights' gradient, or NULL
  void *out;
  int32_t K, N;
};

__device__ __forceinline__ f32x4 mul(bf16x8 x, bf16x8 w, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
}

// A value of an FP8 row as it enters the products.
__device__ __forceinline__ uint16_t fp8_bf16(uint8_t code, float scale) {
  return f32_to_bf16(__builtin_amdgcn_cvt_f32_fp8((int)code, 0) * scale);
}

// Any sizes and alignments: tiles of 64 x 64 x 32, loaded value by value.
constexpr int kAnyTile = 64, kAnyDepth = 32, kAnyGrid = 1024;

template <Kind KIND, bool FP8, bool SWIGLU, typename OUT>
__global__ __launch_bounds__(256) void product_any_kernel(ProductArgs a) {
  __shared__ __align__(16) uint16_t as[kAnyTile][kAnyDepth + 8], bs[kAnyTile][kAnyDepth + 8];
  __shared__ int32_t starts[EP_MAX_EXPERTS + 1], totals[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int E = a.rows.E, K = a.K, N = a.N;
  const uint8_t *x8 = static_cast<const uint8_t *>(a.x);
  const uint16_t *x16 = static_cast<const uint16_t *>(a.x);
  const int out_cols = KIND == kProduct ? (SWIGLU ? N / 2 : N) : K;
  constexpr int kCols = SWIGLU ? kAnyTile / 2 : kAnyTile;  // output columns of a tile
  const int col_tiles = (out_cols + kCols - 1) / kCols;
  const int row_tiles = (N + kAnyTile - 1) / kAnyTile;  // weights' gradient
  int64_t items;
  if (KIND == kWeightsGrad) {
    items = (int64_t)E * row_tiles * col_tiles;
  } else {
    number_blocks(a.rows, starts, totals,
                  [](int64_t rows) { return (rows + kAnyTile - 1) / kAnyTile; });
    items = (int64_t)starts[E] * col_tiles;
  }
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int n0 = (int)(item % col_tiles) * kCols;
    const int64_t block = item / col_tiles;
    int e, m0;
    int64_t first, rows;
    if (KIND == kWeightsGrad) {
      e = (int)(block / row_tiles);
      m0 = (int)(block % row_tiles) * kAnyTile;
      rows_inside(a.rows.offsets[e], a.rows.counts[e], a.rows.capacity, &first, &rows);
    } else {
      e = expert_of(starts, E, (int32_t)block);
      rows_inside(a.rows.offsets[e], a.rows.counts[e], a.rows.capacity, &first, &rows);
      const int64_t skip = (block - starts[e]) * kAnyTile;
      first += skip;
      rows -= skip;
      m0 = 0;
    }
    const int64_t length = KIND == kProduct ? K : KIND == kRowsGrad ? N : rows;
    const uint16_t *w = a.w + (int64_t)e * N * K;
    const auto a_value = [&](int m, int64_t l) -> uint16_t {
      if (l >= length) return 0;
      if (KIND == kProduct) {
        if (m >= rows) return 0;
        if (FP8)
          return fp8_bf16(x8[(first + m) * K + l], a.x_scales[(first + m) * (K / 128) + l / 128]);
        return x16[(first + m) * K + l];
      }
      if (KIND == kRowsGrad) return m < rows ? a.grad[(first + m) * N + l] : (uint16_t)0;
      return m0 + m < N ? a.grad[(first + l) * N + m0 + m] : (uint16_t)0;
    };
    const auto b_value = [&](int n, int64_t l) -> uint16_t {
      if (l >= length) return 0;
      if (KIND == kProduct) {
        const int c = n0 + n % kCols;
        return c < out_cols ? w[(int64_t)(c + n / kCols * out_cols) * K + l] : (uint16_t)0;
      }
      const int c = n0 + n;
      if (c >= K) return 0;
      if (KIND == kRowsGrad) return w[l * K + c];
      if (FP8)
        return fp8_bf16(x8[(first + l) * K + c], a.x_scales[(first + l) * (K / 128) + c / 128]);
      return x16[(first + l) * K + c];
    };
    f32x4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f32x4{0, 0, 0, 0};
    for (int64_t l0 = 0; l0 < length; l0 += kAnyDepth) {
      for (int i = tid; i < kAnyTile * kAnyDepth; i += 256) {
        // neighbouring threads read neighbouring values
        const int across = i % kAnyTile, al = i / kAnyTile;
        const int along = i % kAnyDepth, am = i / kAnyDepth;
        if (KIND == kWeightsGrad)
          as[across][al] = a_value(across, l0 + al);
        else
          as[am][along] = a_value(am, l0 + along);
        if (KIND == kProduct)
          bs[am][along] = b_value(am, l0 + along);
        else
          bs[across][al] = b_value(across, l0 + al);
      }
      __syncthreads();
      const bf16x8 av = *reinterpret_cast<const bf16x8 *>(&as[wave * 16 + col][quad * 8]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i] = mul(av, *reinterpret_cast<const bf16x8 *>(&bs[i * 16 + col][quad * 8]), acc[i]);
      __syncthreads();
    }
    constexpr int kOut = SWIGLU ? 2 : 4;
#pragma unroll
    for (int i = 0; i < kOut; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int m = wave * 16 + quad * 4 + v, c = n0 + i * 16 + col;
        if (c >= out_cols || (KIND == kWeightsGrad ? m0 + m >= N : m >= rows)) continue;
        float y = acc[i][v];
        if (SWIGLU) y = silu_of(y) * acc[2 + i][v];
        const int64_t at = KIND == kWeightsGrad ? ((int64_t)e * N + m0 + m) * K + c
                                                : (first + m) * out_cols + c;
        if constexpr (std::is_same<OUT, float>::value) {
          if (a.add != nullptr) y += static_cast<const float *>(a.add)[at];
          static_cast<float *>(a.out)[at] = y;
        } else {
          if (KIND == kWeightsGrad && a.add != nullptr)
            y += bf16_to_f32(static_cast<const uint16_t *>(a.add)[at]);
          static_cast<uint16_t *>(a.out)[at] = f32_to_bf16(y);
        }
      }
  }
}

#define EP_TRY(expr)                \
  do {                              \
    const ep_status_t st_ = (expr); \
    if (st_ != EP_OK) return st_;   \
  } while (0)

// The checks that the three calls share.
ep_status_t check_experts(const ep_experts_t *x, const int32_t *offsets, const int32_t *counts,
                          int64_t capacity) {
  if (x == nullptr) return failf(EP_ERR_INVALID_ARG, "experts is NULL");
  if (x->num_experts < 1 || x->num_experts > EP_MAX_EXPERTS)
    return failf(EP_ERR_INVALID_ARG, "num_experts %d outside [1, %d]", x->num_experts,
                 EP_MAX_EXPERTS);
  if (x->in_features < 1 || x->in_features >= (1 << 20))
    return failf(EP_ERR_INVALID_ARG, "in_features %d outside [1, 2^20)", x->in_features);
  if (x->out_features < 1 || x->out_features >= (1 << 20))
    return failf(EP_ERR_INVALID_ARG, "out_features %d outside [1, 2^20)", x->out_features);
  if (capacity < 0 || capacity >= INT32_MAX)
    return failf(EP_ERR_INVALID_ARG, "capacity %lld outside [0, 2^31 - 1)", (long long)capacity);
  // the row blocks of all experts are numbered in 32 bits, each expert's at most the buffer's
  if ((capacity / 64 + 1) * x->num_experts >= INT32_MAX)
    return failf(EP_ERR_INVALID_ARG, "capacity %lld x %d experts has too many row blocks",
                 (long long)capacity, x->num_experts);
  if (offsets == nullptr || counts == nullptr)
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  return EP_OK;
}

// x and its scales; NULL where there are no rows.
ep_status_t check_x(const ep_experts_t *experts, ep_dtype_t dtype, const void *x,
                    const float *x_scales, int64_t capacity) {
  if (dtype != EP_DTYPE_BF16 && dtype != EP_DTYPE_FP8_E4M3)
    return failf(EP_ERR_INVALID_ARG, "x dtype %d must be bf16 or FP8", (int)dtype);
  const bool fp8 = dtype == EP_DTYPE_FP8_E4M3;
  if (fp8 && experts->in_features % 128 != 0)
    return failf(EP_ERR_INVALID_ARG, "FP8 rows need in_features %% 128 == 0 (in_features %d)",
                 experts->in_features);
  if (capacity > 0 && (x == nullptr || (fp8 && x_scales == nullptr)))
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned_to(x, 16) || !aligned_to(x_scales, 4))
    return failf(EP_ERR_INVALID_ARG, "x must be 16-byte, x_scales 4-byte aligned");
  return EP_OK;
}

bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && p < q + (uintptr_t)b_bytes && q < p + (uintptr_t)a_bytes;
}

int64_t weight_values(const ep_experts_t *x) {
  return (int64_t)x->num_experts * x->in_features * x->out_features;
}

ProductArgs product_args(const ep_experts_t *x, const int32_t *offsets, const int32_t *counts,
                         int64_t capacity) {
  ProductArgs a = {};
  a.rows = ExpertRows{offsets, counts, capacity, x->num_experts};
  a.K = x->in_features;
  a.N = x->out_features;
  return a;
}

}  // namespace
}  // namespace ep

extern "C" {

ep_status_t ep_expert_product(const ep_experts_t *experts, ep_dtype_t x_dtype, const void *x,
                              const float *x_scales, const uint16_t *w, int32_t swiglu,
                              const int32_t *expert_offsets, const int32_t *num_tokens_per_expert,
                              int64_t capacity, uint16_t *out, hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_experts(experts, expert_offsets, num_tokens_per_expert, capacity));
  EP_TRY(check_x(experts, x_dtype, x, x_scales, capacity));
  const int K = experts->in_features, N = experts->out_features;
  if (swiglu && N % 2 != 0)
    return failf(EP_ERR_INVALID_ARG, "SwiGLU needs an even out_features (%d)", N);
  if (w == nullptr || (capacity > 0 && out == nullptr))
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned_to(w, 16) || !aligned_to(out, 2))
    return failf(EP_ERR_INVALID_ARG, "w must be 16-byte, out 2-byte aligned");
  if (capacity == 0) return EP_OK;
  const bool fp8 = x_dtype == EP_DTYPE_FP8_E4M3;
  const int64_t out_bytes = capacity * (swiglu ? N / 2 : N) * 2;
  if (overlap(out, out_bytes, x, capacity * K * (fp8 ? 1 : 2)) ||
      overlap(out, out_bytes, x_scales, fp8 ? capacity * (K / 128) * 4 : 0) ||
      overlap(out, out_bytes, w, weight_values(experts) * 2))
    return failf(EP_ERR_INVALID_ARG, "out overlaps an input");
  ProductArgs a = product_args(experts, expert_offsets, num_tokens_per_expert, capacity);
  a.x = x;
  a.x_scales = x_scales;
  a.w = w;
  a.out = out;
  const auto launch = [&](auto f, auto s) {
    hipLaunchKernelGGL((product_any_kernel<kProduct, f.value, s.value, uint16_t>), dim3(kAnyGrid),
                       dim3(256), 0, stream, a);
  };
  const auto by_swiglu = [&](auto f) {
    if (swiglu)
      launch(f, std::true_type{});
    else
      launch(f, std::false_type{});
  };
  if (fp8)
    by_swiglu(std::true_type{});
  else
    by_swiglu(std::false_type{});
  return launched("expert product launch");
}

ep_status_t ep_expert_product_backward_rows(const ep_experts_t *experts, const uint16_t *grad_out,
                                            const uint16_t *w, const int32_t *expert_offsets,
                                            const int32_t *num_tokens_per_expert,
                                            int64_t capacity, uint16_t *grad_x,
                                            hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_experts(experts, expert_offsets, num_tokens_per_expert, capacity));
  if (w == nullptr || (capacity > 0 && (grad_out == nullptr || grad_x == nullptr)))
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned_to(w, 16) || !aligned_to(grad_out, 16) || !aligned_to(grad_x, 2))
    return failf(EP_ERR_INVALID_ARG, "w and grad_out must be 16-byte, grad_x 2-byte aligned");
  if (capacity == 0) return EP_OK;
  const int64_t out_bytes = capacity * experts->in_features * 2;
  if (overlap(grad_x, out_bytes, grad_out, capacity * experts->out_features * 2) ||
      overlap(grad_x, out_bytes, w, weight_values(experts) * 2))
    return failf(EP_ERR_INVALID_ARG, "grad_x overlaps an input");
  ProductArgs a = product_args(experts, expert_offsets, num_tokens_per_expert, capacity);
  a.w = w;
  a.grad = grad_out;
  a.out = grad_x;
  hipLaunchKernelGGL((product_any_kernel<kRowsGrad, false, false, uint16_t>), dim3(kAnyGrid),
                     dim3(256), 0, stream, a);
  return launched("expert rows' gradient launch");
}

ep_status_t ep_expert_product_backward_weights(
    const ep_experts_t *experts, ep_dtype_t x_dtype, const void *x, const float *x_scales,
    const uint16_t *grad_out, const int32_t *expert_offsets, const int32_t *num_tokens_per_expert,
    int64_t capacity, ep_dtype_t grad_dtype, const void *add, void *grad_w, hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_experts(experts, expert_offsets, num_tokens_per_expert, capacity));
  EP_TRY(check_x(experts, x_dtype, x, x_scales, capacity));
  if (grad_dtype != EP_DTYPE_BF16 && grad_dtype != EP_DTYPE_F32)
    return failf(EP_ERR_INVALID_ARG, "gradient dtype %d must be bf16 or fp32", (int)grad_dtype);
  if (grad_w == nullptr || (capacity > 0 && grad_out == nullptr))
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned_to(grad_out, 16) || !aligned_to(add, 16) || !aligned_to(grad_w, 16))
    return failf(EP_ERR_INVALID_ARG, "grad_out, add and grad_w must be 16-byte aligned");
  const bool fp8 = x_dtype == EP_DTYPE_FP8_E4M3, f32 = grad_dtype == EP_DTYPE_F32;
  const int K = experts->in_features, N = experts->out_features;
  const int64_t out_bytes = weight_values(experts) * (f32 ? 4 : 2);
  if (overlap(grad_w, out_bytes, x, capacity * K * (fp8 ? 1 : 2)) ||
      overlap(grad_w, out_bytes, x_scales, fp8 ? capacity * (K / 128) * 4 : 0) ||
      overlap(grad_w, out_bytes, grad_out, capacity * N * 2) ||
      (add != grad_w && overlap(grad_w, out_bytes, add, out_bytes)))
    return failf(EP_ERR_INVALID_ARG, "grad_w overlaps an input");
  ProductArgs a = product_args(experts, expert_offsets, num_tokens_per_expert, capacity);
  a.x = x;
  a.x_scales = x_scales;
  a.grad = grad_out;
  a.add = add;
  a.out = grad_w;
  const auto launch = [&](auto f, auto value) {
    hipLaunchKernelGGL((product_any_kernel<kWeightsGrad, f.value, false, decltype(value)>),
                       dim3(kAnyGrid), dim3(256), 0, stream, a);
  };
  const auto by_type = [&](auto f) {
    if (f32)
      launch(f, float{});
    else
      launch(f, uint16_t{});
  };
  if (fp8)
    by_type(std::true_type{});
  else
    by_type(std::false_type{});
  return launched("expert weights' gradient launch");
}

}  // extern "C"
