// The experts' products with 4-bit weights for gfx950: packing, and the
// product on expert-major rows.  Contracts and the packed layout in
// include/ep_moe.h.
//
// How 4 bits enter the matrix instructions exactly, without a conversion:
//   bf16 rows: a code q in mantissa bits 3..6 of 0x3F80 is the bf16 1 + q/16,
//     so sum x (1 + q/16) = X + sum(x q)/16 with X = sum x, and
//     sum x (q - z) = 16 (sum x (1 + q/16) - X (1 + z/16));
//   FP8 rows: a code q in the low bits of a byte is the E4M3 number q 2^-9 (a
//     subnormal below 8, the first binade from there), so
//     sum x (q - z) = 2^9 (sum x (q 2^-9) - z 2^-9 X).
// X comes from the same instruction with a matrix of ones, once per row tile.
// Group scales are applied to the fp32 sums of a group.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ep.h"
#include "ep_host.h"
#include "ep_moe.h"

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileN = 16;       // output columns of a weight tile
constexpr int kTileK = 128;      // columns of the sum in a weight tile
constexpr int kTileBytes = 1024;
constexpr int kRows = 16;        // rows of x per matrix instruction

__device__ __forceinline__ float bf16_to_f32(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}

// Nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// By exp(-|y|): exp(-y) of a y below -88 is infinite while silu(y) is still a
// fp32 number.
__device__ __forceinline__ float silu(float y) {
  const float t = expf(-fabsf(y));
  return y * ((y < 0.0f ? t : 1.0f) / (1.0f + t));
}

// --------------------------------------------------------------------------
// Packing
// --------------------------------------------------------------------------

struct PackArgs {
  const uint8_t *codes, *zeros;
  const uint16_t *scales;
  uint8_t *w_codes, *w_zeros;
  uint16_t *w_scales;
  int32_t N, K, group, N16, K128;
};

// One workgroup per 16 rows of one matrix.
__global__ __launch_bounds__(256) void w4_pack_kernel(PackArgs a) {
  const int64_t tile_row = blockIdx.x;  // (expert, half, row tile)
  const int64_t matrix = tile_row / a.N16;
  const int n0 = (int)(tile_row % a.N16) * kTileN;
  const uint8_t *src = a.codes + matrix * a.N * (a.K / 2);
  uint32_t *dst = reinterpret_cast<uint32_t *>(a.w_codes) + tile_row * a.K128 * (kTileBytes / 4);
  for (int i = threadIdx.x; i < a.K128 * (kTileBytes / 4); i += 256) {
    const int w = i % 4, lane = i / 4 % 64, kt = i / 256;
    const int n = n0 + lane % 16;
    const int c = kt * kTileK + w * 32 + lane / 16 * 8;
    uint32_t word = 0;
    if (n < a.N && c < a.K) {  // K is a multiple of 32: 8 columns are in or out
      const uint8_t *p = src + (int64_t)n * (a.K / 2) + c / 2;
      for (int b = 0; b < 4; ++b)
        word |= (uint32_t)(p[b] & 15) << (4 * b) | (uint32_t)(p[b] >> 4) << (16 + 4 * b);
    }
    dst[i] = word;
  }
  const int G = a.K / a.group;
  for (int i = threadIdx.x; i < G * kTileN; i += 256) {
    const int n = n0 + i % kTileN, g = i / kTileN;
    const int64_t from = (matrix * a.N + n) * G + g;
    const int64_t to = tile_row * G * kTileN + i;
    a.w_scales[to] = n < a.N ? a.scales[from] : (uint16_t)0;
    if (a.w_zeros != nullptr) a.w_zeros[to] = n < a.N ? (uint8_t)(a.zeros[from] & 15) : (uint8_t)0;
  }
}

// --------------------------------------------------------------------------
// Product
// --------------------------------------------------------------------------

struct ProductArgs {
  const void *x;
  const float *x_scales;
  const uint8_t *w_codes, *w_zeros;
  const uint16_t *w_scales;
  const int32_t *offsets, *counts;
  uint16_t *out;
  int64_t capacity;
  int32_t N, K, N16, K128;
};

// Rows of expert e inside the buffers.
__device__ __forceinline__ void expert_rows(const ProductArgs &a, int e, int64_t *first,
                                            int64_t *rows) {
  const int64_t o = a.offsets[e], c = a.counts[e];
  *first = o;
  *rows = 0;
  if (o < 0 || c <= 0 || o >= a.capacity) return;
  *rows = c < a.capacity - o ? c : a.capacity - o;
}

// The pairs of codes of one word as bf16 pairs 1 + q/16.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w) {
  u32x4 v;
  v[0] = ((w << 3) & 0x00780078u) | 0x3F803F80u;
  v[1] = ((w >> 1) & 0x00780078u) | 0x3F803F80u;
  v[2] = ((w >> 5) & 0x00780078u) | 0x3F803F80u;
  v[3] = ((w >> 9) & 0x00780078u) | 0x3F803F80u;
  return __builtin_bit_cast(bf16x8, v);
}

// The codes of one word as E4M3 q 2^-9, in the byte order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ long codes_fp8(uint32_t w) {
  const uint64_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  return (long)(lo | hi << 32);
}

// Eight bytes of x in that order.
__device__ __forceinline__ long rows_fp8(uint2 v) {
  const uint64_t lo = __builtin_amdgcn_perm(v.y, v.x, 0x05010400u);
  const uint64_t hi = __builtin_amdgcn_perm(v.y, v.x, 0x07030602u);
  return (long)(lo | hi << 32);
}

// One workgroup: 16 rows of x at a time against kTiles column tiles of one
// expert (with SwiGLU the first half of them gate, the other half up).  Its
// four waves take every fourth piece of the sum and add theirs at the end
// in LDS.
template <bool FP8, int GROUP, bool ZEROS, bool SWIGLU, int kTiles>
__global__ __launch_bounds__(256) void product_kernel(ProductArgs a) {
  constexpr int kHalves = SWIGLU ? 2 : 1;
  constexpr int kOut = kTiles / kHalves;       // column tiles of the output
  constexpr int kGroups = kTileK / GROUP;      // groups in a tile
  constexpr int kPer = GROUP / 32;             // matrix instructions per group
  __shared__ float part[4][kTiles][kRows * kTileN];
  const int e = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, quad = lane >> 4;
  int64_t first, rows;
  expert_rows(a, e, &first, &rows);
  const int G = a.K / GROUP;
  const int ot = blockIdx.x * kOut;
  int64_t tile_row[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    int n = ot + i % kOut;
    n = n < a.N16 ? n : a.N16 - 1;
    tile_row[i] = ((int64_t)e * kHalves + i / kOut) * a.N16 + n;
  }
  for (int64_t r0 = 0; r0 < rows; r0 += kRows) {
    f32x4 acc[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[i] = f32x4{0, 0, 0, 0};
    const int64_t left = rows - r0;
    const int64_t xrow = first + r0 + (col < left ? col : left - 1);
    for (int kt = wave; kt < a.K128; kt += 4) {
      u32x4 w[kTiles];
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        w[i] = *reinterpret_cast<const u32x4 *>(
            a.w_codes + (tile_row[i] * a.K128 + kt) * kTileBytes + lane * 16);
      f32x4 sx;
      if (FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = quad * 4 + i;
          const int64_t r = first + r0 + (m < left ? m : left - 1);
          sx[i] = a.x_scales[r * a.K128 + kt];
        }
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int c0 = kt * kTileK + g * GROUP;
        if (kGroups > 1 && c0 >= a.K) break;
        f32x4 sum = {0, 0, 0, 0}, dot[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) dot[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int c = c0 + j * 32 + quad * 8;
          if (FP8) {
            const long xv = rows_fp8(*reinterpret_cast<const uint2 *>(
                static_cast<const uint8_t *>(a.x) + xrow * a.K + c));
            sum = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(xv, 0x3838383838383838l, sum, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
              dot[i] = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(
                  xv, codes_fp8(w[i][g * kPer + j]), dot[i], 0, 0, 0);
          } else {
            const bf16x8 xv = __builtin_bit_cast(
                bf16x8, *reinterpret_cast<const u32x4 *>(
                            static_cast<const uint16_t *>(a.x) + xrow * a.K + c));
            sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                xv, __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u,
                                                     0x3F803F80u}),
                sum, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
              dot[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  xv, codes_bf16(w[i][g * kPer + j]), dot[i], 0, 0, 0);
          }
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const int64_t at = (tile_row[i] * G + kt * kGroups + g) * kTileN + col;
          const float s = bf16_to_f32(a.w_scales[at]);
          const float z = ZEROS ? (float)a.w_zeros[at] : 8.0f;
          const float zc = FP8 ? z * 0x1p-9f : 1.0f + z * 0x1p-4f;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float d = __builtin_fmaf(-zc, sum[v], dot[i][v]);
            acc[i][v] = __builtin_fmaf(FP8 ? s * 0x1p9f * sx[v] : s * 0x1p4f, d, acc[i][v]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][i][(quad * 4 + v) * kTileN + col] = acc[i][v];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
      const int m = threadIdx.x >> 4, n = (ot + i) * kTileN + (threadIdx.x & 15);
      float y = 0.0f, up = 0.0f;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        y += part[s][i][threadIdx.x];
        if (SWIGLU) up += part[s][kOut + i][threadIdx.x];
      }
      if (SWIGLU) y = silu(y) * up;
      if (m < left && n < a.N) a.out[(first + r0 + m) * a.N + n] = f32_to_bf16(y);
    }
    __syncthreads();
  }
}

ep_status_t check_w4(const ep_w4_t *w) {
  if (w == nullptr) return failf(EP_ERR_INVALID_ARG, "w4 is NULL");
  if (w->num_experts < 1 || w->num_experts > EP_MAX_EXPERTS)
    return failf(EP_ERR_INVALID_ARG, "num_experts %d outside [1, %d]", w->num_experts,
                 EP_MAX_EXPERTS);
  if (w->group != 32 && w->group != 64 && w->group != 128)
    return failf(EP_ERR_INVALID_ARG, "group %d must be 32, 64 or 128", w->group);
  if (w->in_features < 1 || w->in_features >= (1 << 24) || w->in_features % w->group != 0)
    return failf(EP_ERR_INVALID_ARG, "in_features %d must be a positive multiple of group %d, "
                 "below 2^24", w->in_features, w->group);
  if (w->out_features < 1 || w->out_features >= (1 << 20))
    return failf(EP_ERR_INVALID_ARG, "out_features %d outside [1, 2^20)", w->out_features);
  return EP_OK;
}

#define EP_TRY(expr)                \
  do {                              \
    const ep_status_t st_ = (expr); \
    if (st_ != EP_OK) return st_;   \
  } while (0)

// Calls f with the compile-time forms of the four choices.
template <typename F>
void with_product(bool fp8, int group, bool zeros, bool swiglu, F f) {
  const auto by_swiglu = [&](auto p, auto g, auto z) {
    if (swiglu)
      f(p, g, z, std::true_type{});
    else
      f(p, g, z, std::false_type{});
  };
  const auto by_zeros = [&](auto p, auto g) {
    if (zeros)
      by_swiglu(p, g, std::true_type{});
    else
      by_swiglu(p, g, std::false_type{});
  };
  const auto by_group = [&](auto p) {
    if (group == 32)
      by_zeros(p, std::integral_constant<int, 32>{});
    else if (group == 64)
      by_zeros(p, std::integral_constant<int, 64>{});
    else
      by_zeros(p, std::integral_constant<int, 128>{});
  };
  if (fp8)
    by_group(std::true_type{});
  else
    by_group(std::false_type{});
}

}  // namespace
}  // namespace ep

extern "C" {

ep_status_t ep_w4_packed_sizes(const ep_w4_t *w4, int64_t *code_bytes_host,
                               int64_t *scale_values_host) {
  using namespace ep;
  EP_TRY(check_w4(w4));
  if (code_bytes_host == nullptr || scale_values_host == nullptr)
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  const int64_t rows = (int64_t)w4->num_experts * (w4->swiglu ? 2 : 1) *
                       ((w4->out_features + kTileN - 1) / kTileN);
  *code_bytes_host = rows * ((w4->in_features + kTileK - 1) / kTileK) * kTileBytes;
  *scale_values_host = rows * (w4->in_features / w4->group) * kTileN;
  return EP_OK;
}

ep_status_t ep_w4_pack(const ep_w4_t *w4, const uint8_t *codes, const uint16_t *scales,
                       const uint8_t *zeros, uint8_t *w_codes, uint16_t *w_scales,
                       uint8_t *w_zeros, hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_w4(w4));
  if (codes == nullptr || scales == nullptr || w_codes == nullptr || w_scales == nullptr)
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((zeros == nullptr) != (w_zeros == nullptr))
    return failf(EP_ERR_INVALID_ARG, "zeros and w_zeros must both be given or both be NULL");
  if (!aligned_to(w_codes, 16))
    return failf(EP_ERR_INVALID_ARG, "w_codes must be 16-byte aligned");
  PackArgs a;
  a.codes = codes;
  a.zeros = zeros;
  a.scales = scales;
  a.w_codes = w_codes;
  a.w_zeros = w_zeros;
  a.w_scales = w_scales;
  a.N = w4->out_features;
  a.K = w4->in_features;
  a.group = w4->group;
  a.N16 = (a.N + kTileN - 1) / kTileN;
  a.K128 = (a.K + kTileK - 1) / kTileK;
  const int64_t grid = (int64_t)w4->num_experts * (w4->swiglu ? 2 : 1) * a.N16;
  if (grid >= (int64_t{1} << 24))
    return failf(EP_ERR_INVALID_ARG, "%lld row tiles do not fit one launch", (long long)grid);
  hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)grid), dim3(256), 0, stream, a);
  return launched("pack launch");
}

ep_status_t ep_expert_product_w4(const ep_w4_t *w4, ep_dtype_t x_dtype, const void *x,
                                 const float *x_scales, const uint8_t *w_codes,
                                 const uint16_t *w_scales, const uint8_t *w_zeros,
                                 const int32_t *expert_offsets,
                                 const int32_t *num_tokens_per_expert, int64_t capacity,
                                 uint16_t *out, hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_w4(w4));
  if (x_dtype != EP_DTYPE_BF16 && x_dtype != EP_DTYPE_FP8_E4M3)
    return failf(EP_ERR_INVALID_ARG, "x dtype %d must be bf16 or FP8", (int)x_dtype);
  const bool fp8 = x_dtype == EP_DTYPE_FP8_E4M3;
  if (fp8 && w4->in_features % 128 != 0)
    return failf(EP_ERR_INVALID_ARG, "FP8 rows need in_features %% 128 == 0 (in_features %d)",
                 w4->in_features);
  if (capacity < 0 || capacity >= INT32_MAX)
    return failf(EP_ERR_INVALID_ARG, "capacity %lld outside [0, 2^31 - 1)", (long long)capacity);
  if (w_codes == nullptr || w_scales == nullptr || expert_offsets == nullptr ||
      num_tokens_per_expert == nullptr ||
      (capacity > 0 && (x == nullptr || out == nullptr || (fp8 && x_scales == nullptr))))
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned_to(x, 16) || !aligned_to(w_codes, 16))
    return failf(EP_ERR_INVALID_ARG, "x and w_codes must be 16-byte aligned");
  if (capacity == 0) return EP_OK;
  ProductArgs a;
  a.x = x;
  a.x_scales = x_scales;
  a.w_codes = w_codes;
  a.w_zeros = w_zeros;
  a.w_scales = w_scales;
  a.offsets = expert_offsets;
  a.counts = num_tokens_per_expert;
  a.out = out;
  a.capacity = capacity;
  a.N = w4->out_features;
  a.K = w4->in_features;
  a.N16 = (a.N + kTileN - 1) / kTileN;
  a.K128 = (a.K + kTileK - 1) / kTileK;
  with_product(fp8, w4->group, w_zeros != nullptr, w4->swiglu != 0,
               [&](auto p, auto g, auto z, auto s) {
                 constexpr int kTiles = 4;
                 constexpr int kOut = s.value ? kTiles / 2 : kTiles;
                 const dim3 grid((unsigned)((a.N16 + kOut - 1) / kOut),
                                 (unsigned)w4->num_experts);
                 hipLaunchKernelGGL(
                     (product_kernel<p.value, g.value, z.value, s.value, kTiles>), grid,
                     dim3(256), 0, stream, a);
               });
  return launched("expert product launch");
}

}  // extern "C"
