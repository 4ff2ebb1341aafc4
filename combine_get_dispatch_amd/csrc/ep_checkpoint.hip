// SwiGLU of the experts' gate and up rows with an 8-bit checkpoint of them,
// and its gradient from the checkpoint, for gfx950.  Contracts in
// include/ep_moe.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ep.h"
#include "ep_host.h"
#include "ep_moe.h"
#include "ep_rows.h"

namespace ep {
namespace {

constexpr int kBlockCols = 128;  // columns that share a scale: 16 lanes x 8
constexpr int kUnroll = 4;       // blocks of gate and up in flight per 16 lanes
constexpr int kItemBlocks = 16 * kUnroll;  // at least, in large calls; 16 x 16 lanes
constexpr int kGrid = 256 * 8;

struct CheckpointArgs {
  ExpertRows rows;
  const uint16_t *gate_up, *grad_h;
  uint8_t *codes;
  float *scales;
  uint16_t *h, *grad_gate_up;
  int32_t F, blocks, item_rows;
};

// The scale's exponent for values of at most this magnitude: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float most) {
  const int e = (int)((__float_as_uint(most) + 0x1FFFFFu) >> 23) - 127 - 8;
  return e < -100 ? -100 : e;
}

__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ bool finite(float v) {
  return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
}

// Largest over the 16 lanes of a block.
__device__ __forceinline__ float most_of_block(float v) {
  const auto turn = [](float x, auto by) {
    const int i = __builtin_bit_cast(int, x);
    return fmaxf(x, __builtin_bit_cast(
                        float, __builtin_amdgcn_update_dpp(i, i, 0x120 + decltype(by)::value, 0xF,
                                                           0xF, false)));
  };
  v = turn(v, std::integral_constant<int, 8>{});
  v = turn(v, std::integral_constant<int, 4>{});
  v = turn(v, std::integral_constant<int, 2>{});
  return turn(v, std::integral_constant<int, 1>{});
}

__device__ __forceinline__ void store_bf16(uint16_t *p, int n, const float *y) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
  if (n >= 8) {
    reinterpret_cast<Any16 *>(p)->v = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = (uint16_t)(v[i / 2] >> (i % 2 * 16));
}

__device__ __forceinline__ void store_codes(uint8_t *p, int n, u32x2 v) {
  if (n >= 8) {
    reinterpret_cast<Any8 *>(p)->v = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = (uint8_t)(v[i / 4] >> (i % 4 * 8));
}

__device__ __forceinline__ void unpack(u32x4 v, float *y) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = __uint_as_float(i % 2 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
}

// 1 / (1 + exp(-y)) and 1 minus it of eight values, by t = exp(-|y|): the
// hardware's exp2 of y log2 e, whose rounding is put back to first order, and
// its reciprocal; off by few half steps.  Past 80 t comes near the smallest
// normal number, where exp2 ends: there by expf.
__device__ __forceinline__ void sigmoids8(const float *y, float *s, float *rest) {
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(y[i]));
  if (most > 80.0f) {  // not by the wave: a row's results are the same beside any other
#pragma unroll
    for (int i = 0; i < 8; ++i) sigmoids(y[i], &s[i], &rest[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
    const float x = -fabsf(y[i]), n = x * kLog2e;
    const float lost = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -n));
    const float e = __builtin_amdgcn_exp2f(n);
    const float t = __builtin_fmaf(e * kLn2, lost, e);
    const float d = __builtin_amdgcn_rcpf(1.0f + t), td = t * d;
    s[i] = y[i] < 0.0f ? td : d;
    rest[i] = y[i] < 0.0f ? d : td;
  }
}

// Eight codes of 16 lanes' values, and the block's scale.
__device__ __forceinline__ u32x2 encode(const float *y, float *scale) {
  float most = 0.0f, v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = y[i];
    most = fmaxf(most, fabsf(v[i]));  // passes over NaN
  }
  if (__any(!finite(most))) {
    most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (finite(v[i]))
        most = fmaxf(most, fabsf(v[i]));
      else
        v[i] = __builtin_nanf("");
    }
  }
  const int e = scale_exponent(most_of_block(most));
  *scale = power_of_two(e);
  const float inverse = power_of_two(-e);
  u32x2 codes;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inverse, v[4 * i + 1] * inverse, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inverse, v[4 * i + 3] * inverse, w, true);
    codes[i] = (uint32_t)w;
  }
  return codes;
}

// Calls f(row, block) for the blocks of all rows, each with 16 lanes, kUnroll
// calls of load before those of work.
template <typename Load, typename Work>
__device__ __forceinline__ void for_blocks(const CheckpointArgs &a, Load load, Work work) {
  __shared__ int32_t starts[EP_MAX_EXPERTS + 1], totals[4];
  const int item_rows = a.item_rows;
  number_blocks(a.rows, starts, totals,
                [=](int64_t rows) { return (rows + item_rows - 1) / item_rows; });
  const int64_t items = starts[a.rows.E];
  for (int64_t i0 = blockIdx.x; i0 < items; i0 += gridDim.x) {
    const int32_t item = (int32_t)i0;
    const int e = expert_of(starts, a.rows.E, item);
    int64_t first, rows;
    rows_inside(a.rows.offsets[e], a.rows.counts[e], a.rows.capacity, &first, &rows);
    const int64_t skip = (int64_t)(item - starts[e]) * item_rows;
    const int n = (int)(rows - skip < item_rows ? rows - skip : item_rows) * a.blocks;
    for (int q0 = threadIdx.x / 16; q0 < n; q0 += kItemBlocks) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = q0 + 16 * u;
        if (q < n) load(u, first + skip + q / a.blocks, q % a.blocks);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = q0 + 16 * u;
        if (q < n) work(u, first + skip + q / a.blocks, q % a.blocks);
      }
    }
  }
}

__global__ __launch_bounds__(256) void swiglu_checkpoint_kernel(CheckpointArgs a) {
  const int l16 = threadIdx.x & 15;
  const int F = a.F, blocks = a.blocks;
  u32x4 gate[kUnroll], up[kUnroll];
  for_blocks(
      a,
      [&](int u, int64_t row, int b) {
        const int c = b * kBlockCols + l16 * 8;
        const uint16_t *p = a.gate_up + row * 2 * F + c;
        gate[u] = load_bf16(p, F - c, c);
        up[u] = load_bf16(p + F, F - c, c);
      },
      [&](int u, int64_t row, int b) {
        const int c = b * kBlockCols + l16 * 8;
        float x[8], y[8], s[8], rest[8], scale;
        unpack(gate[u], x);
        unpack(up[u], y);
        uint8_t *codes = a.codes + row * 2 * F + c;
        float *scales = a.scales + row * 2 * blocks + b;
        store_codes(codes, F - c, encode(x, &scale));
        if (l16 == 0) scales[0] = scale;
        store_codes(codes + F, F - c, encode(y, &scale));
        if (l16 == 0) scales[blocks] = scale;
        sigmoids8(x, s, rest);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * s[i] * y[i];
        store_bf16(a.h + row * F + c, F - c, x);
      });
}

__global__ __launch_bounds__(256) void swiglu_backward_kernel(CheckpointArgs a) {
  const int l16 = threadIdx.x & 15;
  const int F = a.F, blocks = a.blocks;
  u32x2 gate[kUnroll], up[kUnroll];
  u32x4 grad[kUnroll];
  float gate_scale[kUnroll], up_scale[kUnroll];
  for_blocks(
      a,
      [&](int u, int64_t row, int b) {
        const int c = b * kBlockCols + l16 * 8;
        const uint8_t *codes = a.codes + row * 2 * F + c;
        const float *scales = a.scales + row * 2 * blocks + b;
        gate[u] = load_codes(codes, F - c, c);
        up[u] = load_codes(codes + F, F - c, c);
        gate_scale[u] = scales[0];
        up_scale[u] = scales[blocks];
        grad[u] = load_bf16(a.grad_h + row * F + c, F - c, c);
      },
      [&](int u, int64_t row, int b) {
        const int c = b * kBlockCols + l16 * 8;
        float x[8], y[8], d[8], s[8], rest[8], dx[8], dy[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const auto g = i % 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)gate[u][i / 2], true)
                               : __builtin_amdgcn_cvt_pk_f32_fp8((int)gate[u][i / 2], false);
          const auto p = i % 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)up[u][i / 2], true)
                               : __builtin_amdgcn_cvt_pk_f32_fp8((int)up[u][i / 2], false);
          x[2 * i] = g[0] * gate_scale[u];
          x[2 * i + 1] = g[1] * gate_scale[u];
          y[2 * i] = p[0] * up_scale[u];
          y[2 * i + 1] = p[1] * up_scale[u];
        }
        unpack(grad[u], d);
        sigmoids8(x, s, rest);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // the sigmoid first: where it is 0 no product before it may overflow
          const float silu = x[i] * s[i];
          dx[i] = s[i] * __builtin_fmaf(x[i], rest[i], 1.0f) * y[i] * d[i];
          dy[i] = silu * d[i];
          x[i] = silu * y[i];
        }
        uint16_t *out = a.grad_gate_up + row * 2 * F + c;
        store_bf16(out, F - c, dx);
        store_bf16(out + F, F - c, dy);
        if (a.h != nullptr) store_bf16(a.h + row * F + c, F - c, x);
      });
}

// Rows, their blocks, and how many rows make an item.
CheckpointArgs checkpoint_args(int32_t E, int32_t F, const int32_t *offsets,
                               const int32_t *counts, int64_t capacity) {
  CheckpointArgs a = {};
  a.rows = ExpertRows{offsets, counts, capacity, E};
  a.F = F;
  a.blocks = (F + kBlockCols - 1) / kBlockCols;
  // where they do not fill the chip otherwise, items of one block per 16 lanes
  const int item = capacity * a.blocks < 512 * kItemBlocks ? 16 : kItemBlocks;
  a.item_rows = (item + a.blocks - 1) / a.blocks;
  if (item == kItemBlocks && a.item_rows < 4) a.item_rows = 4;
  return a;
}

int checkpoint_grid(const CheckpointArgs &a) {
  const int64_t items = a.rows.capacity / a.item_rows + a.rows.E;
  return (int)(items < kGrid ? items : kGrid);
}

ep_status_t check_checkpoint(int32_t E, int32_t F, const int32_t *offsets, const int32_t *counts,
                             int64_t capacity) {
  if (E < 1 || E > EP_MAX_EXPERTS)
    return failf(EP_ERR_INVALID_ARG, "num_experts %d outside [1, %d]", E, EP_MAX_EXPERTS);
  if (F < 1 || F >= (1 << 20))
    return failf(EP_ERR_INVALID_ARG, "features %d outside [1, 2^20)", F);
  if (capacity < 0 || capacity >= INT32_MAX)
    return failf(EP_ERR_INVALID_ARG, "capacity %lld outside [0, 2^31 - 1)", (long long)capacity);
  if ((capacity / 4 + 1) * E >= INT32_MAX)
    return failf(EP_ERR_INVALID_ARG, "capacity %lld x %d experts has too many row blocks",
                 (long long)capacity, E);
  if (offsets == nullptr || counts == nullptr)
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  return EP_OK;
}

struct Range {
  const void *p;
  int64_t bytes;
};

bool apart(const Range &a, const Range &b) { return !overlap(a.p, a.bytes, b.p, b.bytes); }

}  // namespace
}  // namespace ep

extern "C" {

ep_status_t ep_swiglu_checkpoint(int32_t num_experts, int32_t features, const uint16_t *gate_up,
                                 const int32_t *expert_offsets,
                                 const int32_t *num_tokens_per_expert, int64_t capacity,
                                 uint16_t *h, uint8_t *codes, float *scales, hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_checkpoint(num_experts, features, expert_offsets, num_tokens_per_expert, capacity));
  if (capacity == 0) return EP_OK;
  if (gate_up == nullptr || h == nullptr || codes == nullptr || scales == nullptr)
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned_to(gate_up, 16) || !aligned_to(h, 16) || !aligned_to(codes, 16) ||
      !aligned_to(scales, 4))
    return failf(EP_ERR_INVALID_ARG,
                 "gate_up, h and codes must be 16-byte, scales 4-byte aligned");
  const int64_t values = capacity * features, blocks = (features + kBlockCols - 1) / kBlockCols;
  const Range all[4] = {{gate_up, values * 4}, {h, values * 2}, {codes, values * 2},
                        {scales, capacity * 2 * blocks * 4}};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (!apart(all[i], all[j])) return failf(EP_ERR_INVALID_ARG, "two of the arrays overlap");
  CheckpointArgs a =
      checkpoint_args(num_experts, features, expert_offsets, num_tokens_per_expert, capacity);
  a.gate_up = gate_up;
  a.h = h;
  a.codes = codes;
  a.scales = scales;
  hipLaunchKernelGGL(swiglu_checkpoint_kernel, dim3(checkpoint_grid(a)), dim3(256), 0,
                     stream, a);
  return launched("checkpoint launch");
}

ep_status_t ep_swiglu_checkpoint_backward(int32_t num_experts, int32_t features,
                                          const uint8_t *codes, const float *scales,
                                          const uint16_t *grad_h, const int32_t *expert_offsets,
                                          const int32_t *num_tokens_per_expert, int64_t capacity,
                                          uint16_t *grad_gate_up, uint16_t *h,
                                          hipStream_t stream) {
  using namespace ep;
  EP_TRY(check_checkpoint(num_experts, features, expert_offsets, num_tokens_per_expert, capacity));
  if (capacity == 0) return EP_OK;
  if (codes == nullptr || scales == nullptr || grad_h == nullptr || grad_gate_up == nullptr)
    return failf(EP_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned_to(codes, 16) || !aligned_to(scales, 4) || !aligned_to(grad_h, 16) ||
      !aligned_to(grad_gate_up, 16) || !aligned_to(h, 16))
    return failf(EP_ERR_INVALID_ARG,
                 "codes, grad_h, grad_gate_up and h must be 16-byte, scales 4-byte aligned");
  const int64_t values = capacity * features, blocks = (features + kBlockCols - 1) / kBlockCols;
  const Range all[5] = {{grad_gate_up, values * 4}, {h, values * 2}, {codes, values * 2},
                        {scales, capacity * 2 * blocks * 4}, {grad_h, values * 2}};
  for (int i = 0; i < 2; ++i)  // the outputs against all
    for (int j = i + 1; j < 5; ++j)
      if (!apart(all[i], all[j])) return failf(EP_ERR_INVALID_ARG, "two of the arrays overlap");
  CheckpointArgs a =
      checkpoint_args(num_experts, features, expert_offsets, num_tokens_per_expert, capacity);
  a.codes = const_cast<uint8_t *>(codes);
  a.scales = const_cast<float *>(scales);
  a.grad_h = grad_h;
  a.grad_gate_up = grad_gate_up;
  a.h = h;
  hipLaunchKernelGGL(swiglu_backward_kernel, dim3(checkpoint_grid(a)), dim3(256), 0,
                     stream, a);
  return launched("checkpoint backward launch");
}

}  // extern "C"
