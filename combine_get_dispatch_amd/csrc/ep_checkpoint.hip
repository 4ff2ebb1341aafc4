// SwiGLU of the experts' gate and up rows with an 8-bit checkpoint of them,
// and its gradient from the checkpoint, for gfx950.  Contracts in
// include/ep_moe.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep.h"
#include "ep_host.h"
#include "ep_moe.h"
#include "ep_rows.h"

namespace ep {
namespace {

constexpr int kBlockCols = 128;   // columns that share a scale
constexpr int kItemRows = 4;      // rows of an item: one per wave
constexpr int kGrid = 256 * 8;

struct CheckpointArgs {
  ExpertRows rows;
  const uint16_t *gate_up, *grad_h;
  uint8_t *codes;
  float *scales;
  uint16_t *h, *grad_gate_up;
  int32_t F;
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

__device__ __forceinline__ uint8_t code_of(float v, float inverse) {
  if (!finite(v)) return 0x7F;
  return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v * inverse, 0.0f, 0, false);
}

// A wave takes a row's blocks of gate and up, two columns of each per lane.
__global__ __launch_bounds__(256) void swiglu_checkpoint_kernel(CheckpointArgs a) {
  __shared__ int32_t starts[EP_MAX_EXPERTS + 1], totals[4];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  number_blocks(a.rows, starts, totals,
                [](int64_t rows) { return (rows + kItemRows - 1) / kItemRows; });
  const int F = a.F, blocks = (F + kBlockCols - 1) / kBlockCols;
  const int64_t items = starts[a.rows.E];
  for (int64_t i0 = blockIdx.x; i0 < items; i0 += gridDim.x) {
    const int32_t item = (int32_t)i0;
    const int e = expert_of(starts, a.rows.E, item);
    int64_t first, rows;
    rows_inside(a.rows.offsets[e], a.rows.counts[e], a.rows.capacity, &first, &rows);
    const int64_t r = (int64_t)(item - starts[e]) * kItemRows + wave;
    if (r >= rows) continue;
    const uint16_t *in = a.gate_up + (first + r) * 2 * F;
    for (int b = 0; b < blocks; ++b) {
      float v[2][2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = b * kBlockCols + lane + 64 * i;
          v[half][i] = c < F ? bf16_to_f32(in[half * F + c]) : 0.0f;
          if (finite(v[half][i])) most = fmaxf(most, fabsf(v[half][i]));
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
        const int x = scale_exponent(most);
        if (lane == 0) a.scales[((first + r) * 2 + half) * blocks + b] = power_of_two(x);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = b * kBlockCols + lane + 64 * i;
          if (c < F)
            a.codes[((first + r) * 2 + half) * F + c] = code_of(v[half][i], power_of_two(-x));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = b * kBlockCols + lane + 64 * i;
        if (c < F) a.h[(first + r) * F + c] = f32_to_bf16(silu_of(v[0][i]) * v[1][i]);
      }
    }
  }
}

__global__ __launch_bounds__(256) void swiglu_backward_kernel(CheckpointArgs a) {
  __shared__ int32_t starts[EP_MAX_EXPERTS + 1], totals[4];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  number_blocks(a.rows, starts, totals,
                [](int64_t rows) { return (rows + kItemRows - 1) / kItemRows; });
  const int F = a.F, blocks = (F + kBlockCols - 1) / kBlockCols;
  const int64_t items = starts[a.rows.E];
  for (int64_t i0 = blockIdx.x; i0 < items; i0 += gridDim.x) {
    const int32_t item = (int32_t)i0;
    const int e = expert_of(starts, a.rows.E, item);
    int64_t first, rows;
    rows_inside(a.rows.offsets[e], a.rows.counts[e], a.rows.capacity, &first, &rows);
    const int64_t r = (int64_t)(item - starts[e]) * kItemRows + wave;
    if (r >= rows) continue;
    const uint8_t *codes = a.codes + (first + r) * 2 * F;
    const float *scales = a.scales + (first + r) * 2 * blocks;
    for (int c = lane; c < F; c += 64) {
      const int b = c / kBlockCols;
      const float g = __builtin_amdgcn_cvt_f32_fp8((int)codes[c], 0) * scales[b];
      const float u = __builtin_amdgcn_cvt_f32_fp8((int)codes[F + c], 0) * scales[blocks + b];
      const float d = bf16_to_f32(a.grad_h[(first + r) * F + c]);
      float s, t;
      sigmoids(g, &s, &t);
      uint16_t *out = a.grad_gate_up + (first + r) * 2 * F + c;
      out[0] = f32_to_bf16(s * (1.0f + g * t) * u * d);
      out[F] = f32_to_bf16(g * s * d);
      if (a.h != nullptr) a.h[(first + r) * F + c] = f32_to_bf16(g * s * u);
    }
  }
}

ep_status_t check_checkpoint(int32_t E, int32_t F, const int32_t *offsets, const int32_t *counts,
                             int64_t capacity) {
  if (E < 1 || E > EP_MAX_EXPERTS)
    return failf(EP_ERR_INVALID_ARG, "num_experts %d outside [1, %d]", E, EP_MAX_EXPERTS);
  if (F < 1 || F >= (1 << 20))
    return failf(EP_ERR_INVALID_ARG, "features %d outside [1, 2^20)", F);
  if (capacity < 0 || capacity >= INT32_MAX)
    return failf(EP_ERR_INVALID_ARG, "capacity %lld outside [0, 2^31 - 1)", (long long)capacity);
  if ((capacity / kItemRows + 1) * E >= INT32_MAX)
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

bool apart(const Range &a, const Range &b) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
  return a.p == nullptr || b.p == nullptr || p >= q + (uintptr_t)b.bytes ||
         q >= p + (uintptr_t)a.bytes;
}

#define EP_TRY(expr)                \
  do {                              \
    const ep_status_t st_ = (expr); \
    if (st_ != EP_OK) return st_;   \
  } while (0)

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
  CheckpointArgs a = {};
  a.rows = ExpertRows{expert_offsets, num_tokens_per_expert, capacity, num_experts};
  a.gate_up = gate_up;
  a.h = h;
  a.codes = codes;
  a.scales = scales;
  a.F = features;
  hipLaunchKernelGGL(swiglu_checkpoint_kernel, dim3(kGrid), dim3(256), 0, stream, a);
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
  CheckpointArgs a = {};
  a.rows = ExpertRows{expert_offsets, num_tokens_per_expert, capacity, num_experts};
  a.codes = const_cast<uint8_t *>(codes);
  a.scales = const_cast<float *>(scales);
  a.grad_h = grad_h;
  a.grad_gate_up = grad_gate_up;
  a.h = h;
  a.F = features;
  hipLaunchKernelGGL(swiglu_backward_kernel, dim3(kGrid), dim3(256), 0, stream, a);
  return launched("checkpoint backward launch");
}

}  // extern "C"
