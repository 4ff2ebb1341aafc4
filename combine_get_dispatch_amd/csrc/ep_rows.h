// What the kernels on expert-major rows share (the products with 4-bit and with
// bf16 weights, the checkpoint): an expert's rows inside the buffers, their
// blocks, and a few conversions.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep.h"

namespace ep {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float bf16_to_f32(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}

// Nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Two of them, by one instruction.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// 1 / (1 + exp(-y)) and 1 minus it, by exp(-|y|): neither loses bits where it
// is small.
__device__ __forceinline__ void sigmoids(float y, float *s, float *one_minus) {
  const float t = expf(-fabsf(y)), d = 1.0f / (1.0f + t);
  *s = (y < 0.0f ? t : 1.0f) * d;
  *one_minus = (y < 0.0f ? 1.0f : t) * d;
}

// exp(-y) of a y below -88 is infinite while silu(y) is still a fp32 number.
__device__ __forceinline__ float silu_of(float y) {
  const float t = expf(-fabsf(y));
  return y * ((y < 0.0f ? t : 1.0f) / (1.0f + t));
}

// Rows of odd widths begin anywhere: the hardware loads and stores 16 bytes at
// any address.
struct __attribute__((packed, aligned(1))) Any16 {
  u32x4 v;
};
struct __attribute__((packed, aligned(1))) Any8 {
  u32x2 v;
};

// Eight columns of a row, of which there are n, zeros for the others; `before`
// columns of the row come before them.  A row's last columns come with the ones
// before them, in one load.
__device__ __forceinline__ u32x4 load_bf16(const uint16_t *p, int n, int before) {
  u32x4 v = {0, 0, 0, 0};
  if (n >= 8) return reinterpret_cast<const Any16 *>(p)->v;
  if (n <= 0) return v;
  if (before + n >= 8) {
    const u32x4 all = reinterpret_cast<const Any16 *>(p - (8 - n))->v;
    const int drop = (8 - n) * 16;
    uint64_t lo = all[0] | (uint64_t)all[1] << 32, hi = all[2] | (uint64_t)all[3] << 32;
    lo = drop >= 64 ? hi >> (drop - 64) : lo >> drop | hi << 1 << (63 - drop);
    hi = drop >= 64 ? 0 : hi >> drop;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) v[i / 2] |= (uint32_t)p[i] << (i % 2 * 16);
  return v;
}

__device__ __forceinline__ u32x2 load_codes(const uint8_t *p, int n, int before) {
  u32x2 v = {0, 0};
  if (n >= 8) return reinterpret_cast<const Any8 *>(p)->v;
  if (n <= 0) return v;
  if (before + n >= 8) {
    const u32x2 all = reinterpret_cast<const Any8 *>(p - (8 - n))->v;
    const uint64_t w = (all[0] | (uint64_t)all[1] << 32) >> (8 - n) * 8;
    return u32x2{(uint32_t)w, (uint32_t)(w >> 32)};
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) v[i / 4] |= (uint32_t)p[i] << (i % 4 * 8);
  return v;
}

// Rows of an expert inside the buffers.
__device__ __forceinline__ void rows_inside(int32_t offset, int32_t count, int64_t capacity,
                                            int64_t *first, int64_t *rows) {
  *first = offset;
  *rows = 0;
  if (offset < 0 || count <= 0 || offset >= capacity) return;
  *rows = count < capacity - offset ? count : capacity - offset;
}

struct ExpertRows {
  const int32_t *offsets, *counts;
  int64_t capacity;
  int32_t E;
};

// First block of each expert, numbered through all of them: starts[0 .. E],
// where blocks_of(rows) is an expert's number of blocks.  Of a workgroup of at
// least 256 threads; totals holds one value per wave.
template <typename F>
__device__ __forceinline__ void number_blocks(const ExpertRows &x, int32_t *starts,
                                              int32_t *totals, F blocks_of) {
  static_assert(EP_MAX_EXPERTS <= 1024, "four experts per thread");
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  int32_t mine[4], total = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = tid * 4 + i;
    int64_t first = 0, rows = 0;
    if (e < x.E) rows_inside(x.offsets[e], x.counts[e], x.capacity, &first, &rows);
    mine[i] = (int32_t)blocks_of(rows);
    total += mine[i];
  }
  int32_t at = total;  // of this lane and those before it
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int32_t before = __shfl_up(at, d);
    at += lane >= d ? before : 0;
  }
  if (lane == 63) totals[wave] = at;
  __syncthreads();
  at -= total;
  for (int w = 0; w < wave; ++w) at += totals[w];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (tid * 4 + i <= x.E) starts[tid * 4 + i] = at;
    at += mine[i];
  }
  if (tid == 255 && x.E == 1024) starts[x.E] = at;
  __syncthreads();
}

// The expert that block belongs to: the last that starts at or before it.
__device__ __forceinline__ int expert_of(const int32_t *starts, int E, int32_t block) {
  int e = 0, hi = E - 1;
  while (e < hi) {
    const int mid = (e + hi + 1) / 2;
    if (starts[mid] <= block)
      e = mid;
    else
      hi = mid - 1;
  }
  return uniform(e);
}

}  // namespace ep
