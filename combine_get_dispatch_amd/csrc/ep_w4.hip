// The experts' products with 4-bit weights for gfx950: packing, and the
// product on expert-major rows.  Contracts and the packed layout in
// include/ep_moe.h.
//
// How 4 bits enter the matrix instructions exactly, without a conversion: a code
// q in mantissa bits 3..6 of 0x3B80 is the bf16 u (1 + q/16) with u = 2^-8, so
//     sum x u (1 + q/16) = X + u sum(x q)/16  with X = sum x u, and
//     sum x (q - z) = 2^12 (sum x u (1 + q/16) - X (1 + z/16)).
// X comes from the same instruction with a matrix of u, once per row tile.  With
// u the sums over a group stay finite for every finite row (128 terms of at
// most 31/16 u), and no bit is lost at the other end (x is a whole number of
// 2^-133, a term of 2^-145).  The 2^12 comes last, so that only a result that
// is itself out of range leaves it.
// FP8 rows are turned into bf16, which holds every E4M3 number: the FP8
// instruction keeps, of eight products, only what is less than 2^14 below the
// largest (measured: of two, the smaller is lost from there on), while the bf16
// one, of the same rate, sums them in 32 bits.
// Group scales are applied to the fp32 sums of a group.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ep.h"
#include "ep_host.h"
#include "ep_moe.h"
#include "ep_rows.h"

namespace ep {
namespace {

constexpr int kTileN = 16;       // output columns of a weight tile
constexpr int kTileK = 128;      // columns of the sum in a weight tile
constexpr int kTileBytes = 1024;
constexpr int kRows = 16;        // rows of x per matrix instruction

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
  int32_t stream_rows;  // experts with more rows are tiled
};

// Rows of an expert that the whole wave works on.
__device__ __forceinline__ void expert_rows(const ProductArgs &a, int e, int64_t *first,
                                            int64_t *rows) {
  rows_inside(uniform(a.offsets[e]), uniform(a.counts[e]), a.capacity, first, rows);
}

// The pairs of codes of one word as bf16 pairs u (1 + q/16): a shift and one
// and-or each.  The instruction takes one constant from a scalar register and
// none from its own encoding, so the other is kept in a vector register.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w) {
  uint32_t mask = 0x00780078u, u = 0x3B803B80u;
  asm("" : "+s"(mask));
  asm("" : "+v"(u));
  u32x4 v;
  v[0] = ((w << 3) & mask) | u;
  v[1] = ((w >> 1) & mask) | u;
  v[2] = ((w >> 5) & mask) | u;
  v[3] = ((w >> 9) & mask) | u;
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x4 mul(bf16x8 x, bf16x8 w, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
}

__device__ __forceinline__ bf16x8 units() {
  return __builtin_bit_cast(bf16x8, u32x4{0x3B803B80u, 0x3B803B80u, 0x3B803B80u, 0x3B803B80u});
}

// dot of codes = kUnit * (dot of what codes_bf16() makes - zero_of(z) * dot of units())
constexpr float kUnit = 0x1p12f;
__device__ __forceinline__ float zero_of(float z) { return 1.0f + z * 0x1p-4f; }

// The rows of x: eight columns per lane and matrix instruction, as they are
// loaded and as the instruction takes them.
template <bool FP8>
struct Rows {
  typedef u32x4 Raw;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ Raw load(const uint8_t *x, uint32_t at) {
    return *reinterpret_cast<const u32x4 *>(reinterpret_cast<const uint16_t *>(x) + at);
  }
  static __device__ __forceinline__ bf16x8 bf16(Raw v) { return __builtin_bit_cast(bf16x8, v); }
};

template <>
struct Rows<true> {
  typedef u32x2 Raw;
  static constexpr int kBytes = 1;
  static __device__ __forceinline__ Raw load(const uint8_t *x, uint32_t at) {
    return *reinterpret_cast<const u32x2 *>(x + at);
  }
  static __device__ __forceinline__ bf16x8 bf16(Raw v) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[2 * i] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, false));
      w[2 * i + 1] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, true));
    }
    return __builtin_bit_cast(bf16x8, w);
  }
};

// Experts with at most kStreamRows rows are streamed (product_stream_kernel),
// the others tiled (product_tile_kernel).  Past 16 rows a streamed expert's
// weights are read twice; where the blocks of the tiles fill the chip several
// times over (kTileRounds), those experts are tiled too.  Streamed and tiled, us
// (FP8 rows: the same to 8 %), with every expert at 17 rows, at 32, and with an
// average of 12, 16, 20 and 24 rows of random experts:
//   64 experts, 2048 x 7168 (3584 blocks)
//       184, 142   206, 155   102, 109   143, 134   187, 147   200, 157
//   64, 7168 x 2 x 2048 (2048)
//       332, 271   399, 278   189, 218   261, 257   370, 261   400, 295
//   32, 7168 x 2 x 2048 (1024)
//       169, 165   202, 167    99, 143   135, 137   167, 183   224, 182
//   16, 7168 x 2 x 2048 (512)
//        83,  85    93,  87    56, 117    76, 101    84, 103   163, 100
//   8, 4096 x 2048 (128)
//        18,  32    19,  32
// How many experts have more than 16 rows only the device knows: few of them,
// tiled, wait for the longest, so the tiles are left to calls where that costs
// little.
constexpr int kStreamRows = 32;
constexpr int kStreamWaves = 8;
constexpr int64_t kInfinityCache = int64_t{256} << 20;

// Few rows: the weights are read once, straight into registers, and their
// reading is the bound.  One workgroup: kTiles column tiles of one expert
// (with SwiGLU half of them gate, half up) and all its rows, 16 at a time;
// its waves take every eighth piece of the sum and add theirs in LDS at the
// end.  No rows are staged and no wave waits for another before that; the
// loads in flight are those of 16 waves per compute unit.  (Holding a second
// piece in flight per wave measured slower: its registers halve the waves.)
//
// ONCE (non-temporal loads): where a call's weights exceed the Infinity Cache
// nothing of them is found there again.  480 MB per call: 77 us with, 86
// without; below it the two differ by 5 % either way, and where 17 to 32 rows
// read the weights twice (16 experts, 4096 x 2 x 2048) 59 with, 58 without.
// 480 MB (32 experts, 7168 x 2 x 2048, 4 rows each): bf16 77 us, FP8 79 with the
// tiled kernel's empty launch, 6.1 TB/s of the 6.9 that reading alone reaches.
template <bool FP8, int GROUP, bool ZEROS, bool SWIGLU, int kTiles, bool ONCE>
__global__ __launch_bounds__(kStreamWaves * 64, 4) void product_stream_kernel(ProductArgs a) {
  typedef Rows<FP8> F;
  constexpr int kHalves = SWIGLU ? 2 : 1;
  constexpr int kOut = kTiles / kHalves;   // column tiles of the output
  constexpr int kGroups = kTileK / GROUP;  // groups in a tile
  constexpr int kPer = GROUP / 32;         // matrix instructions per group
  __shared__ float part[kStreamWaves][kTiles][kRows * kTileN];
  const int e = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  int64_t first, rows;
  expert_rows(a, e, &first, &rows);
  if (rows == 0 || rows > a.stream_rows) return;
  const int G = a.K / GROUP;
  const int ot = blockIdx.x * kOut;
  int64_t tile_row[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    int n = ot + i % kOut;
    n = n < a.N16 ? n : a.N16 - 1;
    tile_row[i] = ((int64_t)e * kHalves + i / kOut) * a.N16 + n;
  }
  struct Piece {
    u32x4 w[kTiles];
    uint16_t s[kTiles][kGroups];
    uint8_t z[kTiles][kGroups];
    typename F::Raw x[4];
    f32x4 sx;
  };
  for (int64_t r0 = 0; r0 < rows; r0 += kRows) {
    const int left = (int)(rows - r0);
    // this lane's row of x and its four rows of scales, from the first row on
    const uint8_t *x0 = static_cast<const uint8_t *>(a.x) + (first + r0) * F::kBytes * a.K;
    const uint32_t xat = (uint32_t)(col < left ? col : left - 1) * a.K + quad * 8;
    const float *sx0 = FP8 ? a.x_scales + (first + r0) * a.K128 : nullptr;
    f32x4 acc[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[i] = f32x4{0, 0, 0, 0};
    const auto load = [&](int kt, Piece &p) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const u32x4 *w = reinterpret_cast<const u32x4 *>(
                             a.w_codes + (tile_row[i] * a.K128 + kt) * kTileBytes) + lane;
        p.w[i] = ONCE ? __builtin_nontemporal_load(w) : *w;
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          // past the last group of a partial tile the last one's scale is read
          const int gg = kt * kGroups + g < G ? kt * kGroups + g : G - 1;
          const int64_t at = (tile_row[i] * G + gg) * kTileN;
          p.s[i][g] = (a.w_scales + at)[col];
          if (ZEROS) p.z[i][g] = (a.w_zeros + at)[col];
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = kt * kTileK + j * 32;
        p.x[j] = typename F::Raw{};
        if (GROUP == kTileK || c < a.K) p.x[j] = F::load(x0 + c * F::kBytes, xat);
      }
      if (FP8) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int m = quad * 4 + v;
          p.sx[v] = (sx0 + kt)[(uint32_t)(m < left ? m : left - 1) * a.K128];
        }
      }
    };
    // One step of all tiles after the other, so that a step's rows are turned
    // into bf16 only then.
    const auto work = [&](const Piece &p) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        f32x4 sum = {0, 0, 0, 0}, dot[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) dot[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const bf16x8 x = F::bf16(p.x[g * kPer + j]);
          sum = mul(x, units(), sum);
#pragma unroll
          for (int i = 0; i < kTiles; ++i) dot[i] = mul(x, codes_bf16(p.w[i][g * kPer + j]), dot[i]);
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const float s = bf16_to_f32(p.s[i][g]);
          const float z = zero_of(ZEROS ? (float)p.z[i][g] : 8.0f);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float d = __builtin_fmaf(-z, sum[v], dot[i][v]);
            acc[i][v] = __builtin_fmaf(s, FP8 ? d * p.sx[v] : d, acc[i][v]);
          }
        }
      }
    };
    for (int kt = wave; kt < a.K128; kt += kStreamWaves) {
      Piece p;
      load(kt, p);
      // all loads before the first wait: the compiler would put those of the
      // scales behind it, a second trip to memory (FP8, 480 MB: 90 us)
      __builtin_amdgcn_sched_barrier(0);
      work(p);
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][i][(quad * 4 + v) * kTileN + col] = acc[i][v];
    __syncthreads();
    for (int o = threadIdx.x; o < kOut * kRows * kTileN; o += kStreamWaves * 64) {
      const int i = o / (kRows * kTileN), at = o % (kRows * kTileN);
      const int m = at / kTileN, n = (ot + i) * kTileN + at % kTileN;
      float y = 0.0f, up = 0.0f;
#pragma unroll
      for (int s = 0; s < kStreamWaves; ++s) {
        y += part[s][i][at];
        if (SWIGLU) up += part[s][kOut + i][at];
      }
      y *= kUnit;
      if (SWIGLU) y = silu_of(y) * (up * kUnit);
      if (m < left && n < a.N) a.out[(first + r0 + m) * a.N + n] = f32_to_bf16(y);
    }
    __syncthreads();
  }
}

constexpr int kBlockRows = 64;  // rows of a block
constexpr int kBlockTiles = 8;  // weight column tiles of a block
// Waves per SIMD: 168 registers each, which hold all but 7 or 8 of the FP8
// kernels of groups of 32 with zero points (those keep them in scratch).
constexpr int kTileWaves = 3;
constexpr int kTileGrid = 256 * kTileWaves;  // persistent workgroups, all resident
constexpr int kTileRounds = 4;

// Many rows: blocks of 64 rows x 128 weight columns (with SwiGLU 64 gate and
// the same 64 up), taken in turn by persistent workgroups; the blocks of an
// expert's rows follow its row count, which only the device knows.  Each of
// the four waves has all rows and two column tiles.  A piece's rows go through
// registers to LDS, in the order the matrix instructions take them, one
// piece ahead of its use and one behind its load; on the way a wave sums
// its 16 rows over the groups.  So a piece needs one barrier.
// 4096 rows of 32 experts, 2048 x 7168: 207 us, 580 TFLOP/s; 8 experts of 512
// rows each: 160 us, 750; FP8 rows, 7168 x 2 x 2048 with SwiGLU: 430 us, 560.  Bound by neither memory (with the weights of one
// piece read again and again 192 us) nor one kind of instruction (matrix
// instructions 29 % of the time, others 38 %): by each wave's waits in its
// chain of LDS reads, products and group scales.  128 rows per block, two waves
// per SIMD: 246; reading a step's rows from LDS one step ahead: 214 to 225; no
// waiting for the loads of x in the same piece: 217.
template <bool FP8, int GROUP, bool ZEROS, bool SWIGLU>
__global__ __launch_bounds__(256, kTileWaves) void product_tile_kernel(ProductArgs a, int E) {
  typedef Rows<FP8> F;
  constexpr int kHalves = SWIGLU ? 2 : 1;
  constexpr int kTiles = kBlockTiles / 4;       // of a wave
  constexpr int kOut = kTiles / kHalves;        // output tiles of a wave
  constexpr int kGroups = kTileK / GROUP;
  constexpr int kPer = GROUP / 32;
  constexpr int kMT = kBlockRows / kRows;       // row tiles of a block
  static_assert(kMT == 4, "one row tile per wave is staged");
  __shared__ __align__(16) bf16x8 xs[2][kMT][4][64];
  __shared__ float sums[2][kMT][kGroups][kRows];  // of x over a group
  __shared__ float sxs[2][kMT][kRows];            // FP8: scales of the rows
  __shared__ int32_t starts[EP_MAX_EXPERTS + 1];  // first block of each expert
  __shared__ int32_t totals[4];                   // row blocks of a wave's experts
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int G = a.K / GROUP;

  // blocks of rows per expert, and their prefix sums
  {
    int32_t mine[4], total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid * 4 + i;
      int64_t first = 0, rows = 0;
      if (e < E) rows_inside(a.offsets[e], a.counts[e], a.capacity, &first, &rows);
      mine[i] = rows > a.stream_rows ? (int32_t)((rows + kBlockRows - 1) / kBlockRows) : 0;
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
      if (tid * 4 + i <= E) starts[tid * 4 + i] = at;
      at += mine[i];
    }
    if (tid == 255 && E == EP_MAX_EXPERTS) starts[E] = at;
    __syncthreads();
  }
  const int nblocks = (a.N16 + kBlockTiles / kHalves - 1) / (kBlockTiles / kHalves);
  const int64_t items = (int64_t)starts[E] * nblocks;
  // The items of an XCD (workgroups id % 8) are consecutive, the row blocks of
  // a column block next to each other, so that the workgroups that share its L2
  // share their weights (4096 rows of 32 experts, 2048 x 7168: 215 us; with the
  // column blocks of a row block next to each other 222).
  const int64_t per_xcd = (items + 7) / 8;
  const int64_t from = (blockIdx.x % 8) * per_xcd;
  const int64_t to = from + per_xcd < items ? from + per_xcd : items;

  for (int64_t item = from + blockIdx.x / 8; item < to; item += gridDim.x / 8) {
    int e = 0, hi = E - 1;
    while (e < hi) {  // the last expert that starts at or before the item
      const int mid = (e + hi + 1) / 2;
      if ((int64_t)starts[mid] * nblocks <= item)
        e = mid;
      else
        hi = mid - 1;
    }
    e = uniform(e);
    int64_t first, rows;
    expert_rows(a, e, &first, &rows);
    const int blocks = (int)((rows + kBlockRows - 1) / kBlockRows);
    const int64_t in_expert = item - (int64_t)uniform(starts[e]) * nblocks;
    const int nb = uniform((int)(in_expert / blocks));
    const int64_t per = ((rows + kRows - 1) / kRows + blocks - 1) / blocks * kRows;
    const int64_t r0 = uniform((int)(in_expert % blocks)) * per;
    const int left = (int)(rows - r0 < per ? rows - r0 : per);  // <= 0: a last block of none
    const int mts = left > 0 ? (left + kRows - 1) / kRows : 0;
    if (mts == 0) continue;
    const int ot = (nb * 4 + wave) * kOut;
    int64_t tile_row[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      int n = ot + i % kOut;
      n = n < a.N16 ? n : a.N16 - 1;
      tile_row[i] = ((int64_t)e * kHalves + i / kOut) * a.N16 + n;
    }
    // this lane's row of the wave's row tile
    const int mine = wave * kRows + col;
    const uint8_t *x0 = static_cast<const uint8_t *>(a.x) + (first + r0) * F::kBytes * a.K;
    const uint32_t xat = (uint32_t)(mine < left ? mine : left - 1) * a.K + quad * 8;
    const float *sx0 = FP8 ? a.x_scales + (first + r0) * a.K128 : nullptr;
    const uint32_t sxat = (uint32_t)(mine < left ? mine : left - 1) * a.K128;
    typename F::Raw stage[4];
    float row_scale = 0.0f;
    const auto load_x = [&](int kt) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = kt * kTileK + j * 32;
        stage[j] = typename F::Raw{};
        if (GROUP == kTileK || c < a.K) stage[j] = F::load(x0 + (int64_t)c * F::kBytes, xat);
      }
      if (FP8) row_scale = (sx0 + kt)[sxat];
    };
    const auto stage_x = [&](int buf) {
#pragma unroll
      for (int j = 0; j < 4; ++j) xs[buf][wave][j][lane] = F::bf16(stage[j]);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        f32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum = mul(F::bf16(stage[g * kPer + j]), units(), sum);
        if (!ZEROS) sum *= -zero_of(8.0f);
        if (col == 0) *reinterpret_cast<f32x4 *>(&sums[buf][wave][g][quad * 4]) = sum;
      }
      if (FP8 && quad == 0) sxs[buf][wave][col] = row_scale;
    };
    u32x4 codes[kTiles];
    uint16_t scale[kTiles][kGroups];
    uint8_t zero[kTiles][kGroups];
    const auto load_w = [&](int kt) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        codes[i] = reinterpret_cast<const u32x4 *>(
            a.w_codes + (tile_row[i] * a.K128 + kt) * kTileBytes)[lane];
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const int gg = kt * kGroups + g < G ? kt * kGroups + g : G - 1;
          const int64_t at = (tile_row[i] * G + gg) * kTileN;
          scale[i][g] = (a.w_scales + at)[col];
          if (ZEROS) zero[i][g] = (a.w_zeros + at)[col];
        }
    };
    // The block with the row tiles it has: all of a step's products are
    // independent of each other, and its codes turn into numbers beside the
    // matrix instructions of the step before.
    const auto block = [&](auto count) {
      constexpr int kM = decltype(count)::value;
      f32x4 acc[kM][kTiles];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int i = 0; i < kTiles; ++i) acc[m][i] = f32x4{0, 0, 0, 0};
      // Past the last piece the last one is read again: no load is under a
      // branch, after which every earlier load would have to be waited for.
      const int last = a.K128 - 1;
      load_x(0);
      load_w(0);
      stage_x(0);
      load_x(last < 1 ? last : 1);
      for (int kt = 0; kt <= last; ++kt) {
        const int buf = kt & 1;
        __syncthreads();  // this piece is in LDS, and the other buffer is free
        stage_x(buf ^ 1);
        load_x(kt + 2 < last ? kt + 2 : last);
        u32x4 raw[kTiles];
        float s[kTiles][kGroups], z[kTiles][kGroups];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          raw[i] = codes[i];
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            s[i][g] = bf16_to_f32(scale[i][g]);
            z[i][g] = -zero_of(ZEROS ? (float)zero[i][g] : 8.0f);
          }
        }
        load_w(kt + 1 < last ? kt + 1 : last);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          if (kGroups > 1 && kt * kGroups + g >= G) break;
          f32x4 dot[kM][kTiles];
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            bf16x8 w[kTiles];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) w[i] = codes_bf16(raw[i][g * kPer + j]);
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              const bf16x8 x = xs[buf][m][g * kPer + j][lane];
              f32x4 sum;
              if (j == 0) sum = *reinterpret_cast<const f32x4 *>(&sums[buf][m][g][quad * 4]);
#pragma unroll
              for (int i = 0; i < kTiles; ++i) {
                if (j == 0) dot[m][i] = ZEROS ? sum * z[i][g] : sum;
                dot[m][i] = mul(x, w[i], dot[m][i]);
              }
            }
          }
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            f32x4 sx;
            if (FP8) sx = *reinterpret_cast<const f32x4 *>(&sxs[buf][m][quad * 4]);
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
              for (int v = 0; v < 4; ++v)
                acc[m][i][v] = __builtin_fmaf(s[i][g], FP8 ? dot[m][i][v] * sx[v] : dot[m][i][v],
                                              acc[m][i][v]);
          }
        }
      }
      __syncthreads();  // the buffers are free for the next item
      uint16_t *out0 = a.out + (first + r0) * a.N + ot * kTileN;
      // kept here: worked out before the loop over items, the addresses of all
      // stores would be held (and spilled) through it
      uint32_t at = (uint32_t)(quad * 4) * a.N + col;
      int32_t rows_left = left - quad * 4;
      asm volatile("" : "+v"(at), "+v"(rows_left));
#pragma unroll
      for (int m = 0; m < kM; ++m) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (m * kRows + v >= rows_left) continue;
          uint16_t *row = out0 + (int64_t)(m * kRows + v) * a.N;
#pragma unroll
          for (int i = 0; i < kOut; ++i) {
            float y = acc[m][i][v] * kUnit;
            if (SWIGLU) y = silu_of(y) * (acc[m][kOut + i][v] * kUnit);
            if ((ot + i) * kTileN + col < a.N) row[at + i * kTileN] = f32_to_bf16(y);
          }
        }
      }
    };
    switch (mts) {
      case 4: block(std::integral_constant<int, 4>{}); break;
      case 3: block(std::integral_constant<int, 3>{}); break;
      case 2: block(std::integral_constant<int, 2>{}); break;
      default: block(std::integral_constant<int, 1>{}); break;
    }
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
  // the row blocks of all experts are numbered in 32 bits, each expert's at most the buffer's
  if ((capacity / kBlockRows + 1) * w4->num_experts >= INT32_MAX)
    return failf(EP_ERR_INVALID_ARG, "capacity %lld x %d experts has too many row blocks",
                 (long long)capacity, w4->num_experts);
  if (capacity == 0) return EP_OK;
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), out0 = reinterpret_cast<uintptr_t>(out);
  if (x0 < out0 + (uintptr_t)capacity * w4->out_features * 2 &&
      out0 < x0 + (uintptr_t)capacity * w4->in_features * (fp8 ? 1 : 2))
    return failf(EP_ERR_INVALID_ARG, "out overlaps x");
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
  const int64_t blocks = (a.N16 * (w4->swiglu ? 2 : 1) + kBlockTiles - 1) / kBlockTiles;
  const int64_t experts = capacity / kRows < w4->num_experts ? capacity / kRows : w4->num_experts;
  a.stream_rows = experts * blocks >= kTileRounds * kTileGrid ? kRows : kStreamRows;
  with_product(fp8, w4->group, w_zeros != nullptr, w4->swiglu != 0,
               [&](auto p, auto g, auto z, auto s) {
                 // groups of 32: half the tiles, as four scales each leave no room
                 constexpr int kTiles = g.value == 32 ? 2 : 4;
                 constexpr int kOut = s.value ? kTiles / 2 : kTiles;
                 const dim3 grid((unsigned)((a.N16 + kOut - 1) / kOut),
                                 (unsigned)w4->num_experts);
                 const int64_t hit = capacity < w4->num_experts ? capacity : w4->num_experts;
                 const int64_t bytes = hit * (s.value ? 2 : 1) * a.N16 * a.K128 * kTileBytes;
                 if (bytes > kInfinityCache)
                   hipLaunchKernelGGL(
                       (product_stream_kernel<p.value, g.value, z.value, s.value, kTiles, true>),
                       grid, dim3(kStreamWaves * 64), 0, stream, a);
                 else
                   hipLaunchKernelGGL(
                       (product_stream_kernel<p.value, g.value, z.value, s.value, kTiles, false>),
                       grid, dim3(kStreamWaves * 64), 0, stream, a);
                 if (capacity > a.stream_rows)
                   hipLaunchKernelGGL((product_tile_kernel<p.value, g.value, z.value, s.value>),
                                      dim3(kTileGrid), dim3(256), 0, stream, a,
                                      w4->num_experts);
               });
  return launched("expert product launch");
}

}  // extern "C"
