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
  int32_t out_any;  // product: out is not 16-byte aligned
};

__device__ __forceinline__ f32x4 mul(bf16x8 x, bf16x8 w, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Two transposing reads, at l 0 .. 3 and 4 .. 7 of a lane's eight.
__device__ __forceinline__ bf16x8 read_transposed(const uint8_t *lo, const uint8_t *hi) {
  struct {
    s16x4 lo, hi;
  } v;
  v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)lo);
  v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)hi);
  return __builtin_bit_cast(bf16x8, v);
}

// Eight FP8 codes times their scale, rounded to bf16.
__device__ __forceinline__ u32x4 scaled_bf16(u32x2 codes, float scale) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[i], true);
    w[2 * i] = pack_bf16(lo[0] * scale, lo[1] * scale);
    w[2 * i + 1] = pack_bf16(hi[0] * scale, hi[1] * scale);
  }
  return w;
}

// Rows that begin between 16-byte boundaries (K or N no multiple of 8): tiles of
// 64 x 64, 64 of the sum at a time, through registers, two stages ahead of their
// use.  Layouts in LDS as in the large tiles: "along", where l is consecutive,
// 64 rows of 128 bytes; "across", where m or n is, 64 l of 128 bytes.
// 333 rows of 11 experts, rows' gradient of 1480 x 1001: 18.3 us, bound by the
// latency of 16 stages; 32768 rows of 32 experts, 2047 x 7168: 3.73 ms, 258 TFLOP/s
// (rows' gradient 6.75 ms, weights' 6.86 ms, 140).
constexpr int kAnyTile = 64, kAnyDepth = 64, kAnyGrid = 1024;
constexpr int kAnySide = kAnyTile * kAnyDepth * 2;

template <Kind KIND, bool FP8, bool SWIGLU, typename OUT>
__global__ __launch_bounds__(256) void product_any_kernel(ProductArgs a) {
  static_assert(KIND == kWeightsGrad || !FP8, "FP8 rows of a product are in whole pieces");
  constexpr bool kRowsAcross = KIND == kWeightsGrad, kColsAcross = KIND != kProduct;
  constexpr int kCols = SWIGLU ? kAnyTile / 2 : kAnyTile;  // output columns of a tile
  __shared__ __align__(16) uint8_t stage[2][2][kAnySide];  // of a buffer: rows, columns
  __shared__ int32_t starts[EP_MAX_EXPERTS + 1], totals[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int wr = wave >> 1, wc = wave & 1;
  const int E = a.rows.E, K = a.K, N = a.N;
  const uint8_t *x8 = static_cast<const uint8_t *>(a.x);
  const uint16_t *x16 = static_cast<const uint16_t *>(a.x);
  const int out_cols = KIND == kProduct ? (SWIGLU ? N / 2 : N) : K;
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
    // Piece i of this thread: eight values, of row i of the side and l on from l0
    // (along), or of l i and on from the tile's first row or column (across).
    const auto there = [](int64_t n) { return (int)(n < 0 ? 0 : n < 8 ? n : 8); };
    const auto row_piece = [&](int64_t l0, int i) -> u32x4 {
      const int at = i >> 3, p = (i & 7) * 8;
      if (kRowsAcross) {
        if (l0 + at >= length) return u32x4{0, 0, 0, 0};
        return load_bf16(a.grad + (first + l0 + at) * N + m0 + p, there(N - m0 - p), m0 + p);
      }
      if (at >= rows) return u32x4{0, 0, 0, 0};
      const uint16_t *from = KIND == kProduct ? x16 + (first + at) * K : a.grad + (first + at) * N;
      return load_bf16(from + l0 + p, there(length - l0 - p), (int)l0 + p);
    };
    const auto col_piece = [&](int64_t l0, int i) -> u32x4 {
      const int at = i >> 3, p = (i & 7) * 8;
      if (!kColsAcross) {
        const int c = n0 + at % kCols;
        if (c >= out_cols) return u32x4{0, 0, 0, 0};
        return load_bf16(w + (int64_t)(c + at / kCols * out_cols) * K + l0 + p,
                         there(length - l0 - p), (int)l0 + p);
      }
      if (l0 + at >= length) return u32x4{0, 0, 0, 0};
      if (KIND == kRowsGrad)
        return load_bf16(w + (l0 + at) * K + n0 + p, there(K - n0 - p), n0 + p);
      const int64_t r = first + l0 + at;
      if (FP8) {  // K is a multiple of 128
        if (n0 + p >= K) return u32x4{0, 0, 0, 0};
        return scaled_bf16(load_codes(x8 + r * K + n0 + p, 8, 0),
                           a.x_scales[r * (K / 128) + (n0 + p) / 128]);
      }
      return load_bf16(x16 + r * K + n0 + p, there(K - n0 - p), n0 + p);
    };
    const auto place = [](bool across, int i) {  // of piece i in LDS
      const int at = i >> 3, p = i & 7;
      return at * 128 + (p ^ (across ? (at >> 1 & 3) << 1 : at >> 1 & 7)) * 16;
    };
    struct Pieces {
      u32x4 rows[2], cols[2];
    };
    const auto load = [&](int64_t l0, Pieces *p) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        p->rows[i] = row_piece(l0, tid + i * 256);
        p->cols[i] = col_piece(l0, tid + i * 256);
      }
    };
    const auto put = [&](int buffer, const Pieces &p) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<u32x4 *>(&stage[buffer][0][place(kRowsAcross, tid + i * 256)]) = p.rows[i];
        *reinterpret_cast<u32x4 *>(&stage[buffer][1][place(kColsAcross, tid + i * 256)]) = p.cols[i];
      }
    };
    // 16 rows (or columns) from `from` on, l 32 ks .. + 31
    const auto read = [&](const uint8_t *side, bool across, int from, int ks) -> bf16x8 {
      if (across) {
        const int l = ks * 32 + quad * 8 + l16 / 4, p = from / 8 + l16 % 4 / 2;
        const auto at = [&](int l) { return l * 128 + (p ^ (l >> 1 & 3) << 1) * 16 + l16 % 2 * 8; };
        return read_transposed(side + at(l), side + at(l + 4));
      }
      const int r = from + l16;
      return *reinterpret_cast<const bf16x8 *>(side + r * 128 + ((ks * 4 + quad) ^ (r >> 1 & 7)) * 16);
    };
    f32x4 acc[2][2];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[f][j] = f32x4{0, 0, 0, 0};
    const int64_t steps = (length + kAnyDepth - 1) / kAnyDepth;
    const auto step = [&](int64_t s, Pieces *mine, const Pieces *next) {
      const int buffer = (int)(s & 1);
      __syncthreads();  // this stage is in LDS, the other buffer free
      put(buffer ^ 1, *next);
      load((s + 3) * kAnyDepth, mine);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        bf16x8 r[2], c[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) r[f] = read(stage[buffer][0], kRowsAcross, wr * 32 + f * 16, ks);
#pragma unroll
        for (int j = 0; j < 2; ++j) c[j] = read(stage[buffer][1], kColsAcross, j * 32 + wc * 16, ks);
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[f][j] = mul(c[j], r[f], acc[f][j]);
      }
    };
    if (steps > 0) {
      Pieces p[2];
      load(0, &p[0]);
      __syncthreads();  // the buffers are free of the last item
      put(0, p[0]);
      load(kAnyDepth, &p[1]);
      load(2 * kAnyDepth, &p[0]);
      // stage s + 1 is in p[(s + 1) & 1], s + 2 in the other
      for (int64_t s = 0; s < steps; s += 2) {
        step(s, &p[1], &p[1]);
        if (s + 1 < steps) step(s + 1, &p[0], &p[0]);
      }
    }
    constexpr int kOut = SWIGLU ? 1 : 2;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int j = 0; j < kOut; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int m = wr * 32 + f * 16 + l16, c = n0 + j * 32 + wc * 16 + quad * 4 + v;
          if (c >= out_cols || (KIND == kWeightsGrad ? m0 + m >= N : m >= rows)) continue;
          float y = acc[f][j][v];
          if (SWIGLU) y = silu_of(y) * acc[f][1][v];
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

// --------------------------------------------------------------------------
// Tiles
// --------------------------------------------------------------------------
//
// c[m, n] = sum_l a[m, l] b[n, l] in tiles of 256 x 256, 64 of l at a time.
// "Rows" is the side of m, "columns" that of n.  The matrix instruction takes
// columns first, so that a lane's results are consecutive columns of one row.
//
// A persistent workgroup per compute unit; eight waves of 128 x 64 each, two per
// SIMD, one of which multiplies while the other waits.  Both sides go from memory
// to LDS without registers, whole 128-byte lines (32 of l at a time, half lines,
// need twice the requests: 1018 us in the first case below), and from there to
// the 16 x 16 x 32 instruction, which needs less power than 32 x 32 x 16 for the
// same sums (of random numbers, alone: 2159 and 1885 TFLOP/s).
//   32768 rows of 32 experts, 2048 x 7168        860 to 900 us, 1070 to 1120 TFLOP/s
//   one expert, 4096 x 4096                      800 to 835 us, 1320 to 1370 TFLOP/s
//   rows' gradient of 32, 4096 x 7168           1730 to 1795 us, 1070 to 1110 TFLOP/s
//   weights' gradient of 32, 4096 x 7168        1775 to 1853 us, 1040 to 1080 TFLOP/s
//     with FP8 rows                             2057 to 2160 us,  890 to  935 TFLOP/s
//   128 FP8 rows of 32, 7168 x 2 x 2048          273 us, 6.9 TB/s of weights
// (medians on two boxes: by their power, large cases differ by 5 %)
// What bounds it: of one expert's time the matrix instructions are busy 70 %; the
// clock is then at 1.9 GHz, by power (2.4 with rows and weights of zeros).  With
// 32 uneven experts they are busy 60 %: last tiles of few rows, items that do not
// come out even, and the end of a tile, 8 % of the time.  Tried and slower: four
// waves of 128 x 128 (a third less LDS traffic, but no second wave: 947 us for
// 791), loads all together after the barrier, raised priority of waves that
// multiply, compute units that start apart.

constexpr int kTile = 256;            // rows and columns of a tile
constexpr int kDepth = 64;            // of the sum, per stage
constexpr int kTileWaves = 8;
constexpr int kTileWorkgroups = 256;  // one per compute unit, by its LDS
// Row tiles that go through the columns together (32768 rows, 4096 x 4096, one
// expert: 848 us; 4: 852, 16: 966; 32 experts, 2048 x 7168: 888, 905, 888).
constexpr int kBand = 8;

typedef __attribute__((address_space(3))) uint8_t lds_byte;

// 16 bytes per lane from global memory to LDS, at lds + 16 * lane; zeros where
// the offset is outside the buffer.  Written in assembly because the compiler
// has every LDS read wait for all of its own such loads.  Nothing comes back in
// registers; stage_barrier() waits.  The buffer's words come out of vector
// instructions, after which a vector memory instruction may not read them for
// five wait states; the hardware does not wait, and the compiler does so for its
// own instructions alone.  s_mov_b32 and s_nop 3 are five, whatever comes before
// (and m0's one); in the tiles that takes up to 1.4 % (rows' gradient of 32
// experts, 4096 x 7168: 1730 us, with s_nop 0 1712).  m0 is reserved and no
// clobber can name it: nothing else in these kernels may use it, which a test of
// the built library holds.
// ONCE: non-temporal, for what no other workgroup and no later call reads again.
template <bool ONCE = false>
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t offset, u32x4 buffer) {
  if constexpr (ONCE)
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
        :
        : "s"(uniform((int)lds)), "v"(offset), "s"(buffer)
        : "memory");
  else
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(uniform((int)lds)), "v"(offset), "s"(buffer)
        : "memory");
}

// 4 bytes per lane, at lds + 4 * lane.
__device__ __forceinline__ void load_word_to_lds(uint32_t lds, uint32_t offset, u32x4 buffer) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds"
      :
      : "s"(uniform((int)lds)), "v"(offset), "s"(buffer)
      : "memory");
}

// FP8 rows: codes enter the products times a power of two, and their sums of 128
// leave them times the scale over that power, so that sums are in fp32's range
// where the result is, for weights of any size (by raw codes, those of 2^112 and
// more gave infinities).  Both are exact.  2^-16: 128 codes below 2^9, so scaled,
// sum up to less than the largest weight.  Products then lose what is below
// 2^-133 of the scale (matrix instructions keep fp32's denormal numbers), which
// for scales from 2^32 on would be too much; those take 2^10, with which sums past
// the range are of results past it.
__device__ __forceinline__ bool large_scale(float scale) {  // at least 2^32 and finite
  const uint32_t lo = (127u + 32u) << 23;
  return (__float_as_uint(scale) & 0x7FFFFFFFu) - lo < 0x7F800000u - lo;
}

__device__ __forceinline__ float codes_power(bool large) { return large ? 0x1p10f : 0x1p-16f; }
__device__ __forceinline__ float sums_power(bool large) { return large ? 0x1p-10f : 0x1p16f; }

// Eight FP8 codes times a power of two as bf16.
__device__ __forceinline__ bf16x8 codes_bf16(u32x2 codes, float power) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[2 * i] = __builtin_bit_cast(
        uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], power, false));
    w[2 * i + 1] = __builtin_bit_cast(
        uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], power, true));
  }
  return __builtin_bit_cast(bf16x8, w);
}

template <int kLeft>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(kLeft) : "memory");
}

__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

__device__ __forceinline__ void lds_done() {
  asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
}

// All but the newest kLeft loads and stores are done, and this wave's LDS
// reads, and so for every wave of the workgroup.
template <int kLeft>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(kLeft) : "memory");
}

// Two 16 bytes of a row per lane, rows by lane % 16, become those of rows
// lane % 8 (a) and lane % 8 + 8 (b), the second ones in lanes 8 .. 15 of each 16.
__device__ __forceinline__ void halve_rows(u32x4 *a, u32x4 *b) {
  constexpr int kRor8 = 0x128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = (int)(*a)[i], y = (int)(*b)[i];
    (*a)[i] = (uint32_t)__builtin_amdgcn_update_dpp(x, y, kRor8, 0xF, 0xC, false);
    (*b)[i] = (uint32_t)__builtin_amdgcn_update_dpp(y, x, kRor8, 0xF, 0x3, false);
  }
}

__device__ __forceinline__ u32x4 buffer_of(const void *base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)uniform((int)p), (uint32_t)uniform((int)(p >> 32)) & 0xFFFFu,
               (uint32_t)uniform((int)bytes), 0x00020000u};
}

constexpr uint32_t kNowhere = 0x80000000u;  // an offset outside every buffer

// A piece of work: one tile of one expert.
struct Item {
  int e;
  int64_t first;   // the expert's first row
  int rows;        // rows of the tile (its rows of the weights for the weights' gradient)
  int row0;        // of the tile, inside the expert's (or the weight's) rows
  int col0;        // first output column
  int length;      // of the sum
};

// The numbering of items: an expert's tiles are consecutive, in bands of kBand
// row tiles that take the columns one after the other.  A wave finds its items
// in ascending order by itself: it holds the row tiles of 64 experts, one per
// lane, and goes on to the next 64 when it is past them.
template <Kind KIND, int kRowTile, typename OUT>
struct Items {
  const ProductArgs &a;
  int row_tiles, col_tiles;  // of the weights' gradient; of all kinds
  int chunk = -1;            // experts 64 chunk .. + 63
  int32_t before = 0, end = 0;     // row tiles before the chunk's, and through it
  int32_t first_tile = 0, tiles = 0;  // of this lane's expert
  static constexpr int64_t kManyItems = 4 * kTileWorkgroups;

  __device__ __forceinline__ int64_t lane_rows(int c) const {  // of expert 64 c + lane
    const int e = c * 64 + (threadIdx.x & 63);
    int64_t first, rows = 0;
    if (e < a.rows.E)
      rows_inside(a.rows.offsets[e], a.rows.counts[e], a.rows.capacity, &first, &rows);
    return rows;
  }
  __device__ __forceinline__ int lane_tiles(int c) const {
    return (int)((lane_rows(c) + kRowTile - 1) / kRowTile);
  }
  static __device__ __forceinline__ uint32_t scan(uint32_t v) {  // of the lanes up to this one
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t up = (uint32_t)__shfl_up((int)v, d);
      v += (int)(threadIdx.x & 63) >= d ? up : 0;
    }
    return v;
  }
  static __device__ __forceinline__ uint32_t lane_of(uint32_t v, int l) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, l);
  }
  // The first items of an XCD and of the next one.  An item of the products costs
  // about the same whatever its rows, as its columns are loaded all the same:
  // eighths of the items.  (By rows the prefill share in FP8 takes 515 us, so 450.)
  // An item of the weights' gradient goes by its expert's rows: eighths of the
  // steps, with the end of an item by what it loads and stores.  (32 experts whose
  // rows differ by a third, 4096 x 7168: 1796 us, by items 1914; FP8 rows 2067,
  // 2303; fp32 added up, 8 experts of 2048 x 7168: 252, 269.)  Few items have to
  // come out even instead (experts of 2048 x 2048, 64 items and 1024 rows each, by
  // steps and by items: 4 experts 55, 39; 8 82, 72; 12 116, 113; 16 140, 138; 24
  // 203, 214; of 128 rows each 12 experts 38, 33 and 16 47, 44).
  __device__ __forceinline__ void eighth(int part, int64_t *from, int64_t *to) const {
    const int lane = threadIdx.x & 63;
    if constexpr (KIND != kWeightsGrad) {
      uint32_t tiles = 0;
      for (int c = 0; c * 64 < a.rows.E; ++c) tiles += lane_tiles(c);
      const int64_t all = (int64_t)lane_of(scan(tiles), 63) * col_tiles, per = (all + 7) / 8;
      *from = part * per < all ? part * per : all;
      *to = *from + per < all ? *from + per : all;
    } else {
      const int64_t items = (int64_t)row_tiles * col_tiles;  // of an expert
      if (a.rows.E * items < kManyItems) {  // few rounds: these have to come out even
        const int64_t all = a.rows.E * items, per = (all + 7) / 8;
        *from = part * per < all ? part * per : all;
        *to = *from + per < all ? *from + per : all;
        return;
      }
      const uint32_t end = (sizeof(OUT) == 4 ? 6 : 4) * (a.add != nullptr ? 2 : 1);
      const auto cost = [&](int c) -> uint32_t {
        return c * 64 + lane < a.rows.E ? (uint32_t)((lane_rows(c) + 63) / 64) + end : 0;
      };
      uint32_t all = 0;
      for (int c = 0; c * 64 < a.rows.E; ++c) all += cost(c);
      all = lane_of(scan(all), 63);
      const uint64_t p0 = (uint64_t)all * part / 8, p1 = (uint64_t)all * (part + 1) / 8;
      *from = *to = a.rows.E * items;
      uint32_t before_chunk = 0;
      for (int c = 0; c * 64 < a.rows.E; ++c) {
        const uint32_t w = cost(c), through = before_chunk + scan(w), w0 = through - w;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t p = i == 0 ? p0 : p1;
          const uint64_t here = __ballot(w0 <= p && p < through);
          if (here == 0) continue;
          const int l = __builtin_ctzll(here);
          *(i == 0 ? from : to) =
              (c * 64 + l) * items + (int64_t)(p - lane_of(w0, l)) * items / lane_of(w, l);
        }
        before_chunk = lane_of(through, 63);
      }
    }
  }
  // item is one of them, and not less than at the call before
  __device__ __forceinline__ void get(int64_t item, Item *it, int out_cols_per_tile) {
    const int32_t block = uniform((int)(item / col_tiles));  // as if rows came first
    int e, high, start;
    if (KIND == kWeightsGrad) {
      e = uniform(block / row_tiles);
      high = row_tiles;
      start = e * row_tiles;
    } else {
      while (block >= end) {
        ++chunk;
        before = end;
        tiles = lane_tiles(chunk);
        int at = tiles;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const int up = __shfl_up(at, d);
          at += (int)(threadIdx.x & 63) >= d ? up : 0;
        }
        first_tile = before + at - tiles;
        end = before + __builtin_amdgcn_readlane(at, 63);
      }
      const uint64_t from_here = __ballot(tiles > 0 && first_tile <= block);
      const int l = 63 - __builtin_clzll(from_here);
      e = chunk * 64 + l;
      start = __builtin_amdgcn_readlane(first_tile, l);
      high = __builtin_amdgcn_readlane(tiles, l);
    }
    int64_t rows;
    rows_inside(uniform(a.rows.offsets[e]), uniform(a.rows.counts[e]), a.rows.capacity, &it->first,
                &rows);
    const int64_t in_expert = item - (int64_t)start * col_tiles;
    const int band = (int)(in_expert / ((int64_t)kBand * col_tiles));
    const int in_band = (int)(in_expert - (int64_t)band * kBand * col_tiles);
    high = high - band * kBand < kBand ? high - band * kBand : kBand;
    const int rt = uniform(band * kBand + in_band % high), ct = uniform(in_band / high);
    it->e = e;
    it->row0 = rt * kRowTile;
    it->col0 = ct * out_cols_per_tile;
    const int64_t all = KIND == kWeightsGrad ? (int64_t)a.N : rows;
    it->rows = (int)(all - it->row0 < kRowTile ? all - it->row0 : kRowTile);
    it->length = KIND == kProduct ? a.K : KIND == kRowsGrad ? a.N : (int)rows;
  }
};

// One side of a stage is four loads per wave.  "Along": l is consecutive in
// memory; 8 rows of 128 bytes per load, the 16-byte pieces of row r in LDS at
// piece ^ (r / 2) % 8, so that the reads of 16 lanes of one piece cover all
// banks.  "Across": m (or n) is consecutive; two l of 512 bytes per load, units
// of 32 bytes at unit ^ across_swizzle(l), so that the 8 l of 32 lanes of a
// transposing read do.  What is past the end of the sum, or of the rows, is
// outside the load's buffer and zero; a column that is not there spoils its own
// results alone.
__device__ __forceinline__ int across_swizzle(int l) { return (l & 3) | (l >> 3 & 1) << 2; }

// Of FP8 codes: 16-byte pieces, for 16 l of 32 lanes, lines of 256 or 128 bytes.
__device__ __forceinline__ int across_swizzle8(int line, int l) {
  return line == 256 ? l & 15 : l >> 1 & 7;
}

template <Kind KIND, bool FP8, bool SWIGLU, typename OUT, bool SMALL, bool ONCE>
__global__ __launch_bounds__(kTileWaves * 64, SMALL ? 4 : 2) void product_tile_kernel(
    ProductArgs a) {
  constexpr bool kRowsAcross = KIND == kWeightsGrad, kColsAcross = KIND != kProduct;
  // Which side is x in FP8.  Rows: codes enter the instructions exactly, and
  // scales are applied to the sums of 128, in accumulators of their own, for which
  // 128 rows leave the registers.  Columns (weights' gradient): x is rounded to
  // bf16, as the scales go by the rows that are summed over; each value once, a
  // stage ahead, into a place that the instructions' operands are read from.
  // (By each wave for itself, two of them the same values, 32 experts, 4096 x 7168:
  // 2503 us, so 2412.)
  constexpr bool kRows8 = KIND == kProduct && FP8, kCols8 = KIND == kWeightsGrad && FP8;
  constexpr int kRowTile = SMALL || kRows8 ? kTile / 2 : kTile;
  constexpr int kColTile = SMALL ? kTile / 2 : kTile;
  constexpr int kOutTile = SWIGLU ? kColTile / 2 : kColTile;
  constexpr int kJ = kColTile / 64;  // 16 columns each, of a wave
  // Stages in LDS: 160 KB, all of it, in bf16.  FP8 rows leave place for one more
  // of both sides (32768 rows of 32 experts, 7168 x 4096: 2125 us, without 2178).
  constexpr bool kDeep = kRows8 && !SMALL;
  constexpr int kColSlots = kDeep ? 4 : 3, kRowSlots = kDeep ? 3 : 2;
  constexpr int kRowElem = kRows8 ? 1 : 2, kColElem = kCols8 ? 1 : 2;
  constexpr int kRowBytes = kRowTile * kDepth * kRowElem, kColBytes = kColTile * kDepth * kColElem;
  constexpr int kRowLoads = kRowBytes / (kTileWaves * 1024);  // of a wave and stage
  constexpr int kColLoads = kColBytes / (kTileWaves * 1024);
  constexpr int kColPart = kColLoads + kCols8;  // with the scales
  constexpr int kRowPart = kRowLoads + kRows8;
  // loads that are newer than the next stage's, before this one's of rows
  constexpr int kNewer = kDeep ? 2 * kColPart + kRowPart : kColPart;
  constexpr int kRowsAt = kColSlots * kColBytes, kWideAt = kRowsAt + kRowSlots * kRowBytes;
  constexpr int kScalesAt = kWideAt + (kCols8 ? kColTile * kDepth * 2 : 0);
  constexpr int kScaleBytes = 512;  // of a stage: 128 rows, or 64 of l for two blocks
  __shared__ __align__(1024) uint8_t
      stage[kScalesAt + (FP8 ? (kColSlots + 1) * kScaleBytes : 0)];
  // non-temporal stores of the weights' gradient, which nobody reads soon (bf16, 32
  // experts of 4096 x 7168: 2056 us, without 2140)
  constexpr int kOnceOut = KIND == kWeightsGrad && !SMALL ? 2 : 0;
  constexpr int kSize = sizeof(OUT);
  constexpr int kHere = SWIGLU ? kJ / 2 : kJ;  // 16 columns of the results each
  // stores of a wave, per 64 rows of a tile
  constexpr int kStores = kSize == 4 ? 2 * kHere : kHere == 4 ? 4 : 2;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int wr = wave >> 2, wc = wave & 3;  // of the wave's rows and columns
  const int K = a.K, N = a.N;
  const int out_cols = KIND == kProduct ? (SWIGLU ? N / 2 : N) : K;
  typedef Items<KIND, kRowTile, OUT> AllItems;
  AllItems items{a, (N + kRowTile - 1) / kRowTile, (out_cols + kOutTile - 1) / kOutTile};
  // The items of an XCD (workgroups id % 8) are consecutive, so that the
  // workgroups that share its L2 share rows and columns.
  int64_t from, to;
  items.eighth(blockIdx.x % 8, &from, &to);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_byte *)stage;

  // Where a lane's 16 bytes of a side's first load come from, from the wave's
  // base on, and how far on each further load is.
  const int row_pitch = (KIND == kProduct ? K : N) * kRowElem, col_pitch = K * kColElem;
  // Across, a row in LDS is one l.
  constexpr int kRowLine = kRowTile * 2, kColLine = kColTile * kColElem;
  constexpr int kRowPer = kRows8 ? 16 : kRowsAcross ? 1024 / kRowLine : 8;  // rows, or l, of a load
  constexpr int kColPer = kColsAcross ? 1024 / kColLine : 8;
  const int piece_along = (lane & 7) ^ ((wave & 1) << 2 | lane >> 4);
  const int piece_along8 = (lane & 3) ^ lane >> 4;
  const auto across_from = [&](int line, int per, int pitch, bool codes) -> uint32_t {
    const int l = lane / (line / 16), piece = lane % (line / 16), at = wave * per + l;
    return l * pitch + (piece ^ (codes ? across_swizzle8(line, at) : across_swizzle(at) << 1)) * 16;
  };
  const uint32_t row_off = kRows8        ? (lane >> 2) * row_pitch + piece_along8 * 16
                           : kRowsAcross ? across_from(kRowLine, kRowPer, row_pitch, false)
                                         : (lane >> 3) * row_pitch + piece_along * 16;
  const uint32_t col_off = kColsAcross ? across_from(kColLine, kColPer, col_pitch, kCols8)
                                       : (lane >> 3) * col_pitch + piece_along * 16;
  const uint32_t row_step = (kRowsAcross ? 8 * kRowPer : 64) * row_pitch;
  const uint32_t col_step = (kColsAcross ? 8 * kColPer : SWIGLU ? 32 : 64) * col_pitch;

  // Where a lane's parts of the instructions' operands are in a slot: of its
  // first 16 rows and columns.
  const int along = l16 * 128 + (quad ^ l16 >> 1) * 16;
  const auto across = [&](int line) {
    return (quad * 8 + l16 / 4) * line + ((quad & 1) << 2 | l16 / 4) * 32 + l16 % 4 * 8;
  };
  const int along8 = l16 * 64 + (quad >> 1 ^ l16 >> 2) * 16 + (quad & 1) * 8;
  const int row_at = kRowsAt + (kRows8        ? along8 + wr * 1024
                                : kRowsAcross ? across(kRowLine) ^ wr * 32
                                              : along + wr * 2048);
  constexpr int kOperandLine = kColTile * 2;
  const int col_at = kColsAcross ? (across(kOperandLine) ^ wc * kJ * 32) + (kCols8 ? kWideAt : 0)
                                 : along + wc * kJ * 2048;
  const auto read_across = [&](int at, int line) {
    return read_transposed(stage + at, stage + at + 4 * line);
  };
  // rows 32 f + 16 wr .. + 15, columns 16 (kJ wc + j) .. + 15, half ks of a stage
  const auto read_row = [&](int slot, int ks, int f) {
    const int at = slot * kRowBytes + row_at;
    if constexpr (kRows8)
      return *reinterpret_cast<const u32x2 *>(stage + (at ^ ks * 32) + f * 2048);
    else if constexpr (kRowsAcross)
      return read_across((at ^ f * 64) + ks * 32 * kRowLine, kRowLine);
    else
      return *reinterpret_cast<const bf16x8 *>(stage + (at ^ ks * 64) + f * 4096);
  };
  const auto read_col = [&](int slot, int ks, int j) {
    const int at = (kCols8 ? 0 : slot * kColBytes) + col_at;
    if constexpr (kColsAcross)
      return read_across((at ^ j * 32) + ks * 32 * kOperandLine, kOperandLine);
    else
      return *reinterpret_cast<const bf16x8 *>(stage + (at ^ ks * 64) + j * 2048);
  };

  // The loads run ahead of the products, through the items' ends: columns two
  // stages ahead (FP8 columns: three, one of them for the rounding), in three
  // slots, and rows one, in two; with FP8 rows one more.  (With two slots of both
  // the decode share in bf16 takes 364 us, so 311, both without non-temporal loads.)
  struct Loads {
    const uint8_t *base = nullptr, *scales = nullptr;
    int bytes = 0;  // along: from the base to the last row's end
    int skip = 0;   // across: bytes before the tile's first column
    int scale_bytes = 0, scale_skip = 0;  // the same of the scales
    int left = 0;      // of the item's sum, from the next stage on
    int there = 0;     // bytes of the next stage from the base on
    uint32_t off = 0;  // of this lane's first load
  };
  Loads rows, cols;
  const int64_t next = gridDim.x / 8;
  int64_t row_item = from + blockIdx.x / 8, col_item = row_item;
  AllItems row_items = items, col_items = items;
  const auto start_rows = [&]() {
    Item it;
    row_items.get(row_item, &it, kOutTile);
    rows.left = it.length;
    if (kRowsAcross) {
      rows.skip = it.row0 * 2;
      rows.base = reinterpret_cast<const uint8_t *>(a.grad) +
                  (it.first + wave * kRowPer) * (int64_t)row_pitch + rows.skip;
    } else {
      rows.base = static_cast<const uint8_t *>(KIND == kProduct ? a.x : a.grad) +
                  (it.first + it.row0 + wave * kRowPer) * (int64_t)row_pitch;
      rows.bytes = (it.rows - wave * kRowPer) * row_pitch;
    }
    if (kRows8) {
      rows.scales = reinterpret_cast<const uint8_t *>(a.x_scales) +
                    (it.first + it.row0) * (int64_t)(K / 128) * 4;
      rows.scale_bytes = it.rows * (K / 128) * 4;
    }
  };
  const auto start_cols = [&]() {
    Item it;
    col_items.get(col_item, &it, kOutTile);
    cols.left = it.length;
    if (kColsAcross) {
      cols.skip = it.col0 * kColElem;
      cols.base = (KIND == kRowsGrad
                       ? reinterpret_cast<const uint8_t *>(a.w) +
                             ((int64_t)it.e * N + wave * kColPer) * col_pitch
                       : static_cast<const uint8_t *>(a.x) +
                             (it.first + wave * kColPer) * (int64_t)col_pitch) +
                  cols.skip;
    } else {
      // SwiGLU: 8 kJ columns of the gate, then the same of up, for each wc
      const int n = it.col0 + (SWIGLU ? wave / (2 * kJ) * 8 * kJ + wave % kJ * 8 : wave * 8);
      const int there = out_cols - n < kTile ? out_cols - n : kTile;
      cols.base = reinterpret_cast<const uint8_t *>(a.w) +
                  ((int64_t)it.e * N + n + (SWIGLU ? wave / kJ % 2 * out_cols : 0)) * col_pitch;
      cols.bytes = there * col_pitch;
    }
    if (kCols8) {
      cols.scale_skip = (it.col0 / 128 + (wave & 1)) * 4;
      cols.scales = reinterpret_cast<const uint8_t *>(a.x_scales) +
                    it.first * (int64_t)(K / 128) * 4 + cols.scale_skip;
    }
  };
  // Loads go out one at a time between products: together they would hold up
  // every wave until the last was taken.
  const auto see = [&](Loads *x, bool is_across, int pitch, uint32_t off, int per) {
    const int l2 = x->left - wave * per < kDepth ? x->left - wave * per : kDepth;
    const int n = x->left <= 0 ? 0 : is_across ? l2 * pitch - x->skip : x->bytes;
    x->there = uniform(n < 0 ? 0 : n);
    // FP8 rows end with whole stages
    x->off = is_across || kRows8 || piece_along * 8 < x->left ? off : kNowhere;
  };
  const auto see_cols = [&]() {
    // a sum's end in the columns: rows of 128 in FP8 have none within a stage
    see(&cols, kColsAcross, col_pitch, col_off, kColPer);
  };
  const auto see_rows = [&]() { see(&rows, kRowsAcross, row_pitch, row_off, kRowPer); };
  // The scales of a stage, by the first two waves; the others' loads bring
  // zeros to a place that nobody reads, so that all waves count alike.
  const auto load_row_scales = [&](int slot) {
    if constexpr (kRows8) {
      const uint32_t at = kScalesAt + (wave < 2 ? slot * kScaleBytes + wave * 256
                                                : kColSlots * kScaleBytes);
      const uint32_t off = (wave * 64 + lane) * (uint32_t)(K / 128) * 4 + (K - rows.left) / 128 * 4;
      load_word_to_lds(lds0 + at, off,
                       buffer_of(rows.scales, wave < 2 && rows.left > 0 ? rows.scale_bytes : 0));
    }
  };
  const auto load_col_scales = [&](int slot) {
    if constexpr (kCols8) {
      const uint32_t at = kScalesAt + (wave < 2 ? slot * kScaleBytes + wave * 256
                                                : kColSlots * kScaleBytes);
      const int there = (cols.left < kDepth ? cols.left : kDepth) * (K / 128) * 4 - cols.scale_skip;
      load_word_to_lds(lds0 + at, lane * (uint32_t)(K / 128) * 4,
                       buffer_of(cols.scales, wave < 2 && there > 0 ? there : 0));
    }
  };
  const auto load_rows = [&](int slot, int i) {
    load_to_lds(lds0 + kRowsAt + slot * kRowBytes + wave * 1024 + i * 8192,
                rows.off + i * row_step, buffer_of(rows.base, rows.there));
    if (i == kRowLoads - 1) load_row_scales(slot);
  };
  const auto load_cols = [&](int slot, int i) {
    load_to_lds<ONCE>(lds0 + slot * kColBytes + wave * 1024 + i * 8192, cols.off + i * col_step,
                      buffer_of(cols.base, cols.there));
    if (i == kColLoads - 1) load_col_scales(slot);
  };
  const auto on = [&](Loads *x, bool is_across, int pitch, int elem) {
    x->base += is_across ? (int64_t)kDepth * pitch : kDepth * elem;
    x->bytes -= kDepth * elem;
    x->left -= kDepth;
  };
  // On to the next item that has a sum.
  const auto find_cols = [&]() {
    while (cols.left <= 0 && col_item < to) {
      col_item += next;
      if (col_item < to) start_cols();
    }
    see_cols();
  };
  const auto find_rows = [&]() {
    while (rows.left <= 0 && row_item < to) {
      row_item += next;
      if (row_item < to) start_rows();
    }
    see_rows();
  };
  const auto cols_on = [&]() {
    on(&cols, kColsAcross, col_pitch, kColElem);
    if (kCols8) cols.scales += (int64_t)kDepth * (K / 128) * 4;
    find_cols();
  };
  const auto rows_on = [&]() {
    on(&rows, kRowsAcross, row_pitch, kRowElem);
    find_rows();
  };
  // FP8 columns: this thread's pieces of 8 codes of a stage, rounded to bf16 and
  // put where the operands are read.  A wave writes whole lines, so that its
  // writes cover all banks (in the case above 5.05 M cycles; with 16 codes per
  // lane, and so gaps of 16 bytes between lanes, 5.40 M).
  constexpr int kPieces = kColLine / 8, kMine = kCols8 ? kPieces / 8 : 1;
  u32x4 wide[kMine];
  const auto widen = [&](int slot) {
    if constexpr (kCols8) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int l = wave * 8 + i * (64 / kPieces) + lane / kPieces, p = lane % kPieces;
        const u32x2 codes = *reinterpret_cast<const u32x2 *>(
            stage + slot * kColBytes + l * kColLine + (p / 2 ^ across_swizzle8(kColLine, l)) * 16 +
            p % 2 * 8);
        const float scale = *reinterpret_cast<const float *>(
            stage + kScalesAt + slot * kScaleBytes + p / 16 * 256 + l * 4);
        wide[i] = scaled_bf16(codes, scale);
      }
    }
  };
  const auto put_wide = [&]() {
    if constexpr (kCols8) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int l = wave * 8 + i * (64 / kPieces) + lane / kPieces, p = lane % kPieces;
        *reinterpret_cast<u32x4 *>(stage + kWideAt + l * kOperandLine +
                                   (p ^ across_swizzle(l) << 1) * 16) = wide[i];
      }
    }
  };

  if (col_item < to) {
    start_cols();
    start_rows();
  }
  find_cols();
  find_rows();
#pragma unroll
  for (int i = 0; i < kColLoads; ++i) load_cols(0, i);
  cols_on();
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) load_rows(0, i);
  rows_on();
#pragma unroll
  for (int i = 0; i < kColLoads; ++i) load_cols(1, i);
  cols_on();
  if constexpr (kCols8) {
#pragma unroll
    for (int i = 0; i < kColLoads; ++i) load_cols(2, i);
    cols_on();
    stage_barrier<kColPart>();
    widen(0);
    put_wide();
    lds_barrier();
  } else if constexpr (kDeep) {
#pragma unroll
    for (int i = 0; i < kRowLoads; ++i) load_rows(1, i);
    rows_on();
#pragma unroll
    for (int i = 0; i < kColLoads; ++i) load_cols(2, i);
    cols_on();
    stage_barrier<kNewer>();
  } else {
    stage_barrier<kColPart>();
  }
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) load_rows(kRowSlots - 1, i);
  rows_on();
  int col_slot = 0, row_slot = 0;  // of the next stage
  int stored = 0;                  // stores behind the newest loads
  // Here and at the end of each item: the next stage is there, and the columns
  // and rows of the one after it (FP8 rows: the two) are on their way.
  for (int64_t item = from + blockIdx.x / 8; item < to; item += next) {
    Item it;
    items.get(item, &it, kOutTile);
    const int steps = (int)(((uint32_t)it.length + kDepth - 1) / kDepth);

    const auto tile = [&](auto count) {
      constexpr int kM = decltype(count)::value;  // 64 rows each
      f32x4 acc[2 * kM][kJ], part[kRows8 ? 2 * kM : 1][kJ];
#pragma unroll
      for (int f = 0; f < 2 * kM; ++f)
#pragma unroll
        for (int j = 0; j < kJ; ++j) acc[f][j] = f32x4{0, 0, 0, 0};
      typedef typename std::conditional<kRows8, u32x2, bf16x8>::type RowRaw;
      bf16x8 c[2][kJ];
      RowRaw r[2][kM];
      float row_scale[2][kM];
      // Of a block of 128, for the codes' power: whether a scale of the wave's rows
      // is.  (A power per row does not fit the registers of the small tiles: 4096
      // rows of 8 experts, 2048 x 2048: 70 us.  So 58.5, all by 2^-16 55.5, by raw
      // codes 56; 32768 rows of 32, 7168 x 4096: 2248, 2244, 2215 and 2191.)
      bool large = false;
      const auto scale_of = [&](int slot, int f) {  // of row fragment f
        return *reinterpret_cast<const float *>(stage + kScalesAt + slot * kScaleBytes +
                                                (f * 32 + wr * 16 + l16) * 4);
      };
      const auto look_at_scales = [&](int slot) {
        if constexpr (kRows8) {
          bool any = false;
#pragma unroll
          for (int f = 0; f < 2 * kM; ++f) any |= large_scale(scale_of(slot, f));
          large = __any(any);
        }
      };
      const auto read_cols = [&](int slot, int ks) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) c[ks][j] = read_col(slot, ks, j);
      };
      const auto read_rows = [&](int slot, int ks, int h) {
#pragma unroll
        for (int f = 0; f < kM; ++f) r[h][f] = read_row(slot, ks, h * kM + f);
      };
      const auto products = [&](bool fresh, int ks, int h, auto loads, auto load_one) {
        constexpr int kCount = decltype(loads)::value;
#pragma unroll
        for (int f = 0; f < kM; ++f) {
          bf16x8 x;
          if constexpr (kRows8)
            x = codes_bf16(r[h][f], codes_power(large));
          else
            x = r[h][f];
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            if constexpr (kRows8)
              part[h * kM + f][j] =
                  mul(c[ks][j], x, fresh ? f32x4{0, 0, 0, 0} : part[h * kM + f][j]);
            else
              acc[h * kM + f][j] = mul(c[ks][j], x, acc[h * kM + f][j]);
          }
#pragma unroll
          for (int i = f * kCount / kM; i < (f + 1) * kCount / kM; ++i) load_one(i);
        }
      };
      const auto add_scaled = [&](int h) {
#pragma unroll
        for (int f = 0; f < kM; ++f)
#pragma unroll
          for (int j = 0; j < kJ; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              acc[h * kM + f][j][v] = __builtin_fmaf(row_scale[h][f], part[h * kM + f][j][v],
                                                     acc[h * kM + f][j][v]);
      };
      const auto none = std::integral_constant<int, 0>{};
      const auto nothing = [](int) {};
      if (steps > 0) {
        read_cols(col_slot, 0);
        read_rows(row_slot, 0, 0);
        look_at_scales(row_slot);
      }
      // A stage.  Each quarter's operands are read during the one before.
      // second: of the two that share a scale of FP8 rows.
      const auto step = [&](int s, auto second) {
        constexpr bool kSecond = decltype(second)::value, kFresh = !kSecond;
        constexpr int kEarly = (kColLoads + 1) / 2;
        const int next_col = col_slot == kColSlots - 1 ? 0 : col_slot + 1;
        const int next_row = row_slot == kRowSlots - 1 ? 0 : row_slot + 1;
        // the next columns go where the last stage's were, or, as FP8 columns have
        // been put elsewhere, this one's
        const int free_col = kCols8 ? col_slot : col_slot == 0 ? kColSlots - 1 : col_slot - 1;
        read_rows(row_slot, 0, 1);
        products(kFresh, 0, 0, std::integral_constant<int, kEarly>{},
                 [&](int i) { load_cols(free_col, i); });
        read_cols(col_slot, 1);
        read_rows(row_slot, 1, 0);
        widen(next_col);
        products(kFresh, 0, 1, std::integral_constant<int, kColLoads - kEarly>{},
                 [&](int i) { load_cols(free_col, i + kEarly); });
        cols_on();
        read_rows(row_slot, 1, 1);
        if constexpr (kRows8 && kSecond) {
#pragma unroll
          for (int f = 0; f < 2 * kM; ++f)
            row_scale[f / kM][f % kM] = scale_of(row_slot, f) * sums_power(large);
        }
        products(false, 1, 0, none, nothing);
        // the next stage is there, and this one's slots are free
        if (s < (kDeep ? 2 : 1) && stored == kStores * (kRowTile / 64))
          stage_barrier<kNewer + kStores * (kRowTile / 64)>();
        else
          stage_barrier<kNewer>();
        if constexpr (kCols8) {
          put_wide();
          products(false, 1, 1, std::integral_constant<int, kRowLoads>{},
                   [&](int i) { load_rows(row_slot, i); });
          lds_barrier();
          read_cols(next_col, 0);
          read_rows(next_row, 0, 0);
        } else {
          read_cols(next_col, 0);
          read_rows(next_row, 0, 0);
          products(false, 1, 1, std::integral_constant<int, kRowLoads>{},
                   [&](int i) { load_rows(row_slot, i); });
        }
        rows_on();
        if constexpr (kRows8 && kSecond) {
          add_scaled(0);
          add_scaled(1);
          look_at_scales(next_row);
        }
        col_slot = next_col;
        row_slot = next_row;
      };
      if constexpr (kRows8) {
        for (int s = 0; s < steps; s += 2) {  // rows of whole blocks of 128
          step(s, std::false_type{});
          step(s + 1, std::true_type{});
        }
      } else {
        for (int s = 0; s < steps; ++s) step(s, std::false_type{});
      }
      // A lane has row l16 and columns 4 quad .. + 3 of each 16.  The values
      // change places between lanes so that a store writes whole lines (with 64
      // bytes per row the weights' gradient of 32 experts, 4096 x 7168, takes 2232
      // us instead of 2040; through LDS 2056).  Rows that are not there are outside
      // the buffer of the stores.
      // rows of results that begin between 16-byte boundaries
      const bool any_store = KIND == kProduct && (out_cols % 8 != 0 || a.out_any);
      stored = steps > 0 && !any_store ? kStores * kM : 0;
      const int64_t to_row =
          KIND == kWeightsGrad ? (int64_t)it.e * N + it.row0 : it.first + it.row0;
      const int pitch = out_cols * kSize;
      const int64_t skip = (to_row * out_cols + it.col0) * kSize;
      const auto out = __builtin_amdgcn_make_buffer_rsrc(
          static_cast<uint8_t *>(a.out) + skip, 0, it.rows * pitch - it.col0 * kSize, 0x00020000);
      const auto add = __builtin_amdgcn_make_buffer_rsrc(
          static_cast<uint8_t *>(const_cast<void *>(a.add)) + skip, 0,
          a.add == nullptr ? 0 : it.rows * pitch - it.col0 * kSize, 0x00020000);
      // kept here: worked out before the loop over items, these would be held
      // in registers through it
      int at_lane = lane;
      asm volatile("" : "+v"(at_lane));
      const int row = wr * 16 + (at_lane & 15), at_quad = at_lane >> 4;
      const int wave_col = wc * 16 * kHere;  // of the wave's first, in the tile
      const auto from = [&](int r, int col) {  // offset of a row and a column of the wave's
        return it.col0 + wave_col + col < out_cols
                   ? (uint32_t)(r * pitch + (wave_col + col) * kSize) : kNowhere;
      };
      const int row8 = wr * 16 + (at_lane & 7), second = at_lane >> 3 & 1;
      // What is added is loaded kAhead rows of 32 before its use, and so before the
      // stores in between: an element has one lane, so it may be the result itself.
      // (One after the other, fp32 gradients of 8 experts, 2048 x 7168, added up:
      // 317 us, so 263.)
      constexpr int kAhead = 1, kAdds = kSize == 4 ? kHere : kHere / 2 + kHere % 2;
      u32x4 added[kAhead + 1][kAdds];
      const auto load_added = [&](int f) {
        const uint32_t down = f * 32 * pitch;
        u32x4 *b = added[f % (kAhead + 1)];
        if constexpr (kSize == 4) {
#pragma unroll
          for (int j = 0; j < kHere; ++j)  // of the pair j / 2: rows 0 .. 7, then 8 .. 15
            b[j] = __builtin_amdgcn_raw_buffer_load_b128(
                add, from(row8 + j % 2 * 8, (j / 2 * 2 + second) * 16 + at_quad * 4) + down, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < kHere; ++j) {
            const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(
                add, from(row, j * 16 + at_quad * 4) + down, 0, 0);
            b[j / 2][j % 2 * 2] = v[0];
            b[j / 2][j % 2 * 2 + 1] = v[1];
          }
        }
      };
      const bool adding = KIND == kWeightsGrad && a.add != nullptr;
      if (adding) {
#pragma unroll
        for (int f = 0; f < kAhead && f < 2 * kM; ++f) load_added(f);
      }
#pragma unroll
      for (int f = 0; f < 2 * kM; ++f) {
        const uint32_t down = f * 32 * pitch;
        if (adding && f + kAhead < 2 * kM) load_added(f + kAhead);
        const u32x4 *b = added[f % (kAhead + 1)];
        if constexpr (kSize == 4) {
#pragma unroll
          for (int j = 0; j < kHere; j += 2) {
            u32x4 y[2] = {__builtin_bit_cast(u32x4, acc[f][j]),
                          __builtin_bit_cast(u32x4, acc[f][j + 1])};
            halve_rows(&y[0], &y[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t at = from(row8 + h * 8, (j + second) * 16 + at_quad * 4) + down;
              if (adding)
                y[h] = __builtin_bit_cast(u32x4, __builtin_bit_cast(f32x4, y[h]) +
                                                     __builtin_bit_cast(f32x4, b[j + h]));
              __builtin_amdgcn_raw_buffer_store_b128(y[h], out, at, 0, kOnceOut);
            }
          }
        } else {
          uint32_t w[kHere][2];
#pragma unroll
          for (int j = 0; j < kHere; ++j) {
            f32x4 y = acc[f][j];
            if constexpr (SWIGLU) {
#pragma unroll
              for (int v = 0; v < 4; ++v) y[v] = silu_of(y[v]) * acc[f][kJ / 2 + j][v];
            }
            if (adding) {
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const uint32_t pair = b[j / 2][j % 2 * 2 + v / 2];
                y[v] += __uint_as_float(v % 2 ? pair & 0xFFFF0000u : pair << 16);
              }
            }
            w[j][0] = pack_bf16(y[0], y[1]);
            w[j][1] = pack_bf16(y[2], y[3]);
          }
          if constexpr (kHere == 1) {
            if (any_store) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(w[0][i / 2] >> (i % 2 * 16)), out,
                                                      from(row, at_quad * 4 + i) + down, 0, 0);
            } else {
              __builtin_amdgcn_raw_buffer_store_b64(u32x2{w[0][0], w[0][1]}, out,
                                                    from(row, at_quad * 4) + down, 0, 0);
            }
          } else {
            // lane quad (q1, q0) with 16 columns (j1, j0) becomes lane quad (j0, q1)
            // with 8 columns q0 of piece j1
            u32x4 v[kHere / 2];
#pragma unroll
            for (int j = 0; j < kHere; j += 2)
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const auto x = __builtin_amdgcn_permlane32_swap(w[j][p], w[j + 1][p], false, false);
                const auto y = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
                v[j / 2][p] = y[0];
                v[j / 2][2 + p] = y[1];
              }
            if (any_store) {
#pragma unroll
              for (int j = 0; j < kHere; j += 2)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  __builtin_amdgcn_raw_buffer_store_b16(
                      (uint16_t)(v[j / 2][i / 2] >> (i % 2 * 16)), out,
                      from(row, j * 16 + at_quad * 8 + i) + down, 0, 0);
            } else if constexpr (kHere == 2) {
              __builtin_amdgcn_raw_buffer_store_b128(v[0], out, from(row, at_quad * 8) + down, 0,
                                                     kOnceOut);
            } else {
              halve_rows(&v[0], &v[1]);
#pragma unroll
              for (int h = 0; h < 2; ++h)
                __builtin_amdgcn_raw_buffer_store_b128(
                    v[h], out, from(row8 + h * 8, second * 32 + at_quad * 8) + down, 0, kOnceOut);
            }
          }
        }
      }
    };
    if constexpr (kRowTile < kTile) {
      if (it.rows <= 64)
        tile(std::integral_constant<int, 1>{});
      else
        tile(std::integral_constant<int, 2>{});
    } else {
      switch ((it.rows + 63) / 64) {
        case 1: tile(std::integral_constant<int, 1>{}); break;
        case 2: tile(std::integral_constant<int, 2>{}); break;
        case 3: tile(std::integral_constant<int, 3>{}); break;
        default: tile(std::integral_constant<int, 4>{}); break;
      }
    }
  }
  stage_barrier<0>();  // no load may write to LDS after the end
}

// --------------------------------------------------------------------------
// Few rows
// --------------------------------------------------------------------------
//
// A workgroup has 32 rows of one expert's weights (SwiGLU: 16 of the gate and 16
// of up), all of the sum and 16 rows of x at a time; the sum is dealt to its
// waves in chunks, and theirs are added in LDS at the end.  Each wave loads for
// itself, two chunks ahead and without barriers: reading the weights is the
// bound, and what counts is how much of it is on its way.  One token, 8 of 64
// experts, 4096 x 2 x 1024: 24.5 us, 5.5 TB/s (by tiles 53); FP8 rows, 7168 x 2 x
// 2048: 76 us (110).
constexpr int kStreamWaves = 4, kStreamStages = 3, kStreamRows = 16, kStreamCols = 32;

template <bool FP8, bool SWIGLU, bool ONCE>
__global__ __launch_bounds__(kStreamWaves * 64) void product_stream_kernel(ProductArgs a) {
  // 128 bytes of each row of x are a chunk
  constexpr int kChunk = FP8 ? 128 : 64;
  constexpr int kWBytes = kStreamCols * kChunk * 2, kXBytes = kStreamRows * 128;
  constexpr int kWLoads = kWBytes / 1024, kXLoads = kXBytes / 1024;
  constexpr int kLoads = kWLoads + kXLoads + FP8;
  constexpr int kStages = kStreamStages;
  constexpr int kBytes = kWBytes + kXBytes + (FP8 ? 256 : 0);
  constexpr int kOutCols = SWIGLU ? kStreamCols / 2 : kStreamCols;
  __shared__ __align__(1024) uint8_t stage[kStreamWaves][kStages][kBytes];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int e = blockIdx.y, K = a.K, N = a.N;
  const int out_cols = SWIGLU ? N / 2 : N;
  const int n0 = blockIdx.x * kOutCols;
  int64_t first, rows;
  rows_inside(uniform(a.rows.offsets[e]), uniform(a.rows.counts[e]), a.rows.capacity, &first, &rows);
  if (rows == 0) return;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_byte *)&stage[wave][0][0];
  const int chunks = (K + kChunk - 1) / kChunk;
  const int x_pitch = K * (FP8 ? 1 : 2), w_pitch = K * 2;
  // Rows of 128 bytes in LDS, 8 per load; in FP8 a row of the weights is two, of
  // 64 columns each.  Pieces swizzled as in the tiles.
  const int at_row = lane >> 3, piece = (lane & 7) ^ (lane >> 4);  // rows 0 .. 7; 8 .. 15: ^ 4
  const uint8_t *w0 = reinterpret_cast<const uint8_t *>(a.w) + ((int64_t)e * N + n0) * w_pitch;
  const int there = out_cols - n0 < kOutCols ? out_cols - n0 : kOutCols;
  for (int64_t r0 = 0; r0 < rows; r0 += kStreamRows) {
    const int left = (int)(rows - r0 < kStreamRows ? rows - r0 : kStreamRows);
    const uint8_t *x0 = static_cast<const uint8_t *>(a.x) + (first + r0) * x_pitch;
    const uint8_t *s0 = reinterpret_cast<const uint8_t *>(a.x_scales) + (first + r0) * (K / 128) * 4;
    const auto issue = [&](int c, int slot) {  // chunk c, or zeros past the last
      const uint32_t lds = lds0 + slot * kBytes;
      const int k0 = c * kChunk;
      const int k_left = c < chunks ? K - k0 : 0;
#pragma unroll
      for (int i = 0; i < kWLoads; ++i) {
        constexpr int kParts = kChunk / 64;           // of a row
        const int part = i % kParts, group = i / kParts;  // 8 rows
        const int p = piece ^ (group & 1) << 2;
        // SwiGLU: rows 0 .. 15 are the gate's, the others up's
        const int n = SWIGLU ? group % 2 * 8 : group * 8;
        const int have = there - n;
        const uint8_t *base = w0 + (int64_t)(n + (SWIGLU ? group / 2 * out_cols : 0)) * w_pitch +
                              (k0 + part * 64) * 2;
        const int bytes = have <= 0 || k_left <= 0
                              ? 0 : (have < 8 ? have : 8) * w_pitch - (k0 + part * 64) * 2;
        const bool in = part * 64 + p * 8 < k_left;
        load_to_lds<ONCE>(lds + i * 1024,
                          in ? (uint32_t)(at_row * w_pitch + p * 16) : kNowhere,
                          buffer_of(base, bytes < 0 ? 0 : bytes));
      }
#pragma unroll
      for (int i = 0; i < kXLoads; ++i) {
        const int p = piece ^ (i & 1) << 2, have = left - i * 8;
        const uint8_t *base = x0 + (int64_t)i * 8 * x_pitch + k0 * (FP8 ? 1 : 2);
        const int bytes = have <= 0 || k_left <= 0
                              ? 0 : (have < 8 ? have : 8) * x_pitch - k0 * (FP8 ? 1 : 2);
        const bool in = p * (FP8 ? 16 : 8) < k_left;
        load_to_lds(lds + kWBytes + i * 1024, in ? (uint32_t)(at_row * x_pitch + p * 16) : kNowhere,
                    buffer_of(base, bytes < 0 ? 0 : bytes));
      }
      if constexpr (FP8)
        load_word_to_lds(lds + kWBytes + kXBytes, (lane * (uint32_t)(K / 128) + c) * 4,
                         buffer_of(s0, k_left > 0 ? left * (K / 128) * 4 : 0));
    };
    f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(wave + i * kStreamWaves, i);
    int slot = 0;
    for (int c = wave; c < chunks; c += kStreamWaves) {
      issue(c + (kStages - 1) * kStreamWaves, slot == 0 ? kStages - 1 : slot - 1);
      wait_loads<(kStages - 1) * kLoads>();
      const uint8_t *here = stage[wave][slot];
      // lane l16: row l16 of 16, eight columns from 32 ks + 8 quad on
      const auto read = [&](int at, int ks) {
        return *reinterpret_cast<const bf16x8 *>(
            here + at + l16 * 128 + ((ks * 4 + quad) ^ (l16 >> 1)) * 16);
      };
      if constexpr (FP8) {
        f32x4 part[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
        float scale = *reinterpret_cast<const float *>(here + kWBytes + kXBytes + l16 * 4);
        const bool large = large_scale(scale);
        scale *= sums_power(large);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          // 16 codes are a piece
          const u32x2 raw = *reinterpret_cast<const u32x2 *>(
              here + kWBytes + l16 * 128 + ((ks * 2 + (quad >> 1)) ^ (l16 >> 1)) * 16 + (quad & 1) * 8);
          const bf16x8 x = codes_bf16(raw, codes_power(large));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // rows 8 g .. + 7 of the weights: part 0 at 2048 g, part 1 1024 on
            const bf16x8 w = *reinterpret_cast<const bf16x8 *>(
                here + j * 4096 + (l16 >> 3) * 2048 + (ks >> 1) * 1024 + (l16 & 7) * 128 +
                (((ks & 1) * 4 + quad) ^ (l16 >> 1)) * 16);
            part[j] = mul(w, x, part[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[j][v] = __builtin_fmaf(scale, part[j][v], acc[j][v]);
      } else {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const bf16x8 x = read(kWBytes, ks);
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[j] = mul(read(j * 2048, ks), x, acc[j]);
        }
      }
      lds_done();  // the slot is free
      slot = slot == kStages - 1 ? 0 : slot + 1;
    }
    // sums of the waves: [wave][row][column]
    stage_barrier<0>();
    float *sums = reinterpret_cast<float *>(&stage[0][0][0]);
    constexpr int kPitch = kStreamCols + 4;
    static_assert(kStreamWaves * kStreamRows * kPitch * 4 <= (int)sizeof(stage), "sums fit");
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<f32x4 *>(sums + (wave * kStreamRows + l16) * kPitch + j * 16 + quad * 4) = acc[j];
    __syncthreads();
    for (int o = tid; o < kStreamRows * kOutCols; o += kStreamWaves * 64) {
      const int m = o / kOutCols, n = o % kOutCols;
      float y = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < kStreamWaves; ++w) {
        const float *p = sums + (w * kStreamRows + m) * kPitch + n;
        y += p[0];
        if (SWIGLU) up += p[kOutCols];
      }
      if (SWIGLU) y = silu_of(y) * up;
      if (m < left && n < there)
        static_cast<uint16_t *>(a.out)[(first + r0 + m) * out_cols + n0 + n] = f32_to_bf16(y);
    }
    __syncthreads();
  }
}

// Calls f with the tiles' size: 128 x 128, two workgroups per compute unit,
// where tiles of 256 x 256 would leave half the chip idle (kSmallTiles).  Of the
// experts' rows only the buffer's are known.
//   tiles of 256       64         96        128        192        256
//   bf16, 8 experts, 2048 x 512 .. 2048, us of 128 and of 256:
//                   32, 47     24, 42                32, 47     47, 48
//   rows' gradient                       24, 44                 48, 51
//   weights' gradient, 2048 x 2048       44, 57     47, 45     48, 39
//     with FP8 rows  38, 63              62, 78     94, 85    122, 84
// FP8 rows' larger tile is of 128 x 256; 8 experts, 2048 x N, of 128 and of 128 x 256:
//   1024 rows       29, 39               50, 43
//   4096 rows, tiles   40 29, 39   80 41, 39   120 42, 40   160 57, 72   200 61, 73
constexpr int64_t kSmallTiles = 160;

template <typename F>
void with_tiles(int64_t tiles, bool once, F f) {
  if (tiles <= kSmallTiles)
    f(std::true_type{}, std::false_type{}, dim3(2 * kTileWorkgroups));
  else if (once)
    f(std::false_type{}, std::true_type{}, dim3(kTileWorkgroups));
  else
    f(std::false_type{}, std::false_type{}, dim3(kTileWorkgroups));
}

// The weights that a call reads are past the Infinity Cache, where the next call
// finds nothing of them again, and most experts have one row tile, so that one
// workgroup reads them.
constexpr int64_t kInfinityCache = int64_t{256} << 20;
// Non-temporal and not, us (32 experts, 7168 x 2 x 2048, but where it says):
//   tiles of 256 rows   4 rows each 280, 311   32 289, 314   128 400, 419
//     rows' gradient, 4096 x 7168   128 396, 399      2048 x 7168   16 139, 159
//     2048 x 7168, rows each   64 190, 190   128 220, 222   192 262, 265
//                              256 346, 321   512 535, 485   1024 964, 907
//     its rows' gradient       64 148, 167   128 224, 243   256 338, 343
//   FP8 rows, tiles of 128          4 272, 309    128 503, 471
//     2048 x 7168              32 194, 202   64 195, 198   96 253, 237   128 293, 249
//   4096 rows of few of 256 experts, 2048 x 2048: of 32 61, 70; of 8, whose weights
//     the cache would hold, 55, 54; FP8 rows 88, 87 and 80, 77
//   streamed: one token's 8 experts, FP8 rows 76, 83
//     64 rows of 2 experts, 4096 x 2048, in the cache and read four times 26, 24
bool read_once(const ProductArgs &a, int row_tile) {
  const int64_t hit = a.rows.capacity < a.rows.E ? a.rows.capacity : a.rows.E;
  return hit * a.N * a.K * 2 > kInfinityCache &&
         a.rows.capacity * 2 <= (int64_t)a.rows.E * row_tile;
}

int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

// Row tiles of a buffer's rows: an expert's last tile is half full.
int64_t row_tiles_of(const ProductArgs &a) {
  const int64_t hit = a.rows.capacity < a.rows.E ? a.rows.capacity : a.rows.E;
  const int64_t n = a.rows.capacity / kTile + (hit + 1) / 2;
  return n > hit ? n : hit;
}

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
  a.out_any = !aligned_to(out, 16);
  const auto launch = [&](auto f, auto s) {
    const int64_t columns = s.value ? N / 2 : N, tile_cols = s.value ? kTile / 2 : kTile;
    const int64_t hit = capacity < experts->num_experts ? capacity : experts->num_experts;
    // Streamed and tiled, us: 16 rows of 32 experts, 4096 x 2048 54, 73; 24 of 32
    // 79, 95; 64 of 16, 2048 x 2048 27, 32; 64 of 8, 4096 x 2048 33, 56; 64 of 2
    // 24, 46.  Past 64 rows, or where tiles fill the chip, rows by 16 read the
    // weights again and again.
    const bool few = capacity <= kStreamRows ||
                     (capacity <= 4 * kStreamRows &&
                      hit * ((columns + tile_cols - 1) / tile_cols) < kTileWorkgroups);
    if (few && (f.value || K % 8 == 0)) {
      constexpr int kCols = s.value ? kStreamCols / 2 : kStreamCols;
      const dim3 grid((unsigned)((columns + kCols - 1) / kCols), (unsigned)experts->num_experts);
      if (read_once(a, kStreamRows))
        hipLaunchKernelGGL((product_stream_kernel<f.value, s.value, true>), grid,
                           dim3(kStreamWaves * 64), 0, stream, a);
      else
        hipLaunchKernelGGL((product_stream_kernel<f.value, s.value, false>), grid,
                           dim3(kStreamWaves * 64), 0, stream, a);
    } else if (f.value || K % 8 == 0) {
      with_tiles(row_tiles_of(a) * tiles_of(N), read_once(a, f.value ? kTile / 2 : kTile),
                 [&](auto small, auto once, dim3 grid) {
                   hipLaunchKernelGGL((product_tile_kernel<kProduct, f.value, s.value, uint16_t,
                                                           small.value, once.value>),
                                      grid, dim3(kTileWaves * 64), 0, stream, a);
                 });
    } else
      hipLaunchKernelGGL((product_any_kernel<kProduct, false, s.value, uint16_t>),
                         dim3(kAnyGrid), dim3(256), 0, stream, a);
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
  if (a.K % 8 == 0 && a.N % 8 == 0 && aligned_to(grad_x, 16))
    with_tiles(row_tiles_of(a) * tiles_of(a.K), read_once(a, kTile),
               [&](auto small, auto once, dim3 grid) {
                 hipLaunchKernelGGL((product_tile_kernel<kRowsGrad, false, false, uint16_t,
                                                         small.value, once.value>),
                                    grid, dim3(kTileWaves * 64), 0, stream, a);
               });
  else
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
  const bool tiled = K % 8 == 0 && N % 8 == 0;
  const auto launch = [&](auto f, auto value) {
    if (tiled)
      with_tiles(a.rows.E * tiles_of(N) * tiles_of(K), false, [&](auto small, auto, dim3 grid) {
        hipLaunchKernelGGL(
            (product_tile_kernel<kWeightsGrad, f.value, false, decltype(value), small.value, false>),
            grid, dim3(kTileWaves * 64), 0, stream, a);
      });
    else
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
