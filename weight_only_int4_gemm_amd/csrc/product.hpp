// Products of rows with their own expert's weights (w4a16_moe_gemm,
// w8a8_moe_gemm) and of e4m3 matrices (w8a8_gemm: one expert that has every
// row).  Two kernels, each for three formats:
//
//   product_stream_kernel  few rows an expert: bound by the weights' way from
//       memory.  The waves of a workgroup take the K blocks of one column
//       tile in turn, weights and activations straight into registers; their
//       sums meet in LDS.
//   product_tile_kernel    many rows: bound by the matrix instructions.  The
//       waves divide an output tile; activations are staged in LDS by direct
//       loads, each row gathered from where its token is; weights go from
//       memory straight into the registers of the waves that use them, which
//       leaves LDS bandwidth to the activations.
//
// In both the weights are the matrix instruction's first operand, so a lane
// holds four neighbouring output columns of one row (row l % 16, columns
// 4 (l / 16) .. +3 of a 16 x 16 block) and stores them as 8 bytes.
//
// How many rows each expert has is known on the device only.  The grid covers
// the most tiles that `rows` sorted rows can make, and every workgroup finds
// its own: the lanes of a wave count the tiles of E / 64 experts each, one
// prefix sum over the wave places them.  Workgroups past the last tile leave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "coherent.hpp"
#include "format.hpp"
#include "internal.hpp"
#include "layout.hpp"
#include "tile_common.hpp"
#include "w4a16_moe.h"

namespace w4a16 {

// Formats of a product: how a 128-deep K block of 16 weight columns and of 16
// rows is loaded and multiplied.
enum : int { kProdF8 = 0, kProdI4F16 = 1, kProdI4Bf16 = 2 };

struct ProductArgs {
  const uint8_t* A;      // rows of row_bytes(K)
  const float* As;       // e4m3: [a_rows][K/128]
  const int32_t* order;  // null: row p of A
  const int32_t* starts; // null: one expert with rows 0 .. rows - 1
  const uint8_t* B;      // permuted weights, b_expert bytes an expert
  const void* S;         // scales, s_expert elements an expert
  uint16_t* C;
  int64_t b_expert, s_expert;
  int a_rows, k, E, rows, K, N;  // N: output columns
  int W;                         // weight columns
  int dtype;
  uint64_t gmagic;               // 4 bits: K block -> group
  int tiles_n, splits;
  unsigned* counters;
  float* partials;
};

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------

// Workgroups go to the eight dies in turn; tile t of `total` for workgroup i
// such that each die has a contiguous share, exact to one tile.  -1: none.
__device__ __forceinline__ int die_share(int i, int total) {
  const int q = total >> 3, r = total & 7, x = i & 7, j = i >> 3;
  if (j >= q + (x < r)) return -1;
  return x * q + (x < r ? x : r) + j;
}

struct RowTile {
  int e, row0, end;  // expert, first row, one past the expert's last
};

// Tiles of `tm` rows of all experts; lane-wise pieces of a wave's count.
struct RowTiles {
  int per, first, lane_tiles, incl, total;
};

__device__ __forceinline__ int start_of(const ProductArgs& p, int e) {
  const int s = p.starts[e];
  return s < 0 ? 0 : s > p.rows ? p.rows : s;
}

__device__ __forceinline__ RowTiles count_tiles(const ProductArgs& p, int tm) {
  RowTiles t;
  const int lane = threadIdx.x & 63;
  if (!p.starts) {
    t.per = 1;
    t.first = 0;
    t.lane_tiles = t.incl = t.total = (p.rows + tm - 1) / tm;
    return t;
  }
  t.per = (p.E + 63) >> 6;
  t.first = lane * t.per;
  int n = 0;
  int lo = start_of(p, t.first < p.E ? t.first : p.E);
  for (int i = 0; i < t.per; ++i) {
    const int e = t.first + i + 1;
    const int hi = start_of(p, e < p.E ? e : p.E);
    n += hi > lo ? (hi - lo + tm - 1) / tm : 0;
    lo = hi;
  }
  t.lane_tiles = n;
  int x = n;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  t.incl = x;
  t.total = __builtin_amdgcn_readlane(x, 63);
  return t;
}

// Row tile m < t.total.
__device__ __forceinline__ RowTile row_tile(const ProductArgs& p, const RowTiles& t, int tm,
                                            int m) {
  if (!p.starts) return RowTile{0, m * tm, p.rows};
  const uint64_t over = __ballot(t.incl > m);
  const int lane = __builtin_ctzll(over);
  int left = m - (__builtin_amdgcn_readlane(t.incl, lane) -
                  __builtin_amdgcn_readlane(t.lane_tiles, lane));
  int e = lane * t.per;
  for (;; ++e) {
    const int lo = start_of(p, e), hi = start_of(p, e + 1);
    const int n = hi > lo ? (hi - lo + tm - 1) / tm : 0;
    if (left < n || e + 1 >= p.E)
      return RowTile{__builtin_amdgcn_readfirstlane(e),
                     __builtin_amdgcn_readfirstlane(lo + left * tm),
                     __builtin_amdgcn_readfirstlane(hi)};
    left -= n;
  }
}

// The row of A that sorted row p takes.
__device__ __forceinline__ int source_row(const ProductArgs& a, int p) {
  unsigned r = (unsigned)p;
  if (a.order) {
    const int i = a.order[p];
    r = i < 0 ? 0u : (unsigned)i / (unsigned)a.k;
  }
  return r < (unsigned)a.a_rows ? (int)r : 0;
}

// ---------------------------------------------------------------------------
// formats
// ---------------------------------------------------------------------------

typedef int int8_vt __attribute__((ext_vector_type(8)));

template <int F>
struct Product {
  static constexpr bool kF8 = F == kProdF8;
  static constexpr bool kOffset = F == kProdI4Bf16;  // codes(): 136 too much
  static constexpr int kFmt = F == kProdI4Bf16 ? kFmtBf16 : kFmtF16;
  static constexpr int kRowBlock = kF8 ? 128 : 256;  // bytes of a row's K block
  static constexpr int kAPieces = kRowBlock / 64;    // 16-byte pieces of a lane
  static constexpr int kBPieces = kF8 ? 2 : 1;
  static constexpr int kBBlock = kBPieces * 1024;    // bytes of 16 columns x 128
};

// One 16x16x128 e4m3 matrix instruction on a lane's 32 bytes of either side.
__device__ __forceinline__ float4_t mma_f8(uint4 b0, uint4 b1, uint4 a0, uint4 a1, float4_t acc) {
  const int8_vt b = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w,
                     (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
  const int8_vt a = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w,
                     (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// Eight 4-bit codes as exact numbers of the type: FP16 q - 8; BF16, which has
// no packed subtraction, 128 + q (seven fraction bits) in 7 vector
// instructions, where (q - 8) s takes 29.  Sums of the latter start from
// minus_offset() times the row, one more matrix instruction a slice.
template <int F>
__device__ __forceinline__ half8_t codes(uint32_t word) {
  if constexpr (Product<F>::kOffset) {
    Half8 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w.u[i] = and_or(i ? word >> (4 * i) : word, 0x000F000Fu, 0x43004300u);
    return w.v;
  } else {
    return codes_minus_eight(word).v;
  }
}

__device__ __forceinline__ half8_t minus_offset() {  // BF16 -136
  Half8 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w.u[i] = 0xC308C308u;
  return w.v;
}

__device__ __forceinline__ float scale16(uint16_t bits, int bf16) {
  return bf16 ? __builtin_bit_cast(float, (uint32_t)bits << 16)
              : (float)__builtin_bit_cast(_Float16, bits);
}

__device__ __forceinline__ uint16_t round16(float x, bool bf16) {
  return bf16 ? __builtin_bit_cast(uint16_t, (__bf16)x)
              : __builtin_bit_cast(uint16_t, (_Float16)x);
}

// x / (1 + exp(-x)) * u with the hardware exponential and reciprocal.  The
// exponent x log2(e) is rounded (the constant and the product), so the result
// is off by up to (2 |x| + 8) 2^-24 of itself: 2^-17 at x = -60, where half a
// step of the output is 2^-11 (FP16) or 2^-8.  Below x = -87.3 the reciprocal,
// under 2^-126, may be 0, and y with it (|y| <= 2^-118 |u|).
__device__ __forceinline__ float silu_gate(float x, float u) {
  return x * __builtin_amdgcn_rcpf(1.f + __expf(-x)) * u;
}

// Four neighbouring columns of one row, rounded.
__device__ __forceinline__ uint2 round4(const ProductArgs& p, float4_t v) {
  ushort4 h;
  if (p.dtype == W4A16_DTYPE_BF16)
    h = ushort4{round16(v[0], true), round16(v[1], true), round16(v[2], true), round16(v[3], true)};
  else
    h = ushort4{round16(v[0], false), round16(v[1], false), round16(v[2], false),
                round16(v[3], false)};
  return __builtin_bit_cast(uint2, h);
}

__device__ __forceinline__ void store4(const ProductArgs& p, int64_t at, float4_t v) {
  *reinterpret_cast<uint2*>(p.C + at) = round4(p, v);
}

// x's odd rows of 16 lanes change places with y's even ones (D = 16), x's
// second half of the wave with y's first (D = 32).
template <int D>
__device__ __forceinline__ void swap_lanes(uint2& x, uint2& y) {
  if constexpr (D == 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(x.x, y.x, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(x.y, y.y, false, false);
    x = uint2{a[0], b[0]};
    y = uint2{a[1], b[1]};
  } else {
    const auto a = __builtin_amdgcn_permlane32_swap(x.x, y.x, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(x.y, y.y, false, false);
    x = uint2{a[0], b[0]};
    y = uint2{a[1], b[1]};
  }
}

// OB blocks of 16 columns from column block ob0, a lane's x[ob] four columns of
// its row in each.  The four lanes of a row exchange theirs, so that each
// stores 16 bytes at a time (64 experts of 1408 x 2048, 768 rows each, and their
// sum: 292 -> 269 us in 256 x 256 tiles).
template <int OB>
__device__ __forceinline__ void store_blocks(const ProductArgs& p, int r, int end, int ob0,
                                             int quarter, uint2 (&x)[OB]) {
  int ob = 0, column = 4 * quarter;
  if constexpr (OB == 2) {
    swap_lanes<16>(x[0], x[1]);  // quarters 2 (q / 2), + 1 of block q % 2
    ob = quarter & 1;
    column = 8 * (quarter >> 1);
  } else if constexpr (OB == 4) {
    swap_lanes<32>(x[0], x[2]);
    swap_lanes<32>(x[1], x[3]);
    swap_lanes<16>(x[0], x[1]);
    swap_lanes<16>(x[2], x[3]);  // all of block q
    ob = quarter;
    column = 0;
  }
  static_assert(OB == 1 || OB == 2 || OB == 4, "blocks");
  if (r >= end || 16 * (ob0 + ob) >= p.N) return;
  uint16_t* const to = p.C + (int64_t)r * p.N + 16 * (ob0 + ob) + column;
  if constexpr (OB == 1)
    *reinterpret_cast<uint2*>(to) = x[0];
  else
#pragma unroll
    for (int i = 0; i < OB; i += 2)
      reinterpret_cast<uint4*>(to)[i / 2] = uint4{x[i].x, x[i].y, x[i + 1].x, x[i + 1].y};
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

// 16 MB rows by NB blocks of 16 weight columns (with GATE, the first half of
// them gate columns and the second their up columns); WAVES waves take the K
// blocks in turn, DEPTH of them in flight.
template <int F, int MB, int NB, int WAVES, int DEPTH, bool GATE>
__global__ __launch_bounds__(64 * WAVES) void product_stream_kernel(ProductArgs p) {
  typedef Product<F> P;
  constexpr int TM = 16 * MB;
  constexpr int OB = GATE ? NB / 2 : NB;  // output column blocks
  __shared__ float4_t red[WAVES][MB * NB][64];
  const int lane = threadIdx.x & 63, l16 = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const RowTiles tiles = count_tiles(p, TM);
  const int m = blockIdx.x / p.tiles_n, tile_n = blockIdx.x - m * p.tiles_n;
  if (m >= tiles.total) return;
  const RowTile rt = row_tile(p, tiles, TM, m);

  const int KB = p.K / kBlockK;
  const uint8_t* arow[MB];
  const float* asrow[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int r = rt.row0 + 16 * mb + l16;
    const int src = source_row(p, r < rt.end ? r : rt.end - 1);
    arow[mb] = p.A + (int64_t)src * KB * P::kRowBlock + quarter * 16;
    if constexpr (P::kF8) asrow[mb] = p.As + (int64_t)src * KB;
  }
  int block[NB];  // 16-column block of the weights
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int ob = tile_n * OB + nb % OB;
    const int last = p.N / 16 - 1;
    block[nb] = (ob < last ? ob : last) + (nb >= OB ? p.N / 16 : 0);
  }
  const uint8_t* bsrc[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
    bsrc[nb] = p.B + rt.e * p.b_expert + (int64_t)block[nb] * KB * P::kBBlock + lane * 16;

  struct Step {
    uint4 b[NB][P::kBPieces];
    uint4 a[MB][P::kAPieces];
    float bs[P::kF8 ? NB : 1];
    float as[P::kF8 ? MB : 1];
    uint2 s[P::kF8 ? 1 : NB];  // the lane's four columns' scales
  };
  auto load = [&](Step& t, int kb) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < P::kBPieces; ++i)
        t.b[nb][i] = *reinterpret_cast<const uint4*>(bsrc[nb] + (int64_t)kb * P::kBBlock + i * 1024);
    if constexpr (P::kF8) {
      const float* S = static_cast<const float*>(p.S) + rt.e * p.s_expert;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) t.bs[nb] = S[(block[nb] >> 3) * KB + kb];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) t.as[mb] = asrow[mb][kb];
    } else {
      const int group = (int)(((uint64_t)(uint32_t)kb * p.gmagic) >> 32);
      const uint16_t* S = static_cast<const uint16_t*>(p.S) + rt.e * p.s_expert +
                          (int64_t)group * p.W;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        t.s[nb] = *reinterpret_cast<const uint2*>(S + 16 * block[nb] + 4 * quarter);
      }
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int i = 0; i < P::kAPieces; ++i)
        t.a[mb][i] = *reinterpret_cast<const uint4*>(arow[mb] + kb * P::kRowBlock + i * 64);
  };

  float4_t acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = float4_t{0.f, 0.f, 0.f, 0.f};
  const float4_t zero = {0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Step& t) {
    if constexpr (P::kF8) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const float4_t d = mma_f8(t.b[nb][0], t.b[nb][1], t.a[mb][0], t.a[mb][1], zero);
          const float f = t.as[mb] * t.bs[nb];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[mb][nb][i] = __builtin_fmaf(d[i], f, acc[mb][nb][i]);
        }
    } else {
      // The sums of the exact integers q - 8 take the scale (BF16: one token
      // through two experts of 4096 x 22016, weights scaled 32.0 us, sums 24.5).
      float4_t base[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        base[mb] = zero;
        if constexpr (P::kOffset)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            base[mb] = mma16<P::kFmt>(minus_offset(), __builtin_bit_cast(half8_t, t.a[mb][j]),
                                      base[mb]);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float4_t d[MB];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const half8_t w = codes<F>(word_of(t.b[nb][0], j));
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            d[mb] = mma16<P::kFmt>(w, __builtin_bit_cast(half8_t, t.a[mb][j]),
                                   j == 0 ? base[mb] : d[mb]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t pair = i < 2 ? t.s[nb].x : t.s[nb].y;
          const float s = scale16((uint16_t)(pair >> (16 * (i & 1))), P::kOffset);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) acc[mb][nb][i] = __builtin_fmaf(d[mb][i], s, acc[mb][nb][i]);
        }
      }
    }
  };

  Step ring[DEPTH];
  const int n = (KB - wave + WAVES - 1) / WAVES;  // this wave's K blocks
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i)
    if (i < n) load(ring[i], wave + i * WAVES);
  for (int t = 0; t < n; t += DEPTH) {
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) {
      if (t + u >= n) break;
      if (t + u + DEPTH - 1 < n)
        load(ring[(u + DEPTH - 1) % DEPTH], wave + (t + u + DEPTH - 1) * WAVES);
      multiply(ring[u]);
    }
  }

  // the waves' sums, added in wave order
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) red[wave][mb * NB + nb][lane] = acc[mb][nb];
  __syncthreads();
  for (int i = wave; i < MB * OB; i += WAVES) {
    const int mb = i / OB, ob = i - mb * OB;
    float4_t x = red[0][mb * NB + ob][lane], u = zero;
    if constexpr (GATE) u = red[0][mb * NB + OB + ob][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      x += red[w][mb * NB + ob][lane];
      if constexpr (GATE) u += red[w][mb * NB + OB + ob][lane];
    }
    if constexpr (GATE)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = silu_gate(x[j], u[j]);
    const int r = rt.row0 + 16 * mb + l16, c = 16 * (tile_n * OB + ob) + 4 * quarter;
    if (r < rt.end && c < p.N) store4(p, (int64_t)r * p.N + c, x);
  }
}

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

// Row tiles that one run of neighbouring tiles takes together, so that the
// tiles in flight on a die share rows and columns.
constexpr int kTileRun = 4;

// 16 MB rows; WAVES waves, each NB blocks of 16 weight columns.  With four
// waves two workgroups or more share a compute unit, so that one's first loads
// and stores run beside the other's products: 128 x 256 e4m3 tiles so against
// 256 x 256 in eight waves 816 : 826 us for 8192 x 28672 at M = 4096, 239 : 284
// for 11008 x 12288 at 2048, 245 : 270 for 64 experts of 1408 x 2048, 768 rows
// each (and their sum).
template <int F, int MB, int NB, int WAVES, bool GATE>
__global__ __launch_bounds__(64 * WAVES, 2) void product_tile_kernel(ProductArgs p) {
  typedef Product<F> P;
  constexpr int TM = 16 * MB;
  constexpr int NS = 4;  // stages of activations
  constexpr int OB = GATE ? NB / 2 : NB;        // output column blocks of a wave
  constexpr int SUB = P::kRowBlock / 128;       // 128-byte slices of a row's K block
  constexpr int ALOADS = SUB * ((TM / 8 + WAVES - 1) / WAVES);  // 1 KiB loads of a wave
  // piece c of row r of a slice at slot c ^ (r & 7): a fragment read's lanes
  // spread over all banks
  struct Stage {
    uint4 a[SUB * TM * 8];
  };
  // one LDS object per stage: the compiler sees that a load into one stage
  // does not touch the others
  __shared__ Stage st0;
  __shared__ Stage st1;
  __shared__ Stage st2;
  __shared__ Stage st3;
  // e4m3: the rows' scales of four K blocks, and of the next four; two objects
  // for the same reason (as one, every fourth block began with a wait for all
  // loads in flight: 4096 x 4096 at M = 256 16.1 -> 13.9 us)
  struct RowScales {
    float4_t of[P::kF8 ? TM : 1];
  };
  __shared__ RowScales rs0;
  __shared__ RowScales rs1;

  const int lane = threadIdx.x & 63, l16 = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const RowTiles tiles = count_tiles(p, TM);
  const int split = blockIdx.y;
  const int t = die_share(blockIdx.x, tiles.total * p.tiles_n);
  if (t < 0) return;
  const int run = t / (kTileRun * p.tiles_n), in_run = t - run * (kTileRun * p.tiles_n);
  const int left = tiles.total - run * kTileRun, height = left < kTileRun ? left : kTileRun;
  const int tile_n = in_run / height;
  const RowTile rt = row_tile(p, tiles, TM, run * kTileRun + in_run - tile_n * height);

  const int KB = p.K / kBlockK;
  const int kb0 = (int)((int64_t)KB * split / p.splits);
  const int kb1 = (int)((int64_t)KB * (split + 1) / p.splits);

  // Activation loads: eight rows of a slice each.
  constexpr int RLOADS = (TM / 8 + WAVES - 1) / WAVES;  // of one slice
  const uint8_t* asrc[RLOADS];
#pragma unroll
  for (int i = 0; i < RLOADS; ++i) {
    const int r = (wave + WAVES * i) % (TM / 8) * 8 + (lane >> 3);
    const int q = rt.row0 + r;
    const int src = source_row(p, q < rt.end ? q : rt.end - 1);
    asrc[i] = p.A + (int64_t)src * KB * P::kRowBlock + ((lane & 7) ^ (r & 7)) * 16;
  }
  // Row scales come four K blocks at a time (a lane reads 16 bytes of its
  // row): loaded block by block, each 4-byte access of a scattered row takes
  // the cache path as long as 64 contiguous bytes (8192 x 28672 at M = 4096:
  // 998 -> 981 us, and 934 with four stages).  TM / WAVES lanes of a wave load
  // one row each; the last group, where the row may end, goes through registers.
  constexpr int SROWS = TM / WAVES;
  const float* scale_src = nullptr;
  if constexpr (P::kF8) {
    const int q = rt.row0 + wave * SROWS + (lane < SROWS ? lane : SROWS - 1);
    scale_src = p.As + (int64_t)source_row(p, q < rt.end ? q : rt.end - 1) * KB;
  }
  auto load_scales = [&](RowScales& to, int kb) {
    if constexpr (P::kF8) {
      if (kb + 4 <= KB) {
        if (lane < SROWS)
          __builtin_amdgcn_global_load_lds((global_ptr_t)(scale_src + kb),
                                           (lds_ptr_t)&to.of[wave * SROWS], 16, 0, 0);
      } else if (kb < KB) {
        float4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = scale_src[kb + i < KB ? kb + i : KB - 1];
        if (lane < SROWS) to.of[wave * SROWS + lane] = v;
      }
    }
  };
  // Load i < ALOADS of a stage.
  auto load_rows = [&](Stage& sg, int kb, int i) {
    const uint8_t* src = asrc[i / SUB] + kb * P::kRowBlock + (i % SUB) * 128;
    uint4* const to = &sg.a[(i % SUB) * TM * 8 + 64 * ((wave + WAVES * (i / SUB)) % (TM / 8))];
    __builtin_amdgcn_global_load_lds((global_ptr_t)src, (lds_ptr_t)to, 16, 0, 0);
  };

  // Weights of a wave: blocks past the last re-read it (never stored).  Their
  // addresses are the wave's own but for the lane's 16 bytes, so buffer loads
  // keep them in scalar registers; one resource for the gate columns, one for
  // the up columns, both from the wave's first block.
  const int ob0 = (tile_n * WAVES + wave) * OB;  // first output column block
  const int blocks = p.N / 16, first = ob0 < blocks ? ob0 : blocks - 1;
  constexpr int HALVES = GATE ? 2 : 1;
  const uint32_t lane16 = lane * 16;
  __amdgpu_buffer_rsrc_t bsrc[HALVES];
  int boff[OB];
#pragma unroll
  for (int i = 0; i < HALVES; ++i)
    bsrc[i] = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(p.B) + rt.e * p.b_expert +
            (int64_t)(first + i * blocks) * KB * P::kBBlock,
        (short)0, 0x7fffffff, 0x00020000);
#pragma unroll
  for (int i = 0; i < OB; ++i)
    boff[i] = ((first + i < blocks ? first + i : blocks - 1) - first) * KB * P::kBBlock;
  // e4m3: a wave's columns lie in one 128-column block of scales (with GATE,
  // one of each half).  4 bits: the scales of the lane's four output columns.
  constexpr int SCALES = P::kF8 ? HALVES : NB;
  // Buffer loads: the waits below count them, so none may become a scalar one.
  const __amdgpu_buffer_rsrc_t ssrc = __builtin_amdgcn_make_buffer_rsrc(
      static_cast<char*>(const_cast<void*>(p.S)) + rt.e * p.s_expert * (P::kF8 ? 4 : 2), (short)0,
      0x7fffffff, 0x00020000);
  struct Weights {
    uint4 b[NB][P::kBPieces];
    float s[P::kF8 ? SCALES : 1];
    uint2 s4[P::kF8 ? 1 : NB];  // four columns' scales
  };
  // Load i < WLOADS of a K block's weights: a column block's, or a scale.
  constexpr int WLOADS = NB + SCALES;
  auto load_weights = [&](Weights& w, int kb, int i) {
    if (i < NB) {
#pragma unroll
      for (int piece = 0; piece < P::kBPieces; ++piece)
        w.b[i][piece] = __builtin_bit_cast(
            uint4, __builtin_amdgcn_raw_buffer_load_b128(bsrc[i / OB], lane16 + piece * 1024,
                                                         boff[i % OB] + kb * P::kBBlock, 0));
    } else if constexpr (P::kF8) {
      const int h = i - NB;
      w.s[h] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(
                     ssrc, 0, (((first + h * blocks) >> 3) * KB + kb) * 4, 0));
    } else {
      const int nb = i - NB;
      const int group = (int)(((uint64_t)(uint32_t)kb * p.gmagic) >> 32);
      const int ob = first + nb % OB < blocks ? first + nb % OB : blocks - 1;
      const int at = (group * p.W + 16 * (ob + (nb >= OB ? blocks : 0))) * 2;
      w.s4[nb] = __builtin_bit_cast(
          uint2, __builtin_amdgcn_raw_buffer_load_b64(ssrc, quarter * 8, at, 0));
    }
  };

  float4_t acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = float4_t{0.f, 0.f, 0.f, 0.f};
  const float4_t zero = {0.f, 0.f, 0.f, 0.f};

  constexpr int SETS = NB <= 2 ? NS : 2;
  constexpr int LOADS = WLOADS + ALOADS;
  constexpr int WINSTRS = NB * P::kBPieces + SCALES;  // load instructions of the weights
  constexpr int NEWER = SETS == NS ? (NS - 2) * (WINSTRS + ALOADS) : ALOADS;
  // Rows of a wave are 16 apart, so a lane's swizzle is one number.
  const int l7 = l16 & 7, arow0 = l16 * 8;
  const int swz0 = arow0 + (quarter ^ l7), swz1 = arow0 + ((quarter + 4) ^ l7);
  // u: the K block's place in its group of four; sc: the group's row scales;
  // issue(i): the i-th of the loads for later K blocks.  They are spread over
  // the matrix instructions: issued together, the waves' loads queue for the
  // address unit before any of them multiplies (8192 x 28672 at M = 4096: 999
  // -> 873 us).
  auto multiply = [&](const Stage& sg, Weights& w, int u, const float4_t* sc, auto&& issue) {
    if constexpr (P::kF8) {
      // Every K block has its own scales, so each matrix instruction starts
      // from zero and its sums are added with one multiply-add each.  These
      // follow LAG instructions later, when the sums are there; row block
      // mb + 1 is read while mb is multiplied.
      constexpr int LAG = 2, RING = 4;
      constexpr int PRE = NB >= 4 ? 1 : NB == 2 ? 2 : 3;  // row blocks read ahead
      constexpr int AS = NB == 1 ? 8 : 4;                 // their scales live LAG longer
      uint4 a[PRE + 1][2];
      float as[AS], f[2][SCALES];
      float4_t d[RING];
      auto read = [&](int mb) {
        a[mb % (PRE + 1)][0] = sg.a[swz0 + mb * 128];
        a[mb % (PRE + 1)][1] = sg.a[swz1 + mb * 128];
        as[mb % AS] = reinterpret_cast<const float*>(sc + l16 + mb * 16)[u];
      };
      auto add = [&](int i) {
        const int mb = i / NB, nb = i % NB;
        if (nb == 0)
#pragma unroll
          for (int s = 0; s < SCALES; ++s)
            f[mb & 1][s] = as[mb % AS] * w.s[s];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[mb][nb][e] = __builtin_fmaf(d[i % RING][e], f[mb & 1][nb / OB], acc[mb][nb][e]);
        asm volatile("" : "+v"(acc[mb][nb]));  // here, not where the loop ends
      };
#pragma unroll
      for (int mb = 0; mb < PRE && mb < MB; ++mb) read(mb);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int i = mb * NB + nb;
          d[i % RING] = mma_f8(w.b[nb][0], w.b[nb][1], a[mb % (PRE + 1)][0], a[mb % (PRE + 1)][1],
                               zero);
          __builtin_amdgcn_sched_barrier(0);
          if (i >= LAG) add(i - LAG);
          if (nb == 0 && mb + PRE < MB) read(mb + PRE);
          constexpr int EVERY = MB * NB / LOADS > 0 ? MB * NB / LOADS : 1;
          if (i % EVERY == EVERY - 1 && i / EVERY < LOADS) issue(i / EVERY);
          __builtin_amdgcn_sched_barrier(0);  // in this order
        }
      }
#pragma unroll
      for (int i = MB * NB < LAG ? 0 : MB * NB - LAG; i < MB * NB; ++i) add(i);
#pragma unroll
      for (int i = MB * NB; i < LOADS; ++i) issue(i);
    } else {
      // The exact integers are multiplied and the scales go onto the FP32 sums
      // of 128, so no weight is rounded.  All of a K block's words are unpacked
      // while its first row block is multiplied; the sums of one row block are
      // scaled and added while the next is.  Against weights scaled and rounded
      // first, 8 experts of 4096 x 22016, FP16 and BF16, in us: 16 rows each
      // 89.5 : 90.9 and 92.8 : 130; 32 rows 115 : 117 and 120 : 155; 256 rows
      // 389 : 410 and 419 : 429; 1024 rows 1400 : 1245 and 1490 : 1500, with
      // a tenth of the error (FP16).
      // fragments are read AHEAD slices before their use, within 256 registers
      constexpr int AHEAD = P::kOffset && NB == 4 ? 3 : 4;
      half8_t wt[4][NB];
      half8_t a[AHEAD + 1];
      float4_t d[NB], base = zero;
      auto read = [&](int i) {  // slice i % 4 of row block i / 4
        const int j = i % 4, mb = i / 4;
        a[i % (AHEAD + 1)] = __builtin_bit_cast(
            half8_t, sg.a[(j >> 1) * TM * 8 + ((j & 1) ? swz1 : swz0) + mb * 128]);
      };
      auto unpack = [&](int j) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) wt[j][nb] = codes<F>(word_of(w.b[nb][0], j));
      };
      auto add = [&](int mb, int nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t pair = e < 2 ? w.s4[nb].x : w.s4[nb].y;
          acc[mb][nb][e] = __builtin_fmaf(P::kOffset ? d[nb][e] + base[e] : d[nb][e],
                                          scale16((uint16_t)(pair >> (16 * (e & 1))), P::kOffset),
                                          acc[mb][nb][e]);
        }
        asm volatile("" : "+v"(acc[mb][nb]));  // here, not where the loop ends
      };
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) read(i);
      unpack(0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4 * MB; ++i) {
        const int j = i % 4;
        if (i + AHEAD < 4 * MB) read(i + AHEAD);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (j == 0 && i > 0) add(i / 4 - 1, nb);
          d[nb] = mma16<P::kFmt>(wt[j][nb], a[i % (AHEAD + 1)], j == 0 ? zero : d[nb]);
        }
        if constexpr (P::kOffset)
          base = mma16<P::kFmt>(minus_offset(), a[i % (AHEAD + 1)], j == 0 ? zero : base);
        if (i < 3) unpack(i + 1);
        constexpr int EVERY = 4 * MB / LOADS > 0 ? 4 * MB / LOADS : 1;
        if (i % EVERY == EVERY - 1 && i / EVERY < LOADS) issue(i / EVERY);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) add(MB - 1, nb);
#pragma unroll
      for (int i = 4 * MB; i < LOADS; ++i) issue(i);
    }
  };

  // While K block kb is multiplied, the stage of kb + NS - 1 is loaded into
  // LDS and the weights of kb + SETS - 1 into registers, weights first.  With
  // as many sets as stages, what block kb waits for is older than the loads of
  // the NS - 2 blocks before it; with fewer, than the newest stage's.
  auto stage = [&](int i) -> Stage& {
    return i == 0 ? st0 : i == 1 ? st1 : i == 2 ? st2 : st3;
  };
  constexpr int UNROLL = P::kF8 ? 8 : NS;
  Weights weights[SETS];
  auto upto = [&](int kb) { return kb < kb1 ? kb : kb1 - 1; };
  auto load_stage = [&](Stage& sg, int kb) {
#pragma unroll
    for (int i = 0; i < ALOADS; ++i) load_rows(sg, kb, i);
  };
  load_scales(rs0, kb0);
  auto load_set = [&](int i) {
#pragma unroll
    for (int n = 0; n < WLOADS; ++n) load_weights(weights[i], upto(kb0 + i), n);
    keep_load_order();
  };
  // in the order of the steps that would have issued them
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) {
    const int set = i - (NS - 1) + (SETS - 1);
    if (set >= 0) load_set(set);
    load_stage(stage(i), upto(kb0 + i));
    keep_load_order();
  }
  auto step = [&](int u, int kb) {
    stage_barrier<NEWER>();
    if (P::kF8 && u % 4 == 0) load_scales(u == 0 ? rs1 : rs0, kb + 4);
    const int kb_w = upto(kb + SETS - 1), kb_a = upto(kb + NS - 1);
    multiply(stage(u % NS), weights[u % SETS], u % 4, (u < 4 ? rs0 : rs1).of, [&](int i) {
      if (i >= WLOADS)
        load_rows(stage((u + NS - 1) % NS), kb_a, i - WLOADS);
      else
        load_weights(weights[(u + SETS - 1) % SETS], kb_w, i);
      keep_load_order();
    });
  };
  int kb = kb0;
  for (; kb + UNROLL <= kb1; kb += UNROLL) {
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) step(u, kb + u);
  }
#pragma unroll
  for (int u = 0; u < UNROLL - 1; ++u)
    if (kb + u < kb1) step(u, kb + u);
  // no direct load may still be landing in LDS when the workgroup ends
  __builtin_amdgcn_s_waitcnt(0);

  if (P::kF8 && p.splits > 1) {  // 4-bit products never split
    // As in the other kernels' split K: partials published, the arrival
    // counted, the last workgroup of the tile adds them in split order.
    constexpr int TE = WAVES * MB * NB * 256;
    const float* base = p.partials + (int64_t)t * p.splits * TE;
    const int frag0 = wave * MB * NB * 64 + lane;
    {
      const __amdgpu_buffer_rsrc_t mine = coherent_rsrc(base + (int64_t)split * TE);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          store_coherent(mine, frag0 + (mb * NB + nb) * 64, acc[mb][nb]);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    int* const flag = reinterpret_cast<int*>(&st0);
    if (threadIdx.x == 0) {
      const unsigned prev =
          __hip_atomic_fetch_add(p.counters + t, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *flag = prev == (unsigned)(p.splits - 1);
    }
    __syncthreads();
    if (!*flag) return;
    // Several partials are loaded before the first of them is added: one
    // by one each costs a trip to memory.
    constexpr int AT_ONCE = MB * NB <= 4 ? 4 : MB * NB <= 8 ? 2 : 1;
    for (int s0 = 0; s0 < p.splits; s0 += AT_ONCE) {
      float4_t x[AT_ONCE][MB][NB];
#pragma unroll
      for (int s = 0; s < AT_ONCE; ++s) {
        const int from = s0 + s < p.splits ? s0 + s : p.splits - 1;
        const __amdgpu_buffer_rsrc_t ps = coherent_rsrc(base + (int64_t)from * TE);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            x[s][mb][nb] = load_coherent(ps, frag0 + (mb * NB + nb) * 64);
      }
#pragma unroll
      for (int s = 0; s < AT_ONCE; ++s) {
        if (s0 + s >= p.splits) break;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            acc[mb][nb] = s0 + s == 0 ? x[s][mb][nb] : acc[mb][nb] + x[s][mb][nb];
      }
    }
    if (threadIdx.x == 0)
      __hip_atomic_store(p.counters + t, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int r = rt.row0 + mb * 16 + l16;
    uint2 out[OB];
#pragma unroll
    for (int ob = 0; ob < OB; ++ob) {
      float4_t x = acc[mb][ob];
      if constexpr (GATE)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = silu_gate(x[j], acc[mb][OB + ob][j]);
      out[ob] = round4(p, x);
    }
    store_blocks<OB>(p, r, rt.end, ob0, quarter, out);
  }
}

}  // namespace w4a16
