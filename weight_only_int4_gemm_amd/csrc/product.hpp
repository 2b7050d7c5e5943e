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
    if (left < n || e + 1 >= p.E) return RowTile{e, lo + left * tm, hi};
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

__device__ __forceinline__ float scale16(uint16_t bits, int bf16) {
  return bf16 ? __builtin_bit_cast(float, (uint32_t)bits << 16)
              : (float)__builtin_bit_cast(_Float16, bits);
}

__device__ __forceinline__ uint16_t round16(float x, bool bf16) {
  return bf16 ? __builtin_bit_cast(uint16_t, (__bf16)x)
              : __builtin_bit_cast(uint16_t, (_Float16)x);
}

// x / (1 + exp(-x)) * u with the hardware exponential and reciprocal (a few
// FP32 ulps); exp overflows to infinity for x below -88, whose reciprocal
// gives the signed zero.
__device__ __forceinline__ float silu_gate(float x, float u) {
  return x * __builtin_amdgcn_rcpf(1.f + __expf(-x)) * u;
}

// Four neighbouring columns of one row.
__device__ __forceinline__ void store4(const ProductArgs& p, int64_t at, float4_t v) {
  ushort4 h;
  if (p.dtype == W4A16_DTYPE_BF16)
    h = ushort4{round16(v[0], true), round16(v[1], true), round16(v[2], true), round16(v[3], true)};
  else
    h = ushort4{round16(v[0], false), round16(v[1], false), round16(v[2], false),
                round16(v[3], false)};
  *reinterpret_cast<ushort4*>(p.C + at) = h;
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
    uint2 s[P::kF8 ? 1 : NB];  // four columns' scales, or the lane's column's
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
        if constexpr (F == kProdI4F16)
          t.s[nb] = *reinterpret_cast<const uint2*>(S + 16 * block[nb] + 4 * quarter);
        else
          t.s[nb].x = S[16 * block[nb] + l16];
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
    } else if constexpr (F == kProdI4F16) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float4_t d[MB];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const half8_t w = codes_minus_eight(word_of(t.b[nb][0], j)).v;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            d[mb] = mma16<P::kFmt>(w, __builtin_bit_cast(half8_t, t.a[mb][j]),
                                   j == 0 ? zero : d[mb]);
        }
        typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
        const half4_t s = __builtin_bit_cast(half4_t, t.s[nb]);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[mb][nb][i] = __builtin_fmaf(d[mb][i], (float)s[i], acc[mb][nb][i]);
      }
    } else {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const ColParams c = make_col<P::kFmt>(
            __builtin_bit_cast(half2_t, t.s[nb].x | (t.s[nb].x << 16)), 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const half8_t w = unpack_col<P::kFmt>(word_of(t.b[nb][0], j), c);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            acc[mb][nb] = mma16<P::kFmt>(w, __builtin_bit_cast(half8_t, t.a[mb][j]), acc[mb][nb]);
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

// WM x WN waves, each 16 MB rows by NB blocks of 16 weight columns; NS stages.
template <int F, int MB, int NB, int WM, int WN, int NS, bool GATE>
__global__ __launch_bounds__(64 * WM * WN) void product_tile_kernel(ProductArgs p) {
  typedef Product<F> P;
  constexpr int WAVES = WM * WN;
  constexpr int TM = 16 * MB * WM;
  constexpr int OB = GATE ? NB / 2 : NB;        // output column blocks of a wave
  constexpr int SUB = P::kRowBlock / 128;       // 128-byte slices of a row's K block
  constexpr int CHUNKS = SUB * TM / 8;          // wave-loads (1 KiB) of activations
  constexpr int ALOADS = (CHUNKS + WAVES - 1) / WAVES;
  constexpr int SROWS = P::kF8 ? (TM < 64 ? 64 : TM) : 64;
  constexpr int SLOADS = P::kF8 ? 1 : 0;        // every wave issues one
  constexpr int LOADS = ALOADS + SLOADS;
  static_assert(NS == 2 || NS == 4, "two or four stages");
  static_assert(SROWS / 64 <= WAVES, "one scale load a wave");
  // piece c of row r of a slice at slot c ^ (r & 7): a fragment read's lanes
  // spread over all banks
  struct Stage {
    uint4 a[SUB * TM * 8];
    float as[SROWS];
  };
  // one LDS object per stage: the compiler sees that a load into one stage
  // does not touch the others
  __shared__ Stage st0;
  __shared__ Stage st1;
  __shared__ typename std::conditional<(NS > 2), Stage, char>::type st2;
  __shared__ typename std::conditional<(NS > 2), Stage, char>::type st3;

  const int lane = threadIdx.x & 63, l16 = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

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

  // Activation loads: chunk (wave + WAVES i) of a stage, 8 rows of a slice.
  const uint8_t* asrc[ALOADS];
#pragma unroll
  for (int i = 0; i < ALOADS; ++i) {
    const int chunk = (wave + WAVES * i) % CHUNKS;
    const int slice = chunk / (TM / 8), r = chunk % (TM / 8) * 8 + (lane >> 3);
    const int q = rt.row0 + r;
    const int src = source_row(p, q < rt.end ? q : rt.end - 1);
    asrc[i] = p.A + (int64_t)src * KB * P::kRowBlock + slice * 128 + ((lane & 7) ^ (r & 7)) * 16;
  }
  const float* scale_src = nullptr;
  if constexpr (P::kF8) {
    const int r = wave % (SROWS / 64) * 64 + lane;
    const int q = rt.row0 + (r < TM ? r : TM - 1);
    scale_src = p.As + (int64_t)source_row(p, q < rt.end ? q : rt.end - 1) * KB;
  }
  auto load_stage = [&](Stage& sg, int kb) {
#pragma unroll
    for (int i = 0; i < ALOADS; ++i) {
      const int chunk = (wave + WAVES * i) % CHUNKS;
      __builtin_amdgcn_global_load_lds((global_ptr_t)(asrc[i] + kb * P::kRowBlock),
                                       (lds_ptr_t)&sg.a[64 * chunk], 16, 0, 0);
    }
    if constexpr (P::kF8)
      __builtin_amdgcn_global_load_lds((global_ptr_t)(scale_src + kb),
                                       (lds_ptr_t)&sg.as[64 * (wave % (SROWS / 64))], 4, 0, 0);
  };

  // Weights of a wave: blocks past the last re-read it (never stored).
  const int ob0 = (tile_n * WN + wn) * OB;  // first output column block
  int block[NB];
  const uint8_t* bsrc[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int ob = ob0 + nb % OB, last = p.N / 16 - 1;
    block[nb] = (ob < last ? ob : last) + (nb >= OB ? p.N / 16 : 0);
    bsrc[nb] = p.B + rt.e * p.b_expert + (int64_t)block[nb] * KB * P::kBBlock + lane * 16;
  }
  constexpr int SCALES = P::kF8 ? (GATE ? 2 : 1) : NB;
  struct Weights {
    uint4 b[NB][P::kBPieces];
    float bs[SCALES];
    uint16_t s[SCALES];
  };
  auto load_weights = [&](Weights& w, int kb) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < P::kBPieces; ++i)
        w.b[nb][i] = *reinterpret_cast<const uint4*>(bsrc[nb] + (int64_t)kb * P::kBBlock + i * 1024);
    if constexpr (P::kF8) {
      // A wave's columns lie in one 128-column block of scales (with GATE,
      // one of each half).
      const float* S = static_cast<const float*>(p.S) + rt.e * p.s_expert;
#pragma unroll
      for (int i = 0; i < SCALES; ++i) w.bs[i] = S[(block[i * OB] >> 3) * KB + kb];
    } else {
      const int group = (int)(((uint64_t)(uint32_t)kb * p.gmagic) >> 32);
      const uint16_t* S = static_cast<const uint16_t*>(p.S) + rt.e * p.s_expert +
                          (int64_t)group * p.W;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) w.s[nb] = S[16 * block[nb] + l16];
    }
  };

  float4_t acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = float4_t{0.f, 0.f, 0.f, 0.f};
  const float4_t zero = {0.f, 0.f, 0.f, 0.f};

  auto multiply = [&](const Stage& sg, const Weights& w) {
    if constexpr (P::kF8) {
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const int r = (wm * MB + mb) * 16 + l16;
        const uint4 a0 = sg.a[r * 8 + (quarter ^ (r & 7))];
        const uint4 a1 = sg.a[r * 8 + ((quarter + 4) ^ (r & 7))];
        const float as = sg.as[r];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float4_t d = mma_f8(w.b[nb][0], w.b[nb][1], a0, a1, zero);
          const float f = as * w.bs[nb / OB];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[mb][nb][i] = __builtin_fmaf(d[i], f, acc[mb][nb][i]);
        }
      }
    } else {
      ColParams c[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        c[nb] = make_col<P::kFmt>(
            __builtin_bit_cast(half2_t, (uint32_t)w.s[nb] | ((uint32_t)w.s[nb] << 16)), 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        half8_t wt[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) wt[nb] = unpack_col<P::kFmt>(word_of(w.b[nb][0], j), c[nb]);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const int r = (wm * MB + mb) * 16 + l16;
          const half8_t a = __builtin_bit_cast(
              half8_t, sg.a[(j >> 1) * TM * 8 + r * 8 + ((4 * (j & 1) + quarter) ^ (r & 7))]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = mma16<P::kFmt>(wt[nb], a, acc[mb][nb]);
        }
      }
    }
  };

  // Weights of K block kb + 1 are loaded into registers and the stage of
  // kb + NS - 1 into LDS, in this order, while block kb is multiplied: what
  // block kb waits for is older than the newest stage's loads.
  Stage* stages[4] = {&st0, &st1, reinterpret_cast<Stage*>(&st2), reinterpret_cast<Stage*>(&st3)};
  Weights weights[2];
  auto upto = [&](int kb) { return kb < kb1 ? kb : kb1 - 1; };
#pragma unroll
  for (int i = 0; i < NS - 2; ++i) load_stage(*stages[i], upto(kb0 + i));
  load_weights(weights[0], kb0);
  keep_load_order();
  load_stage(*stages[NS - 2], upto(kb0 + NS - 2));
  auto step = [&](int u, int kb) {
    stage_barrier<(NS > 2 ? LOADS : 0)>();
    load_weights(weights[(u + 1) & 1], upto(kb + 1));
    keep_load_order();
    load_stage(*stages[(u + NS - 1) % NS], upto(kb + NS - 1));
    keep_load_order();
    multiply(*stages[u], weights[u & 1]);
  };
  int kb = kb0;
  for (; kb + NS <= kb1; kb += NS) {
#pragma unroll
    for (int u = 0; u < NS; ++u) step(u, kb + u);
  }
#pragma unroll
  for (int u = 0; u < NS - 1; ++u)
    if (kb + u < kb1) step(u, kb + u);
  // no direct load may still be landing in LDS when the workgroup ends
  __builtin_amdgcn_s_waitcnt(0);

  if (p.splits > 1) {
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
    for (int s = 0; s < p.splits; ++s) {
      const __amdgpu_buffer_rsrc_t ps = coherent_rsrc(base + (int64_t)s * TE);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float4_t x = load_coherent(ps, frag0 + (mb * NB + nb) * 64);
          acc[mb][nb] = s == 0 ? x : acc[mb][nb] + x;
        }
    }
    if (threadIdx.x == 0)
      __hip_atomic_store(p.counters + t, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int r = rt.row0 + (wm * MB + mb) * 16 + l16;
#pragma unroll
    for (int ob = 0; ob < OB; ++ob) {
      const int c = 16 * (ob0 + ob) + 4 * quarter;
      float4_t x = acc[mb][ob];
      if constexpr (GATE)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = silu_gate(x[j], acc[mb][OB + ob][j]);
      if (r < rt.end && c < p.N) store4(p, (int64_t)r * p.N + c, x);
    }
  }
}

}  // namespace w4a16
