// Attention over the paged 4-bit cache (kv4_attention).
//
// Mathematics.  With key row k_j = (c_j - 8) s_j + z_j (codes c, scale s,
// offset z) a score is  q . k_j = s_j (q . c_j - 8 sum q) + z_j sum q, and
// with value row v_j likewise the output is
//   sum_j p_j v_j = sum_j (p_j s_j)(c_j - 8) + sum_j p_j z_j,
// so the codes go into the matrix instruction as they are and scales and
// offsets touch one number per key or per probability instead of D.
//
// Codes as operands.  Four bits c in the mantissa of an FP16 whose other bits
// are zero are the subnormal c 2^-24 (times a power of two by where they
// sit); the matrix instruction takes subnormals exactly.  One AND per two
// codes is then the unpacking.  The sums, though, are cut off relative to
// what the operands' exponents allow, and leading zeros of a subnormal count
// there.  So the codes are moved to the top of the mantissa, a shift or two
// per word, for 1% of a decode step: at the bottom an FP16 request of 100000
// tokens was four times the output's rounding off (one now), and logits were
// five times as far off.
//
// Layout.  The keys are the first operand (rows = 16 tokens), the queries the
// second (columns = 16 query rows), so lane l holds scores of column l % 16
// for tokens 4 (l / 16) + i.  The product with the values wants exactly those
// probabilities as its second operand (k = tokens), with values transposed as
// the first: lane l reads, for the eight tokens it holds probabilities of, the
// words of channels 8 (l % 16) .. + 7 and pairs tokens byte by byte.  Nothing
// crosses lanes, and every load is 16 bytes per lane.
//
// Softmax.  A running reference m per column (base 2, with the value scales
// in it): weights w = 2^(x - m) s stay below 2^15 for FP16, sums are FP32.  m
// moves only when a weight or the sum would leave its range, so the usual
// tile has no reduction across lanes and no rescaling.  The weights' rounding
// to FP16 is the only one before the output; the -8 is applied to the sum of
// the rounded weights (a product with a row of ones), so it cancels exactly.
// For BF16 outputs that rounding is an eighth of the output's own.  For FP16
// outputs it would be as large as it, so there the weights are two FP16
// numbers, the rounded weight and its remainder, and the product with the
// values runs twice.
//
// Work.  A workgroup has 8 or 16 query rows of one request and key/value
// head and a range of its tokens, which its four waves divide; ranges are
// joined by the workgroup that arrives last.  A tile of 32 tokens is loaded
// one tile ahead, straight into registers: nothing is shared between waves.
//
// What bounds it (D = 128): HBM in decode steps, 64 requests of 4096 tokens
// and 32 heads 129 us (6.1 TB/s), one of 131072 tokens and 8 heads 31 us (4.6
// TB/s: the start and the join take about 8 us); eight dependent trips to
// memory in short calls, one of 1000 tokens and 32 heads 8.5 us; vector and
// matrix instructions, which hardly overlap, with more rows: 24 requests of 5
// queries on windows of 4096 tokens, 32 heads on 8, D = 64, 32 us.
#include "kv4_attention.hpp"

namespace w4a16 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// Reductions without the LDS's lane exchanges (0.1 us each, one after
// another in a workgroup's start and end).  Over the four lane groups (lanes
// l, l ^ 16, l ^ 32, l ^ 48), by swaps of rows and halves:
template <typename Op>
__device__ __forceinline__ float over_groups(float x, Op op) {
  const uint32_t w = __builtin_bit_cast(uint32_t, x);
  const auto rows = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  x = op(__builtin_bit_cast(float, (uint32_t)rows[0]), __builtin_bit_cast(float, (uint32_t)rows[1]));
  const uint32_t v = __builtin_bit_cast(uint32_t, x);
  const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return op(__builtin_bit_cast(float, (uint32_t)halves[0]),
            __builtin_bit_cast(float, (uint32_t)halves[1]));
}
__device__ __forceinline__ float groups_sum(float x) {
  return over_groups(x, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float groups_max(float x) {
  return over_groups(x, [](float a, float b) { return fmaxf(a, b); });
}

// With at most eight rows, columns n and n + 8 are the same row.  The two
// lanes then divide the softmax (one takes the first unit's tokens, the other
// the second's), and FP16's two products with the values become one: columns
// below 8 take the rounded weights, the others the remainders.
template <int ROWS>
constexpr bool kPaired = ROWS == 8;

// The lane of the same four tokens eight columns on.
__device__ __forceinline__ uint32_t pair_lane(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xf, 0xf, true);  // row_ror:8
}
__device__ __forceinline__ float pair_lane(float x) {
  return __builtin_bit_cast(float, pair_lane(__builtin_bit_cast(uint32_t, x)));
}

// What one lane loads of two units.
template <int D, int ROWS>
struct TileData {
  static constexpr int PARAMS = kPaired<ROWS> ? 1 : 2;  // units a lane needs these of
  static constexpr int KV = D / 32;                 // key words per unit
  static constexpr int VV = D == 256 ? 2 : 1;       // value vectors per unit
  uint32_t k[2][KV];
  uint4v v[2][VV];
  uint4v kp[PARAMS], vp[PARAMS];
  bool valid[2];                                    // the unit's page exists
};

// Cache policy of the code loads.  With paired rows a workgroup alone reads
// them, once (non-temporal: 64 requests of 4096 tokens, 32 heads, 128 us, 147
// without); with more rows neighbouring row tiles find them in the L2 (91
// requests of 18 rows, 66 us, 77 with non-temporal loads).
template <int ROWS>
constexpr int kPolicy = kPaired<ROWS> ? 2 : 0;

// Where a head's units lie: page id `p` of it starts at
// cache + head offset + p * page stride.
struct Pages {
  const uint8_t* head;
  uint64_t stride;  // bytes of a page over all heads
  int shift, count; // log2 of a page's tokens, pages of the cache
};

template <int D, int ROWS>
__device__ __forceinline__ void load_tile(TileData<D, ROWS>& d, const Pages& pages, PageIds& ids,
                                          int t) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const uint8_t* base = nullptr;
  const uint8_t* bases[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (u == 0 || pages.shift == 4) {
      const int tu = t + kKvUnit * u;
      const int id = ids.at(tu >> pages.shift);
      d.valid[u] = (unsigned)id < (unsigned)pages.count;
      base = pages.head + (uint64_t)(uint32_t)(d.valid[u] ? id : 0) * pages.stride +
             (uint32_t)((tu & ((1 << pages.shift) - 1)) / kKvUnit * KvUnit<D>::bytes);
    } else {  // a larger page holds both units side by side
      d.valid[u] = d.valid[0];
      base += KvUnit<D>::bytes;
    }
    // one address for the wave, 32-bit offsets for the lanes
    const __amdgpu_buffer_rsrc_t unit = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(base), (short)0, KvUnit<D>::bytes, 0x00020000);
    auto load16 = [&](int at, int plus) {
      return __builtin_bit_cast(
          uint4v, __builtin_amdgcn_raw_buffer_load_b128(unit, at + plus, 0, kPolicy<ROWS>));
    };
    const int key = r * (D / 2) + g * (D / 8);
    if constexpr (D == 64) {
      const uint2v w =
          __builtin_bit_cast(
              uint2v, __builtin_amdgcn_raw_buffer_load_b64(unit, key, 0, kPolicy<ROWS>));
      d.k[u][0] = w[0];
      d.k[u][1] = w[1];
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4v w = load16(key, 16 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) d.k[u][4 * i + j] = w[j];
      }
    }
    const int value = g * (2 * D) + 16 * (D == 64 ? r >> 1 : r);
#pragma unroll
    for (int i = 0; i < TileData<D, ROWS>::VV; ++i)
      d.v[u][i] = load16(value, KvUnit<D>::values + 256 * i);
    if constexpr (!kPaired<ROWS>) {
      const uint8_t* mine = base + 16 * g;
      d.kp[u] = *reinterpret_cast<const uint4v*>(mine + KvUnit<D>::key_params);
      d.vp[u] = *reinterpret_cast<const uint4v*>(mine + KvUnit<D>::value_params);
    }
    bases[u] = base;
  }
  if constexpr (kPaired<ROWS>) {
    const uint8_t* mine = (lane & 8 ? bases[1] : bases[0]) + 16 * g;
    d.kp[0] = *reinterpret_cast<const uint4v*>(mine + KvUnit<D>::key_params);
    d.vp[0] = *reinterpret_cast<const uint4v*>(mine + KvUnit<D>::value_params);
  }
}

// The sums of the query rows over the tokens seen so far, for column (row)
// lane % 16.
template <int D>
struct Sums {
  float4v acc[D / 16];  // sum of w c, in the operands' units
  float4v w;            // sum of w (every element the same)
  float m;              // reference
  float l, z;           // this lane's part of sum p, sum p z
};

// A wave's query rows as operands, and what its columns need.
template <int D>
struct Queries {
  // channels by parity of the nibble; the odd ones, which meet codes of 16
  // times the size, are divided by 16
  uint4v even[D / 64], odd[D / 64];
  float sum8;  // -8 sum q, in the products' units
  float unit;  // product units to base-2 logits
  float sum;   // sum q in base-2 logits
  int lo, hi;  // keys seen: lo <= j <= hi
  float up;    // logits over what unit and sum make, 1 but for large rows, which
               // only the path that moves the reference provides for:
  float most_sum;  // kMostSum, or -1 if some row is large
};

// One tile.  `edge`: some of its tokens are not seen by some row.  What the
// cache holds for those may be anything (NaN included), so they are taken out
// of the probabilities and the weights, never multiplied by zero.
template <int D, int ROWS, bool BF16>
__device__ __forceinline__ void attend(const TileData<D, ROWS>& d, const Queries<D>& q,
                                       Sums<D>& s, int t, bool edge) {
  constexpr bool PAIRED = kPaired<ROWS>;
  constexpr int N = PAIRED ? 4 : 8;  // scores of a lane
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const bool upper = PAIRED && (lane & 8);

  // The sums start from zero, not from -8 sum q: what the matrix unit cuts off
  // goes by the largest addend.
  float4v raw[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    raw[u] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
      const uint32_t w0 = d.k[u][2 * p], w1 = d.k[u][2 * p + 1];
      const uint32_t a0 = w0 << 2, a1 = w1 << 2, b0 = w0 >> 6, b1 = w1 >> 6;
      const uint4v e = {a0 & kLowCodes, a1 & kLowCodes, b0 & kLowCodes, b1 & kLowCodes};
      const uint4v o = {a0 & kHighCodes, a1 & kHighCodes, b0 & kHighCodes, b1 & kHighCodes};
      raw[u] = mfma(e, q.even[p], raw[u]);
      raw[u] = mfma(o, q.odd[p], raw[u]);
    }
  }

  if constexpr (PAIRED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[0][i] = upper ? raw[1][i] : raw[0][i];
  }
#pragma unroll
  for (int u = 0; u < N / 4; ++u) raw[u] += q.sum8;
  auto key_params = [&](int i) { return d.kp[i >> 2][i & 3]; };
  auto value_params = [&](int i) { return d.vp[i >> 2][i & 3]; };
  float scale[N];  // of the keys, times the logits' unit
#pragma unroll
  for (int i = 0; i < N; ++i) scale[i] = times_low_half(q.unit, key_params(i));

  // FP16: the remainders of the weights' rounding as a second operand
  constexpr int kParts = BF16 || PAIRED ? 1 : 2;
  uint4v weights[kParts];
  float p[N], w[N], sum, most;
  auto seen = [&](int i) {
    const int j = (int)apart(t + 4 * g + (upper ? kKvUnit : 0)) + kKvUnit * (i >> 2) + (i & 3);
    return (upper ? d.valid[1] : d.valid[i >> 2]) && j >= q.lo && j <= q.hi;
  };
  // the logit less the reference: scale (q . c) + (offset sum q - m)
  auto logit_less_m = [&](int i) {
    return __builtin_fmaf(scale[i], raw[i >> 2][i & 3],
                          __builtin_fmaf(high_half(key_params(i)), q.sum, -s.m));
  };
  auto weigh = [&](auto&& less_m) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = exp2_hw(less_m(i));
      w[i] = times_low_half(p[i], value_params(i));
    }
    if (edge) {
      keep_branch();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        p[i] = seen(i) ? p[i] : 0.f;
        w[i] = seen(i) ? w[i] : 0.f;
      }
    }
    sum = 0.f;
    most = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += p[i];
#pragma unroll
    for (int i = 0; i < N; i += 2) most = fmaxf(fmaxf(most, w[i]), w[i + 1]);
  };
  weigh(logit_less_m);
  if (__any(most > kMostWeight || sum > q.most_sum)) {
    // Move the reference: the largest weight becomes 2^8, unless that lets
    // a probability exceed 2^40 (values of scale 0).  Each logit is formed
    // once: the reference comes from the same numbers that it is then taken
    // off, so however coarse FP32 is at their size the largest keeps its weight.
    float x[N], top = kNone;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = q.up * __builtin_fmaf(scale[i], raw[i >> 2][i & 3],
                                   high_half(apart(key_params(i))) * q.sum);
      const float y = !edge || seen(i) ? x[i] : -__builtin_inff();
      top = fmaxf(top, y + __builtin_amdgcn_logf(low_half(apart(value_params(i)))) - kTopWeight);
      top = fmaxf(top, y - kSumHeadroom);
    }
    top = groups_max(top);
    if constexpr (PAIRED) top = fmaxf(top, pair_lane(top));
    const float m = fmaxf(s.m, top);
    const float f = exp2_hw(s.m - m);
    s.m = m;
    s.l *= f;
    s.z *= f;
    s.w *= f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) s.acc[c] *= f;
    // (rounding may still say more than the move provides for: held to it)
    weigh([&](int i) { return held(x[i] - m, apart(value_params(i))); });
  }
  s.l += sum;
  if (edge) {
    keep_branch();
#pragma unroll
    for (int i = 0; i < N; ++i) s.z += seen(i) ? p[i] * high_half(apart(value_params(i))) : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s.z += p[i] * high_half(value_params(i));
  }
  uint32_t h[N / 2], rest[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    h[i] = pack_halves(w[2 * i], w[2 * i + 1]);
    if constexpr (!BF16)
      rest[i] = pack_halves(less_low_half(w[2 * i], h[i]), less_high_half(w[2 * i + 1], h[i]));
  }
  if constexpr (PAIRED) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t keep = BF16 ? h[i] : upper ? rest[i] : h[i];
      const uint32_t theirs = pair_lane(BF16 ? h[i] : upper ? h[i] : rest[i]);
      weights[0][i] = upper ? theirs : keep;
      weights[0][i + 2] = upper ? keep : theirs;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      weights[0][i] = h[i];
      if constexpr (kParts == 2) weights[1][i] = rest[i];
    }
  }

  const uint4v ones = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
#pragma unroll
  for (int k = 0; k < kParts; ++k) s.w = mfma(ones, weights[k], s.w);

  // Byte b of two tokens' words into the two halves of a register, moved up
  // by two bits like the keys' codes.  Words moved as they are serve for the
  // first three bytes, whose halves then take a bit field that spans two.
  const uint32_t half = D == 64 ? (lane & 1) * 0x00020002u : 0u;
  constexpr int kBytes = D == 64 ? 2 : 4;
#pragma unroll
  for (int i = 0; i < TileData<D, ROWS>::VV; ++i) {
    uint4v moved[2];
    if constexpr (D > 64) {
#pragma unroll
      for (int u = 0; u < 2; ++u) moved[u] = d.v[u][i] << 2;
    }
#pragma unroll
    for (int b = 0; b < kBytes; ++b) {
      uint4v e, o;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t both;
        if (D > 64 && b < 3) {
          const uint4v& v = moved[k >> 1];
          both = __builtin_amdgcn_perm(v[2 * (k & 1) + 1], v[2 * (k & 1)],
                                       0x05040100u + 0x01010101u * b);
        } else {
          const uint4v& v = d.v[k >> 1][i];
          both = __builtin_amdgcn_perm(v[2 * (k & 1) + 1], v[2 * (k & 1)],
                                       (0x0c040c00u + 0x00010001u * b) + half)
                 << 2;
        }
        e[k] = both & kLowCodes;
        o[k] = both & kHighCodes;
      }
      const int c = 2 * (kBytes * i + b);
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        s.acc[c] = mfma(e, weights[k], s.acc[c]);
        s.acc[c + 1] = mfma(o, weights[k], s.acc[c + 1]);
      }
    }
  }
}

template <int D, int ROWS, bool BF16>
__device__ __forceinline__ void load_queries(Queries<D>& q, const KvAttentionArgs& a,
                                             const Span& sp, int head, int group, int row0) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  uint4v raw[D / 64][2];
  auto element = [&](int p, int c) {
    const uint32_t w = raw[p][c >> 3][(c >> 1) & 3];
    const uint32_t bits = c & 1 ? w >> 16 : w & 0xffffu;
    if constexpr (BF16) return __builtin_bit_cast(float, bits << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  };
  // rows past the last repeat it; they are not stored
  const int want = row0 + (lane & (kPaired<ROWS> ? 7 : 15));
  const int row = want < sp.rows ? want : sp.rows - 1;
  const int i = a.group.of(row);
  const uint16_t* src = a.q.p + (int64_t)(sp.tok0 + i) * a.q.token +
                        (int64_t)(head * group + row - i * group) * a.q.head;
  uint32_t most = 0;
#pragma unroll
  for (int p = 0; p < D / 64; ++p) {
    const uint4v* w = reinterpret_cast<const uint4v*>(src + 8 * (g * (D / 32) + 2 * p));
    raw[p][0] = w[0];
    raw[p][1] = w[1];
#pragma unroll
    for (int c = 0; c < 16; ++c)
      most = max(most, __builtin_bit_cast(uint32_t, element(p, c)) & 0x7fffffffu);
  }
  // the row's largest magnitude, 0 with an infinity or a NaN
  float top = groups_max(
      __builtin_bit_cast(float, most < 0x7f800000u ? most : 0x7f800000u));
  top = top < __builtin_inff() ? top : 0.f;
  const int pos = sp.len - sp.nq + i;
  q.hi = pos;
  q.lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
  // Every row is brought near FP16's upper end by a power of two of its own:
  // a score keeps 2^-30 of the largest one its row could have, however small
  // the queries (the odd channels are divided by 16, which FP16's smallest
  // step would otherwise cut into).
  int e = exponent_of(top);
  e = e < -100 ? -100 : e;
  const float up = power_of_two(13 - e);
  const int by = large_by(a.scale, e);
  q.most_sum = __any(by > 0) ? -1.f : kMostSum;
  q.up = power_of_two(by < 127 ? by : 127);
  const float logits = a.scale * (kLog2e * power_of_two(e - 13 - by));
  q.unit = logits * 0x1p22f;
  float sum = 0.f;
#pragma unroll
  for (int p = 0; p < D / 64; ++p) {
    _Float16 h[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      h[c] = (_Float16)(element(p, c) * (c & 1 ? 0.0625f * up : up));
      sum += (float)h[c] * (c & 1 ? 16.0f : 1.0f);
    }
    const half8 even = {h[0], h[4], h[8], h[12], h[2], h[6], h[10], h[14]};
    const half8 odd = {h[1], h[5], h[9], h[13], h[3], h[7], h[11], h[15]};
    q.even[p] = __builtin_bit_cast(uint4v, even);
    q.odd[p] = __builtin_bit_cast(uint4v, odd);
  }
  sum = groups_sum(sum);
  q.sum8 = sum * -0x1p-19f;
  q.sum = sum * logits;
}

// Rows of D floats of a block in LDS, padded so that the 16 rows of a store
// fall on different banks.
template <int D>
constexpr int kLdsRow = D + 4;

// Waves per SIMD the registers are divided for.
template <int D, int ROWS>
constexpr int kResident = D <= 128 || kPaired<ROWS> ? 2 : 1;

template <int D, int ROWS, bool BF16>
__global__ __launch_bounds__(kThreads, (kResident<D, ROWS>)) void kv_tokens_kernel(
    KvAttentionArgs a, unsigned* __restrict__ counters, float* __restrict__ partials) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = (int)a.group.d, splits = (int)a.splits.d;
  // Row tiles of one token range read the same codes: workgroups 8 apart, in
  // turn on the same XCD, whose L2 then holds them (3 requests of 294 rows
  // over 16600 tokens: 97 -> 74 us).
  int id = blockIdx.x, tile = 0;
  const int tiles = (int)a.tiles.d;
  if (tiles > 1) {
    const int ranges = a.tiles.of(gridDim.x), whole = ranges & ~7;
    if (id < whole * tiles) {
      tile = a.tiles.rest(id >> 3);
      id = (a.tiles.of(id >> 3) << 3) + (id & 7);
    } else {
      const int in = id - whole * tiles, width = ranges - whole;
      tile = in / width;
      id = whole + in % width;
    }
  }
  const int split = a.splits.rest(id);
  id = a.splits.of(id);                     // (request, head)
  const int work = id * tiles + tile;
  const int head = a.heads.rest(id), b = a.heads.of(id);
  const int row0 = tile * ROWS;
  const Span sp = span_of(a, b, row0, ROWS);
  if (row0 >= sp.rows) return;
  const Range range = range_of(a, sp, split);
  if (split >= range.parts) return;
  // the waves divide the range
  const int each = ((range.end - range.begin + kTile - 1) / kTile + kWaves - 1) / kWaves * kTile;
  const int begin = range.begin + wave * each;
  const int end = begin + each < range.end ? begin + each : range.end;

  Queries<D> q;
  load_queries<D, ROWS, BF16>(q, a, sp, head, group, row0);
  Sums<D> s;
  s.m = kNone;
  s.l = s.z = 0.f;
  s.w = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < D / 16; ++c) s.acc[c] = float4v{0.f, 0.f, 0.f, 0.f};

  // Inner tiles, which every row sees whole, need no mask.
  const int row_last = row0 + ROWS < sp.rows ? row0 + ROWS - 1 : sp.rows - 1;
  const int pos_first = sp.len - sp.nq + a.group.of(row0);
  const int pos_last = sp.len - sp.nq + a.group.of(row_last);
  const int inner_end = pos_first + 1;  // exclusive
  const int inner_begin = a.window > 0 && pos_last >= a.window ? pos_last - a.window + 1 : 0;

  if (begin < end) {
    Pages pages;
    pages.shift = 31 - __builtin_clz((unsigned)a.page);
    pages.count = a.pages;
    const uint64_t page_bytes = (uint64_t)(a.page / kKvUnit) * KvUnit<D>::bytes;
    pages.stride = page_bytes * a.H;
    pages.head = a.cache + page_bytes * head;
    PageIds ids{a.table + (int64_t)b * a.max_pages, a.max_pages, 0, -1};
    ids.load(begin >> pages.shift);
    // A ring of tiles in registers: the loads of a tile are issued kAhead
    // tiles before it is used.  They are issued whatever is left (the last
    // tile again, at the end): where a branch could skip them, the wait for a
    // tile would have to allow for both sides and so wait for the next one.
    constexpr int kAhead = 1;
    TileData<D, ROWS> ring[kAhead + 1];
    const int last = begin + (end - begin - 1) / kTile * kTile;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int t = begin + k * kTile;
      load_tile<D, ROWS>(ring[k], pages, ids, t < last ? t : last);
    }
    for (int t0 = begin; t0 < end; t0 += (kAhead + 1) * kTile) {
#pragma unroll
      for (int k = 0; k <= kAhead; ++k) {
        const int t = t0 + k * kTile, then = t + kAhead * kTile;
        if (t >= end) break;
        load_tile<D, ROWS>(ring[(k + kAhead) % (kAhead + 1)], pages, ids,
                           then < last ? then : last);
        const TileData<D, ROWS>& cur = ring[k];
        const bool edge =
            t < inner_begin || t + kTile > inner_end || !cur.valid[0] || !cur.valid[1];
        attend<D, ROWS, BF16>(cur, q, s, t, edge);
      }
    }
  }

  // Each lane's rows as true sums: O (unnormalised), sum p.
  const int g = lane >> 4, n16 = lane & 15;
  if constexpr (kPaired<ROWS>) {
    s.l += pair_lane(s.l);
    s.z += pair_lane(s.z);
    if constexpr (!BF16) {
      s.w[0] += pair_lane(s.w[0]);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) s.acc[c][i] += pair_lane(s.acc[c][i]);
    }
  }
  const float total = groups_sum(s.l);
  const float fixed = groups_sum(s.z) - 8.0f * s.w[0];
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s.acc[c][i] = s.acc[c][i] * (c & 1 ? 0x1p18f : 0x1p22f) + fixed;

  constexpr int kCols = D == 64 ? 4 : 8;  // neighbouring channels of a lane
  // Join the waves, in wave order, through LDS: each leaves its rows and
  // their (m, l), and the threads add them up per element.
  constexpr int kSlab = ROWS * kLdsRow<D>;
  __shared__ float red[kWaves * kSlab];
  __shared__ float s_m[kWaves][ROWS], s_l[kWaves][ROWS];
  __shared__ bool s_last;
  const int rows = sp.rows - row0 < ROWS ? sp.rows - row0 : ROWS;
  if (n16 < rows) {
    if (g == 0) {
      s_m[wave][n16] = s.m;
      s_l[wave][n16] = total;
    }
    float* at = red + wave * kSlab + n16 * kLdsRow<D> + kCols * 4 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < D / 16; c += 4)
        *reinterpret_cast<float4v*>(at + kCols * i + c % kCols + c / kCols * 128) =
            float4v{s.acc[c][i], s.acc[c + 1][i], s.acc[c + 2][i], s.acc[c + 3][i]};
  }
  __syncthreads();
  // Four neighbouring channels of a row over all waves, and its (m, l).
  auto joined = [&](int row, int ch, float* m_out, float* l_out) {
    float m = s_m[0][row], l = 0.f;
#pragma unroll
    for (int o = 1; o < kWaves; ++o) m = fmaxf(m, s_m[o][row]);
    float4_t x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int o = 0; o < kWaves; ++o) {
      const float f = exp2_hw(s_m[o][row] - m);
      l += s_l[o][row] * f;
      x += *reinterpret_cast<const float4_t*>(red + o * kSlab + row * kLdsRow<D> + ch) * f;
    }
    *m_out = m;
    *l_out = l;
    return x;
  };
  constexpr int kVecs = D / 4;
  const Output out(a, sp, head);
  if (range.parts == 1) {
    for (int v = threadIdx.x; v < rows * kVecs; v += kThreads) {
      const int row = v / kVecs, ch = v % kVecs * 4;
      float m, l;
      const float4_t x = joined(row, ch, &m, &l);
      const float y[4] = {x[0], x[1], x[2], x[3]};
      out.store<BF16, 4>(row0 + row, ch, y, l == 0.f ? 0.f : 1.0f / l);
      if (ch == 0) out.store_lse(row0 + row, m, l);
    }
    return;
  }
  // Publish this workgroup's rows, then count the arrival; the last
  // workgroup of the row tile joins them in range order.
  constexpr int kVecsOfPart = ROWS * kPartVecs<D>;
  const float* tile_base = partials + (int64_t)work * splits * kVecsOfPart * 4;
  {
    const __amdgpu_buffer_rsrc_t mine = coherent_rsrc(tile_base + split * kVecsOfPart * 4);
    for (int v = threadIdx.x; v < rows * kVecs; v += kThreads) {
      const int row = v / kVecs, c = v % kVecs;
      float m, l;
      store_coherent(mine, row * kPartVecs<D> + c, joined(row, 4 * c, &m, &l));
      if (c == 0) store_coherent(mine, row * kPartVecs<D> + kVecs, float4_t{m, l, 0.f, 0.f});
    }
  }
  if (last_to_arrive(counters + work, range.parts, &s_last))
    join_parts<D, BF16, kThreads>(tile_base, kVecsOfPart, range.parts, rows, row0, out,
                                  counters + work);
}

template <int D, int ROWS>
hipError_t launch(const KvAttentionPlan& p, const KvAttentionArgs& a, int dtype,
                  unsigned* counters, float* partials, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.B * a.H * p.tiles * p.splits));
  if (dtype == W4A16_DTYPE_BF16)
    hipLaunchKernelGGL((kv_tokens_kernel<D, ROWS, true>), grid, dim3(kThreads), 0, stream, a,
                       counters, partials);
  else
    hipLaunchKernelGGL((kv_tokens_kernel<D, ROWS, false>), grid, dim3(kThreads), 0, stream, a,
                       counters, partials);
  return hipGetLastError();
}

template <int D>
hipError_t launch_d(const KvAttentionPlan& p, const KvAttentionArgs& a, int dtype,
                    unsigned* counters, float* partials, hipStream_t stream) {
  return p.row_tile == 8 ? launch<D, 8>(p, a, dtype, counters, partials, stream)
                         : launch<D, 16>(p, a, dtype, counters, partials, stream);
}

}  // namespace

hipError_t launch_kv_tokens(const KvAttentionPlan& p, const KvAttentionArgs& a, int D, int dtype,
                            unsigned* counters, float* partials, hipStream_t stream) {
  switch (D) {
    case 64: return launch_d<64>(p, a, dtype, counters, partials, stream);
    case 128: return launch_d<128>(p, a, dtype, counters, partials, stream);
    default: return launch_d<256>(p, a, dtype, counters, partials, stream);
  }
}

namespace {

// What partial results may take of a workspace.
constexpr int64_t kMostPartBytes = ((int64_t)192 << 20) - (int64_t)kCounterHeaderBytes;

// A plan for row tiles of `row_tile` rows, and an estimate of its time in us.
//
// A workgroup takes a step of 32 tokens (a wave of four, where waves divide
// the tokens) in `alone`, or in `shared` beside a second one on its compute
// unit; kStart steps go by before and after.  With up to eight rows a second
// one gains nothing: HBM bounds the first.  Rounds of workgroups end
// unevenly, and requests of a batch are taken to hold 0.65 of the longest
// one on average.  Token ranges cost their partial results' way to memory
// and back, and the join, in which one workgroup reads all of a row tile's.
// (Measured, with the best count of ranges and with one: one request of
// 131072 tokens, 8 heads, 32 ranges, 31 us, 208 with 3; 500 queries over
// 8192 tokens, 4, 137 us, 268 with one; 24 x 476 over 6597, 595 with 2, 478
// with one.)
// The 0.65 is a guess that uneven batches need and equal ones bear: 32 requests
// of 8192 tokens, 8 heads, take 50.1 us with it and 50.6 with 1, 8 of 32768
// 53.1 and 51.9; a quarter to all of those lengths 40.6 and 44.6, 43.7 and 48.1;
// 24 x 5 drafted tokens 30 and 37; 9 x 10 over 2636, 32 heads, 26 and 22.
// A request that holds far less than planned gets only the ranges its length
// fills: one of 4000 tokens on 8 heads takes 9.5 us planned for 4000 tokens, 23
// planned for 131072.
double plan_for(KvAttentionPlan* p, int row_tile, int B, int H, int64_t rows, int D,
                int64_t keys, int cus) {
  constexpr double kStart = 5, kJoin = 1.4, kPartsRate = 1e6, kJoinRate = 64e3;  // bytes per us
  constexpr double kUneven = 0.35, kAverage = 0.65;
  p->row_tile = row_tile;
  p->rows = row_tile == 128;
  p->waves = kWaves;
  p->tiles = (int)((rows + row_tile - 1) / row_tile);
  p->splits = 1;
  p->chunk = (int)(keys < (1 << 30) ? keys : (1 << 30));
  const int size = D == 64 ? 0 : D == 128 ? 1 : 2;
  constexpr double kAlone[3][3] = {{0.6, 0.75, 1.3}, {0.7, 0.8, 1.4}, {0.9, 1.05, 2.0}};
  constexpr double kShared[3][3] = {{0.6, 0.75, 1.3}, {0.8, 1.05, 1.4}, {1.2, 1.6, 2.0}};
  const int kind = row_tile == 8 ? 0 : row_tile == 16 ? 1 : 2;
  const double alone = kAlone[kind][size], shared = kShared[kind][size];
  const bool second = shared > alone;
  const int64_t work = (int64_t)B * H * p->tiles;
  const int64_t sharing = p->rows ? 1 : kWaves;  // waves that divide the tokens
  const int64_t steps = keys / kTile;
  const int64_t part = (int64_t)row_tile * (D + 4) * (int64_t)sizeof(float);
  int64_t most = (steps + sharing - 1) / sharing;
  if (most > 16 * (int64_t)cus / work + 1) most = 16 * (int64_t)cus / work + 1;
  if (most > kMostPartBytes / (work * part)) most = kMostPartBytes / (work * part);
  if (most < 1 || work > kMaxSplitTiles) most = 1;
  double best = 0;
  int64_t n = 1;
  for (int64_t i = 1; i <= most; i += 1 + i / 32) {
    const int64_t each = ((steps + i - 1) / i + sharing - 1) / sharing;
    const bool both = second && work * i > cus;
    const double load = (double)(work * i) / (both ? 2 * cus : cus);
    const double rounds = (B > 1 ? load * kAverage : load) + kUneven;
    double cost = (load <= 1 || rounds < 1 ? 1 : rounds) * (each + kStart) *
                  (both ? shared : alone);
    if (i > 1) cost += kJoin + work * i * part / kPartsRate + i * part / kJoinRate;
    if (i == 1 || cost < best) {
      best = cost;
      n = i;
    }
  }
  if (n > 1) {
    p->chunk = (int)((keys + n - 1) / n + kTile - 1) / kTile * kTile;
    p->splits = (int)((keys + p->chunk - 1) / p->chunk);
    p->workspace_bytes = kCounterHeaderBytes + (size_t)(work * p->splits * part);
  }
  return best;
}

}  // namespace

// Up to eight rows pair columns.  Beyond that tiles of 16 rows have the
// waits of two workgroups per compute unit overlap and waste few rows; tiles
// of 128 unpack the codes once for all, which pays when they are full and the
// chip is (2 x 2048 queries: 0.73 ms; 32 x 128 queries over 1024 tokens, 32
// heads: 105 us against 187 in tiles of 16; 8 x 96 over 2048: 78 against 48).
// Between them, at 65 to a few hundred rows per head, both are three to five
// times off what the bytes and flops take.
KvAttentionPlan make_kv_attention_plan(int B, int Hq, int H, int D, int max_q, int max_len,
                                       int window, int cus) {
  const int64_t rows = (int64_t)(Hq / H) * max_q;
  int64_t keys = max_len;
  if (window > 0 && keys > (int64_t)window + max_q) keys = (int64_t)window + max_q;
  keys = (keys + kTile - 1) / kTile * kTile + kTile;
  KvAttentionPlan few{}, many{};
  const double time = plan_for(&few, rows <= 8 ? 8 : 16, B, H, rows, D, keys, cus);
  if (rows <= 64) return few;
  return plan_for(&many, 128, B, H, rows, D, keys, cus) < time ? many : few;
}

hipError_t launch_kv_attention(const KvAttentionPlan& p, const KvAttentionArgs& args, int D,
                               int dtype, void* workspace, hipStream_t stream) {
  KvAttentionArgs a = args;
  a.tiles = Divisor(p.tiles);
  a.splits = Divisor(p.splits);
  a.chunk = Divisor(p.chunk);
  a.group = Divisor(a.Hq / a.H);
  a.heads = Divisor(a.H);
  unsigned* counters = static_cast<unsigned*>(workspace);
  float* partials =
      reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterHeaderBytes);
  return p.rows ? launch_kv_rows(p, a, D, dtype, counters, partials, stream)
                : launch_kv_tokens(p, a, D, dtype, counters, partials, stream);
}

}  // namespace w4a16
