// kv4_attention for many query rows: chunks of prompts, long drafts.
//
// The mathematics of kv4_attention.hip, arranged for rows.  A workgroup of
// four waves takes 128 query rows, 32 per wave, and walks their tokens 64 at
// a time.  Each step's codes are unpacked once per workgroup, into LDS, as
// FP16 and in the order in which the 32x32x16 matrix instruction takes its
// first operand, so a wave spends its vector instructions on the softmax and
// reads every operand with one conflict-free 16-byte LDS read.  The codes of
// the step after next are loaded, and those of the next one unpacked, around
// the products of the current one: one barrier per step, two stages of LDS,
// two workgroups per compute unit.
//
// What bounds it: the issue of vector and matrix instructions.  Measured with
// loops of both, matrix instructions of one wave and vector instructions of
// another hardly overlap on a SIMD (16 products and 120 vector instructions
// take 0.34 us per wave together, 0.22 and 0.17 alone), so a tile of 32 x 32
// scores costs their sum, 512 + about 880 cycles with D = 128, and the kernel
// runs at 0.92 of that: 2 x 2048 queries over up to 8192 keys, 64 heads of
// 128, BF16: 0.81 to 0.86 ms under the profiler, 0.72 to 0.75 without, 760 to
// 800 TFLOP/s (a 16384^3 product of the matrix library: 1364).  FP16 calls
// have the remainders' products too, 24 for 16, and form them: 555 TFLOP/s of
// the formula's (1.33 ms for prompts of 1.3 times the work).  BF16 with D = 64
// reaches 440, where a score's vector instructions serve half the products,
// and with D = 256 and one workgroup per compute unit 475.
// For the same reason these did not help, in ms for the BF16 case: two groups
// of waves that change places between softmax and products at barriers (0.91),
// eight waves per workgroup (0.85), the next tile's products between the
// softmax's instructions (0.87 of the time before the masks left the usual
// path, spills), steps of 32 tokens (0.93), wave priorities around the products
// (0.85).
//
// Operands.  Scores: keys first (rows = 32 tokens), queries second (columns =
// 32 query rows); lane l has column l % 32 and, for i in 0..15, token
// 8 (i / 4) + 4 (l / 32) + i % 4.  Values: transposed values first (rows =
// 32 channels), weights second (k = 16 tokens): half h = l / 32 supplies the
// tokens 4 h + j and 8 + 4 h + j of a unit, the ones it has scores of.  Row r
// of channel block b stands for channel 8 (r % W) + M b + r / W, where
// W = D / 8 words and M = 32 / W, so that a producer lane's word fills 16
// bytes at neighbouring places and a lane ends up with eight neighbouring
// channels.
#include "kv4_attention.hpp"

namespace w4a16 {
namespace {

constexpr int kStep = 64;  // tokens of a step: two tiles, four units

typedef float float16v __attribute__((ext_vector_type(16)));

constexpr int kWaves = 4, kThreads = 64 * kWaves, kRowTile = 32 * kWaves;

template <int D>
struct Stage {
  static constexpr int F = D / 16, CB = D / 32;
  uint4v k[2][F][64];      // [tile][16 channels][lane]
  uint4v v[2][2][CB][64];  // [tile][unit][channel block][lane]
  float ks[kStep];         // key scale, product units to base-2 logits
  float kz[kStep];         // key offset - 8 scales
  uint32_t vp[kStep];      // value (scale, offset)
  uint16_t there[4];       // per unit: all ones if its page exists
};

__device__ __forceinline__ float16v mfma32(const uint4v& a, const uint4v& b, const float16v& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a),
                                                __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

// The codes in bits 0..3 (low) or 4..7 (high) of both halves, less 8: the
// bits of 1024 + c or 64 + c, less 1032 or 72.  The masks are values in
// vector registers, for one instruction that ANDs and ORs.
__device__ __forceinline__ uint32_t low_codes(uint32_t w, uint32_t mask) {
  const half2v h = __builtin_bit_cast(half2v, (w & mask) | 0x64006400u);
  return __builtin_bit_cast(uint32_t, h - half2v{(_Float16)1032.f, (_Float16)1032.f});
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w, uint32_t mask) {
  const half2v h = __builtin_bit_cast(half2v, (w & mask) | 0x54005400u);
  return __builtin_bit_cast(uint32_t, h - half2v{(_Float16)72.f, (_Float16)72.f});
}

// What a wave unpacks of a step, as jobs of 64 lanes.  A key job: 64 / J
// tokens, J = D / 32 lanes with four words each.  A value job: the eight
// tokens of a unit that one lane half multiplies, half of the channels of one
// word per lane.  With D >= 128 a job lies in one unit, so its page is the
// same for all lanes; with D = 64 it covers two.
template <int D>
struct Producer {
  static constexpr int W = D / 8, J = D / 32;
  static constexpr int kJobs = J;                // of each kind, in a step
  static constexpr int kUnits = 4;               // of a step
  static constexpr int kMine = (2 * kJobs + kWaves - 1) / kWaves;
  static constexpr int kUnitsOfJob = D == 64 ? 2 : 1;

  const uint8_t* head;   // the head's first page
  uint64_t stride;       // bytes of a page over all heads
  PageIds ids;           // the request's pages
  int shift, pages, wave;
  uint4v a[kMine], b[kMine];
  uint32_t kp, vp;
  bool valid;

  // Job m of this wave: its kind, and its first unit.  D = 64: waves 0, 1
  // keys, 2, 3 values; D = 128: a unit's keys and values; D = 256: a unit's
  // two key jobs and two value jobs.
  __device__ __forceinline__ bool keys(int m) const {
    return D == 64 ? wave < 2 : m < kMine / 2;
  }
  __device__ __forceinline__ int unit_of(int m) const { return D == 64 ? 2 * (wave & 1) : wave; }
  // which of the unit's jobs of its kind
  __device__ __forceinline__ int part_of(int m) const { return D == 256 ? m & 1 : 0; }

  __device__ __forceinline__ const uint8_t* unit_at(int t, bool* there) {
    const int id = ids.at(t >> shift);
    *there = (unsigned)id < (unsigned)pages;
    return head + (uint64_t)(uint32_t)(*there ? id : 0) * stride +
           (uint32_t)((t & ((1 << shift) - 1)) / kKvUnit * KvUnit<D>::bytes);
  }

  __device__ __forceinline__ void load(int t) {  // codes of the step at t
    const uint32_t lane = threadIdx.x & 63;
    bool there0, there1 = true;
    const uint8_t* base0 = unit_at(t + kKvUnit * unit_of(0), &there0);
    const uint8_t* base1 = base0;
    if constexpr (kUnitsOfJob == 2) base1 = unit_at(t + kKvUnit * (unit_of(0) + 1), &there1);
    const uint8_t* unit = base0;
    if constexpr (kUnitsOfJob == 2) unit = lane < 32 ? base0 : base1;
    valid = kUnitsOfJob == 2 && lane >= 32 ? there1 : there0;
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      if (keys(m)) {
        const uint32_t x = lane + 64 * part_of(m), r = x % 16;
        const uint32_t q = x / 16 % J;
        a[m] = *reinterpret_cast<const uint4v*>(unit + r * (D / 2) + 16 * q);
        if (m == 0) {
          kp = *reinterpret_cast<const uint32_t*>(unit + KvUnit<D>::key_params + 4 * r);
          vp = *reinterpret_cast<const uint32_t*>(unit + KvUnit<D>::value_params + 4 * r);
        }
      } else {
        const uint32_t w = lane % W, h = lane / W % 2;
        const uint32_t at = KvUnit<D>::values + 16 * (h * W + w);
        a[m] = *reinterpret_cast<const uint4v*>(unit + at);
        b[m] = *reinterpret_cast<const uint4v*>(unit + at + 32 * W);
      }
    }
  }

  __device__ __forceinline__ void unpack(Stage<D>& st, float unit_of_logits) {
    const int lane = threadIdx.x & 63;
    constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
    const uint32_t low = apart(kLow), high = apart(kHigh);
    const int unit = unit_of(0) + (kUnitsOfJob == 2 ? lane / 32 : 0);
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      if (keys(m)) {
        const int x = lane + 64 * part_of(m), r = 16 * (unit % 2) + x % 16, q = x / 16 % J;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = a[m][i] << 2, w8 = a[m][i] >> 6;
          // word 4 q + i; subnormals 4 c 2^-24 and 64 c 2^-24, as in the other kernel
          st.k[unit / 2][2 * q + i / 2][32 * (i % 2) + r] =
              uint4v{w & kLowCodes, w & kHighCodes, w8 & kLowCodes, w8 & kHighCodes};
        }
        if (m == 0 && q == 0) {
          const int token = 16 * unit + lane % 16;
          st.ks[token] = low_half(kp) * unit_of_logits * 0x1p22f;
          st.kz[token] = high_half(kp) - 8.f * low_half(kp);
          st.vp[token] = vp;
          if (lane % 16 == 0) st.there[unit] = valid ? 0xffffu : 0u;
        }
      } else {
        constexpr int M = 32 / W;
        const int w = lane % W, h = lane / W % 2;
        const int part = D == 256 ? part_of(m) : lane / (2 * W) % 2;
        const uint4v* src[2] = {&a[m], &b[m]};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t sel = 0x0c040c00u + 0x00010001u * (2 * part + k);
          uint4v even, odd;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4v& s = *src[i / 2];
            const uint32_t both = __builtin_amdgcn_perm(s[2 * (i % 2) + 1], s[2 * (i % 2)], sel);
            even[i] = low_codes(both, low);
            odd[i] = high_codes(both, high);
          }
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int c = 4 * part + 2 * k + o;  // channel of the word
            st.v[unit / 2][unit % 2][c / M][32 * h + w + W * (c % M)] = o ? odd : even;
          }
        }
      }
    }
  }
};

// One tile of 32 tokens for a wave's 32 rows.
template <int D>
struct RowSums {
  float16v acc[D / 32];  // sum of w (c - 8)
  float m, l, z;         // reference; this lane's part of sum p, sum p z
};

template <int D>
__device__ __forceinline__ float16v scores(const Stage<D>& st, int tile, const uint4v* q) {
  const int lane = threadIdx.x & 63;
  float16v raw;
#pragma unroll
  for (int i = 0; i < 16; ++i) raw[i] = 0.f;
#pragma unroll
  for (int f = 0; f < D / 16; ++f) raw = mfma32(st.k[tile][f][lane], q[f], raw);
  return raw;
}

// A logit by itself, where the reference moves; `up` is 1 but for large rows.
__device__ __forceinline__ float logit(float ks, float product, float kz, float sum_q, float up) {
  return up * __builtin_fmaf(ks, product, kz * sum_q);
}

// The probabilities of a tile under reference m: packed weights, and their
// sums.  Parameters are read as they are used, four tokens at a time.  EDGE:
// some token is not seen by some row; what the cache holds for it may be
// anything, so it is taken out, not multiplied by zero.  (Rows of very unlike
// sizes go this way too, with `back`, so that it costs the usual way nothing.)
// AGAIN: after the reference has moved.  most_sum: kMostSum, or -1 where the
// logits are large and only the rare path, which moves it, provides for them.
template <bool BF16>
struct Weights {
  uint4v w[2];                   // [unit]
  uint4v rest[BF16 ? 1 : 2];     // FP16: the remainders of their rounding
  float sum, z;
  bool over;                     // out of the reference's range
};

template <int D, bool BF16, bool EDGE, bool AGAIN = false>
__device__ __forceinline__ void weigh(Weights<BF16>& o, const Stage<D>& st, int tile,
                                      const float16v& raw, float sum_q, float back, float up,
                                      float most_sum, float m, uint32_t there, int t, int lo,
                                      int hi) {
  const int h = (threadIdx.x & 63) >> 5;
  // known here only: the usual path must not compute masks or products
  if constexpr (EDGE) {
    t = (int)apart(t);
    there = apart(there);
    back = __builtin_bit_cast(float, apart(__builtin_bit_cast(uint32_t, back)));
  }
  const _Float16 kMostHalf = (_Float16)kMostWeight;  // what is larger rounds to it, or to infinity
  half2v most;
  o.sum = o.z = 0.f;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int at = 8 * a + 4 * h;
    const float4v ks = *reinterpret_cast<const float4v*>(&st.ks[32 * tile + at]);
    const float4v kz = *reinterpret_cast<const float4v*>(&st.kz[32 * tile + at]);
    const uint4v vp = *reinterpret_cast<const uint4v*>(&st.vp[32 * tile + at]);
    float w[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float product = EDGE ? raw[4 * a + r] * back : raw[4 * a + r];
      const float x = AGAIN ? held(logit(ks[r], product, kz[r], sum_q, up) - m, vp[r])
                            : __builtin_fmaf(ks[r], product, __builtin_fmaf(kz[r], sum_q, -m));
      float p = exp2_hw(x);
      w[r] = times_low_half(p, vp[r]);
      float z = high_half(vp[r]);
      if constexpr (EDGE) {
        const int j = t + at + r;
        const bool seen = (there >> (at + r) & 1) && j >= lo && j <= hi;
        p = seen ? p : 0.f;
        w[r] = seen ? w[r] : 0.f;
        z = seen ? z : 0.f;
      }
      o.sum += p;
      o.z = __builtin_fmaf(p, z, o.z);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t x = pack_halves(w[2 * k], w[2 * k + 1]);
      o.w[a / 2][2 * (a % 2) + k] = x;
      most = a == 0 && k == 0 ? __builtin_bit_cast(half2v, x)
                              : __builtin_elementwise_max(most, __builtin_bit_cast(half2v, x));
      if constexpr (!BF16)
        o.rest[a / 2][2 * (a % 2) + k] =
            pack_halves(less_low_half(w[2 * k], x), less_high_half(w[2 * k + 1], x));
    }
  }
  o.over = most[0] > kMostHalf || most[1] > kMostHalf || o.sum > most_sum;
}

template <int D, bool BF16>
__device__ __forceinline__ void attend_rows(const Stage<D>& st, int tile, const uint4v* q,
                                            float sum_q, float back, float up, float most_sum,
                                            RowSums<D>& s, uint32_t there, int t, bool edge,
                                            int lo, int hi) {
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const float16v raw = scores<D>(st, tile, q);
  Weights<BF16> o;
  if (edge)
    weigh<D, BF16, true>(o, st, tile, raw, sum_q, back, up, most_sum, s.m, there, t, lo, hi);
  else
    weigh<D, BF16, false>(o, st, tile, raw, sum_q, back, up, most_sum, s.m, there, t, lo, hi);
  if (__any(o.over)) {
    // Move the reference, as the other kernel does, from the same logits that
    // `weigh` then takes it off.
    float top = kNone;
    const int t1 = (int)apart(t);
    const uint32_t there1 = apart(there);
    const float back1 = __builtin_bit_cast(float, apart(__builtin_bit_cast(uint32_t, back)));
#pragma unroll 1
    for (int a = 0; a < 4; ++a) {
      const int at = 8 * a + 4 * h;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = t1 + at + r, i = 32 * tile + at + r;
        const float got = a == 0 ? raw[r] : a == 1 ? raw[4 + r] : a == 2 ? raw[8 + r] : raw[12 + r];
        const float x = logit(st.ks[i], got * back1, st.kz[i], sum_q, up);
        const bool seen = (there1 >> (at + r) & 1) && j >= lo && j <= hi;
        const float y = fmaxf(x + __builtin_amdgcn_logf(low_half(st.vp[i])) - kTopWeight,
                              x - kSumHeadroom);
        top = seen ? fmaxf(top, y) : top;
      }
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m = fmaxf(s.m, top);
    const float f = exp2_hw(s.m - m);
    s.m = m;
    s.l *= f;
    s.z *= f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) s.acc[c] *= f;
    weigh<D, BF16, true, true>(o, st, tile, raw, sum_q, back, up, most_sum, s.m, there, t, lo, hi);
  }
  s.l += o.sum;
  s.z += o.z;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const uint4v v = st.v[tile][u][c][lane];
      s.acc[c] = mfma32(v, o.w[u], s.acc[c]);
      if constexpr (!BF16) s.acc[c] = mfma32(v, o.rest[u], s.acc[c]);
    }
}

template <int D, bool BF16>
__global__ __launch_bounds__(kThreads, (D == 256 ? 1 : 2)) void kv_rows_kernel(
    KvAttentionArgs a, unsigned* __restrict__ counters, float* __restrict__ partials) {
  constexpr int F = D / 16, CB = D / 32, W = D / 8, M = 32 / W;
  __shared__ Stage<D> stage[2];
  __shared__ float s_top[kWaves], s_low[kWaves];
  __shared__ bool s_last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5;
  const int group = (int)a.group.d, splits = (int)a.splits.d;
  // Heads next to each other (they go to unlike XCDs), then the row tiles of
  // a request, the last, which see the most tokens, first.  Neighbours in this
  // order are about equally long: the shader engines take workgroups in turn,
  // so requests of unlike lengths side by side would load them unevenly
  // (two requests, one three times as long: 1.21 against 0.87 ms).
  int id = blockIdx.x;
  const int split = a.splits.rest(id), tiles = (int)a.tiles.d;
  id = a.splits.of(id);
  const int head = a.heads.rest(id);
  id = a.heads.of(id);
  const int tile = tiles - 1 - a.tiles.rest(id), b = a.tiles.of(id);
  const int work = (b * a.H + head) * tiles + tile;
  const int row0 = tile * kRowTile;
  const Span sp = span_of(a, b, row0, kRowTile);
  if (row0 >= sp.rows) return;
  const Range range = range_of(a, sp, split);
  if (split >= range.parts) return;

  // This wave's rows; rows past the last repeat it and are not stored.
  const int wave_row0 = row0 + 32 * wave;
  const bool idle = wave_row0 >= sp.rows;
  const int want = wave_row0 + (lane & 31);
  const int row = want < sp.rows ? want : sp.rows - 1;
  const int qi = a.group.of(row);
  const uint16_t* src = a.q.p + (int64_t)(sp.tok0 + qi) * a.q.token +
                        (int64_t)(head * group + row - qi * group) * a.q.head;
  const int pos = sp.len - sp.nq + qi;
  const int lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
  const int pos_first = __shfl(pos, 0), pos_last = __shfl(pos, 31);
  const int lo_first = __shfl(lo, 0), lo_last = __shfl(lo, 31);

  Producer<D> pr;
  const uint64_t page_bytes = (uint64_t)(a.page / kKvUnit) * KvUnit<D>::bytes;
  pr.head = a.cache + page_bytes * head;
  pr.stride = page_bytes * a.H;
  pr.shift = 31 - __builtin_clz((unsigned)a.page);
  pr.ids = PageIds{a.table + (int64_t)b * a.max_pages, a.max_pages, 0, -1};
  pr.pages = a.pages;
  pr.wave = wave;
  const int begin = range.begin;
  const int steps = (range.end - begin + kStep - 1) / kStep;
  if (steps > 0) {
    pr.ids.load(begin >> pr.shift);
    pr.load(begin);
  }

  // Queries as operands: 16-bit floats times one power of two that brings the
  // workgroup's largest finite row near FP16's upper end; the keys' scales
  // are stored in logits with it.  Rows that would lose bits by that, 2^-10
  // of the largest or smaller, are rare: then (`wide`) every row has a power
  // of its own, and its products are brought back by it.  (The unit of the
  // logits then goes by 2^20 or the largest row, if that is smaller: both it
  // and every row's way back are numbers FP32 holds.)  Rows whose logits may
  // be large go that way too, formed 2^`by` times smaller.
  uint4v q[F];
  float sum_q = 0.f, unit, back = 1.f, up_logits, most_sum;
  bool wide;
  {
    uint4v raw[F];
    uint32_t most = 0;
    auto element = [&](int f, int c) {
      const uint32_t w = raw[f][c >> 1];
      const uint32_t bits = c & 1 ? w >> 16 : w & 0xffffu;
      if constexpr (BF16) return __builtin_bit_cast(float, bits << 16);
      else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
    };
#pragma unroll
    for (int f = 0; f < F; ++f) {
      raw[f] = *reinterpret_cast<const uint4v*>(src + 16 * f + 8 * h);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        most = max(most, __builtin_bit_cast(uint32_t, element(f, c)) & 0x7fffffffu);
    }
    most = max(most, (uint32_t)__shfl_xor((int)most, 32));
    float top = most < 0x7f800000u ? __builtin_bit_cast(float, most) : 0.f;
    auto exponent = [](float x) {
      const int e = exponent_of(x);
      return e < -100 ? -100 : e;
    };
    const float mine = top;
    float low = top > 0.f ? top : __builtin_inff();
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      top = fmaxf(top, __shfl_xor(top, d));
      low = fminf(low, __shfl_xor(low, d));
    }
    if (lane == 0) {
      s_top[wave] = top;
      s_low[wave] = low;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      top = fmaxf(top, s_top[w]);
      low = fminf(low, s_low[w]);
    }
    const int most_e = __builtin_amdgcn_readfirstlane(exponent(top));
    const int by = large_by(a.scale, most_e);
    most_sum = by > 0 ? -1.f : kMostSum;
    wide = by > 0 || __builtin_amdgcn_readfirstlane(low < top * 0x1p-10f);
    const int e = wide ? exponent(mine) : most_e, base = wide && most_e > 20 ? 20 : most_e;
    const float up = power_of_two(13 - e);
    up_logits = power_of_two(by < 127 ? by : 127);
    unit = a.scale * (kLog2e * power_of_two(base - 13 - by > -126 ? base - 13 - by : -126));
    if (wide) back = power_of_two(e - base > -126 ? e - base : -126);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      _Float16 x[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        // odd channels meet codes of 16 times the size
        x[c] = (_Float16)(element(f, c) * (c & 1 ? 0.0625f * up : up));
        sum_q += (float)x[c] * (c & 1 ? 16.f : 1.f);
      }
      // the order in which a word's codes are unpacked
      const half8 v = {x[0], x[4], x[1], x[5], x[2], x[6], x[3], x[7]};
      q[f] = __builtin_bit_cast(uint4v, v);
    }
    sum_q += __shfl_xor(sum_q, 32);
    sum_q = sum_q * unit * back;
  }

  RowSums<D> s;
  s.m = kNone;
  s.l = s.z = 0.f;
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) s.acc[c][i] = 0.f;

  if (steps > 0) {
    pr.unpack(stage[0], unit);
    if (steps > 1) pr.load(begin + kStep);
    __syncthreads();
    for (int n = 0; n < steps; ++n) {
      const Stage<D>& st = stage[n & 1];
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const int t = begin + n * kStep + k * kTile;
        // tiles beyond the range belong to the next workgroup, or to none
        if (idle || t >= range.end || t > pos_last || t + kTile <= lo_first) continue;
        const uint32_t there = st.there[2 * k] | (uint32_t)st.there[2 * k + 1] << 16;
        const bool edge = t < lo_last || t + kTile > pos_first + 1 || there != 0xffffffffu || wide;
        attend_rows<D, BF16>(st, k, q, sum_q, back, up_logits, most_sum, s, there, t, edge, lo,
                             pos);
      }
      if (n + 1 < steps) {
        pr.unpack(stage[(n + 1) & 1], unit);
        if (n + 2 < steps) pr.load(begin + (n + 2) * kStep);
      }
      __syncthreads();
    }
  }

  const Output out(a, sp, head);
  const float total = s.l + __shfl_xor(s.l, 32);
  const float fixed = s.z + __shfl_xor(s.z, 32);
  // Eight neighbouring channels of word 8 k + 4 h + r of this lane's row.
  auto channels = [&](int k, int r, float* x) {
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = s.acc[c / M][4 * (k + W / 8 * (c % M)) + r] + fixed;
  };
  if (range.parts == 1) {
    if (want < sp.rows) {
      const float inv = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
      for (int k = 0; k < W / 8; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x[8];
          channels(k, r, x);
          out.store<BF16, 8>(row, 8 * (8 * k + 4 * h + r), x, inv);
        }
      if (h == 0) out.store_lse(row, s.m, total);
    }
    return;
  }
  const int rows = sp.rows - row0 < kRowTile ? sp.rows - row0 : kRowTile;
  constexpr int kVecsOfPart = kRowTile * kPartVecs<D>;
  const float* tile_base = partials + (int64_t)work * splits * kVecsOfPart * 4;
  if (want < sp.rows) {
    const __amdgpu_buffer_rsrc_t mine =
        coherent_rsrc(tile_base + (int64_t)split * kVecsOfPart * 4);
    const int base = (want - row0) * kPartVecs<D>;
#pragma unroll
    for (int k = 0; k < W / 8; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float x[8];
        channels(k, r, x);
        const int at = base + 2 * (8 * k + 4 * h + r);
        store_coherent(mine, at, float4_t{x[0], x[1], x[2], x[3]});
        store_coherent(mine, at + 1, float4_t{x[4], x[5], x[6], x[7]});
      }
    if (h == 0) store_coherent(mine, base + D / 4, float4_t{s.m, total, 0.f, 0.f});
  }
  if (last_to_arrive(counters + work, range.parts, &s_last))
    join_parts<D, BF16, kThreads>(tile_base, kVecsOfPart, range.parts, rows, row0, out,
                                  counters + work);
}

template <int D>
hipError_t launch(const KvAttentionPlan& p, const KvAttentionArgs& a, int dtype,
                  unsigned* counters, float* partials, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.B * a.H * p.tiles * p.splits));
  const dim3 block(kThreads);
  if (dtype == W4A16_DTYPE_BF16)
    hipLaunchKernelGGL((kv_rows_kernel<D, true>), grid, block, 0, stream, a, counters,
                       partials);
  else
    hipLaunchKernelGGL((kv_rows_kernel<D, false>), grid, block, 0, stream, a, counters,
                       partials);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_rows(const KvAttentionPlan& p, const KvAttentionArgs& a, int D, int dtype,
                          unsigned* counters, float* partials, hipStream_t stream) {
  switch (D) {
    case 64: return launch<64>(p, a, dtype, counters, partials, stream);
    case 128: return launch<128>(p, a, dtype, counters, partials, stream);
    default: return launch<256>(p, a, dtype, counters, partials, stream);
  }
}

}  // namespace w4a16
