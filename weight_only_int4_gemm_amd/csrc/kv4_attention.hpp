// Pieces shared by the two kernels of kv4_attention: kv4_attention.hip (few
// query rows, tokens divided over waves) and kv4_prefill.hip (many rows).
#pragma once

#include "../../include/w4a16_kv4.h"
#include "coherent.hpp"
#include "internal.hpp"
#include "kv4.hpp"

namespace w4a16 {

constexpr int kTile = 32;                   // tokens of one step: two units
constexpr int kWaitLoads = 0x0f70;          // s_waitcnt: all vector loads, nothing else
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr uint32_t kLowCodes = 0x003c003cu, kHighCodes = 0x03c003c0u;  // of codes, moved up by two bits
// Reference of a column that has seen no key: below every logit (base 2) that
// FP32 holds, and finite, so that differences of two are numbers.
constexpr float kNone = -0x1.fffffep127f;
constexpr float kMostWeight = 32768.0f;     // of a weight, before the reference moves
constexpr float kTopWeight = 8.0f;          // log2 of the largest weight after it has
constexpr float kMostSum = 0x1p60f;         // of a tile's probabilities, likewise
constexpr float kSumHeadroom = 40.0f;       // log2 of a probability over the reference

// Logits whose size may pass 2^kMostLogits (the scale's exponent plus that of a
// row's largest query) are formed 2^large_by() smaller: FP32 then holds every
// number on the way, whatever the parameters (2^16, 23 of them) and channels.
constexpr int kMostLogits = 95;

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int exponent_of(float x) {  // x >= 0
  return (int)(__builtin_bit_cast(uint32_t, x) >> 23) - 127;
}
__device__ __forceinline__ float power_of_two(int e) {  // -126 <= e <= 127
  return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
}
__device__ __forceinline__ int large_by(float scale, int e) {
  const int by = exponent_of(scale) + e - kMostLogits;
  return by > 0 ? by : 0;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float4v mfma(const uint4v& a, const uint4v& b, const float4v& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float low_half(uint32_t w) {
  return (float)__builtin_bit_cast(half2v, w)[0];
}
__device__ __forceinline__ float high_half(uint32_t w) {
  return (float)__builtin_bit_cast(half2v, w)[1];
}
__device__ __forceinline__ uint32_t pack_halves(float a, float b) {
  const half2v h = {(_Float16)a, (_Float16)b};  // round half to even
  return __builtin_bit_cast(uint32_t, h);
}

// x times, or less, a half of w in one mixed-precision instruction: a fused
// multiply-add whose constant the compiler does not know (with 0 and -1 it
// converts first and multiplies or subtracts then).
__device__ __forceinline__ float unknown(float x) {
  asm("" : "+s"(x));
  return x;
}
__device__ __forceinline__ float times_low_half(float x, uint32_t w) {
  return __builtin_fmaf(x, low_half(w), unknown(0.f));
}
__device__ __forceinline__ float less_low_half(float x, uint32_t w) {
  return __builtin_fmaf(low_half(w), unknown(-1.f), x);
}
__device__ __forceinline__ float less_high_half(float x, uint32_t w) {
  return __builtin_fmaf(high_half(w), unknown(-1.f), x);
}

// Keeps the compiler from doing a rare branch's work always, with selects,
// and from sharing its conversions with the usual path, where they cost
// nothing as operands of a mixed-precision instruction.
__device__ __forceinline__ void keep_branch() { asm volatile(""); }
__device__ __forceinline__ uint32_t apart(uint32_t w) {
  asm volatile("" : "+v"(w));
  return w;
}

// A logit less its moved reference, at most what the move provides for:
// weights 2^kTopWeight (one more for rounding), probabilities 2^kSumHeadroom.
// A NaN stays one.
__device__ __forceinline__ float held(float x, uint32_t value_params) {
  const float most =
      fminf(kTopWeight - __builtin_amdgcn_logf(low_half(value_params)), kSumHeadroom) + 1.f;
  return x > most ? most : x;
}

// Query rows of a workgroup and the tokens they see.
struct Span {
  int len, nq, tok0;    // tokens held, queries, first query row of the request
  int rows;             // query rows (query, head of the group) of the request
  int begin, end;       // tokens any row of the tile sees: begin (multiple of
                        // kTile) <= j < end
};

// The tokens of a row tile.
__device__ __forceinline__ Span span_of(const KvAttentionArgs& a, int b, int row0,
                                        int row_tile) {
  Span s;
  const int64_t most = (int64_t)a.max_pages * a.page;
  const int len = a.lens[b] > 0 ? a.lens[b] : 0;
  s.len = len < most ? len : (int)most;
  if (a.q_start) {
    int lo = a.q_start[b], hi = a.q_start[b + 1];
    lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
    hi = hi < lo ? lo : hi > a.T ? a.T : hi;
    s.tok0 = lo;
    s.nq = hi - lo;
  } else {
    s.tok0 = b;
    s.nq = b < a.T;
  }
  // queries beyond max_q are not computed
  const int nq = s.nq < a.max_q ? s.nq : a.max_q;
  s.rows = nq * (int)a.group.d;
  const int last = row0 + row_tile < s.rows ? row0 + row_tile : s.rows;
  const int first_pos = s.len - s.nq + a.group.of(row0);
  const int last_pos = s.len - s.nq + a.group.of(last > 0 ? last - 1 : 0);
  s.begin = a.window > 0 && first_pos >= a.window ? first_pos - a.window + 1 : 0;
  s.begin &= ~(kTile - 1);
  s.end = last_pos + 1 > s.begin ? last_pos + 1 : s.begin;
  return s;
}

// The page ids of 64 pages from `first`, one per lane.
struct PageIds {
  const int32_t* row;
  int max_pages, first, mine;
  __device__ __forceinline__ void load(int page) {
    first = page;
    const int p = page + (int)(threadIdx.x & 63);
    mine = p < max_pages ? row[p] : -1;
    // Wait here, where it is rare: left to the first use, the wait would
    // stand after the branch and hold up the tiles in flight every time.
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
  }
  // `page` is the same in all lanes
  __device__ __forceinline__ int at(int page) {
    if (page - first >= 64) load(page);
    return __builtin_amdgcn_readlane(mine, page - first);
  }
};

// This workgroup's token range of a row tile: `split` of `splits`, each of
// `chunk` tokens, longer where the request is longer than planned.
struct Range {
  int parts;       // ranges the row tile really has
  int begin, end;  // empty rows: begin == end
};

__device__ __forceinline__ Range range_of(const KvAttentionArgs& a, const Span& sp,
                                            int split) {
  Range r;
  const int splits = (int)a.splits.d;
  int per = (int)a.chunk.d;
  r.parts = a.chunk.of(sp.end - sp.begin + per - 1);
  if (r.parts > splits) {
    per = (a.splits.of(sp.end - sp.begin + splits - 1) + kTile - 1) / kTile * kTile;
    r.parts = (sp.end - sp.begin + per - 1) / per;
  }
  if (r.parts < 1) r.parts = 1;
  r.begin = sp.begin + split * per;
  r.end = r.begin + per < sp.end ? r.begin + per : sp.end;
  return r;
}

// Where a row tile's results go.
struct Output {
  uint16_t* o;
  int64_t o_token, o_head;
  float* lse;
  int tok0, head0, heads;  // head0: the first query head of the group
  Divisor group;

  __device__ __forceinline__ Output(const KvAttentionArgs& a, const Span& sp, int head)
      : o(a.o), o_token(a.o_token), o_head(a.o_head), lse(a.lse), tok0(sp.tok0),
        head0(head * (int)a.group.d), heads(a.Hq), group(a.group) {}

  // N (4 or 8) neighbouring channels of a row, each times inv and rounded.
  template <bool BF16, int N>
  __device__ __forceinline__ void store(int row, int ch, const float* x, float inv) const {
    const int i = group.of(row);
    uint16_t* dst = o + (int64_t)(tok0 + i) * o_token +
                    (int64_t)(head0 + row - i * (int)group.d) * o_head + ch;
    uint32_t w[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      if constexpr (BF16) {
        const __bf16 lo = (__bf16)(x[2 * k] * inv), hi = (__bf16)(x[2 * k + 1] * inv);
        w[k] = (uint32_t)__builtin_bit_cast(uint16_t, lo) |
               (uint32_t)__builtin_bit_cast(uint16_t, hi) << 16;
      } else {
        w[k] = pack_halves(x[2 * k] * inv, x[2 * k + 1] * inv);
      }
    }
    if constexpr (N == 4)
      *reinterpret_cast<uint2v*>(dst) = uint2v{w[0], w[1]};
    else
      *reinterpret_cast<uint4v*>(dst) = uint4v{w[0], w[1], w[2], w[3]};
  }

  __device__ __forceinline__ void store_lse(int row, float m, float l) const {
    if (!lse) return;
    const int i = group.of(row);
    lse[(int64_t)(tok0 + i) * heads + head0 + row - i * (int)group.d] =
        l == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
};

// Parts of a row tile in the workspace: per range and row, D channels and
// (m, l, 0, 0), in 16-byte vectors.
template <int D>
constexpr int kPartVecs = D / 4 + 1;

// After a workgroup of THREADS has stored its part: counts the arrival and
// says whether this was the row tile's last one.
__device__ __forceinline__ bool last_to_arrive(unsigned* counter, int parts, bool* s_last) {
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0)
    *s_last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
              (unsigned)(parts - 1);
  __syncthreads();
  return *s_last;
}

// One vector of a row over all parts, BATCH parts' loads in flight at once.
template <int BATCH>
__device__ __forceinline__ float4_t join_row(__amdgpu_buffer_rsrc_t all, int part_vecs,
                                             int parts, int at, int stat, float* m_out,
                                             float* l_out) {
  float m = kNone, l = 0.f;
  float4_t x = {0.f, 0.f, 0.f, 0.f};
  for (int o0 = 0; o0 < parts; o0 += BATCH) {
    float2_t ml[BATCH];
    float4_t y[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int o = o0 + k < parts ? o0 + k : parts - 1;
      ml[k] = load_coherent2(all, o * part_vecs + stat);
      y[k] = load_coherent(all, o * part_vecs + at);
    }
    float to = m;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) to = fmaxf(to, ml[k][0]);
    const float f = exp2_hw(m - to);
    x *= f;
    l *= f;
    m = to;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float w = o0 + k < parts ? exp2_hw(ml[k][0] - to) : 0.f;
      x += y[k] * w;
      l += ml[k][1] * w;
    }
  }
  *m_out = m;
  *l_out = l;
  return x;
}

// The last workgroup joins `rows` rows over all parts, in range order.
template <int D, bool BF16, int THREADS>
__device__ __forceinline__ void join_parts(const float* tile_base, int part_vecs, int parts,
                                           int rows, int row0, const Output& out,
                                           unsigned* counter) {
  constexpr int kVecs = D / 4;
  // One resource over all parts: the workspace is far smaller than 2 GiB.
  const __amdgpu_buffer_rsrc_t all = coherent_rsrc(tile_base);
  for (int v = threadIdx.x; v < rows * kVecs; v += THREADS) {
    const int row = v / kVecs, c = v % kVecs;
    const int at = row * kPartVecs<D> + c, stat = row * kPartVecs<D> + kVecs;
    float m, l;
    // (loads past the last part are loads again of the last: for few parts
    // most of a large batch would be)
    const float4_t x = parts <= 4 ? join_row<4>(all, part_vecs, parts, at, stat, &m, &l)
                                  : join_row<16>(all, part_vecs, parts, at, stat, &m, &l);
    const float y[4] = {x[0], x[1], x[2], x[3]};
    out.store<BF16, 4>(row0 + row, 4 * c, y, l == 0.f ? 0.f : 1.0f / l);
    if (c == 0) out.store_lse(row0 + row, m, l);
  }
  if (threadIdx.x == 0)  // ready for the next call
    __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Launches of the two kernels; D is 64, 128 or 256.
hipError_t launch_kv_tokens(const KvAttentionPlan& p, const KvAttentionArgs& a, int D, int dtype,
                            unsigned* counters, float* partials, hipStream_t stream);
hipError_t launch_kv_rows(const KvAttentionPlan& p, const KvAttentionArgs& a, int D, int dtype,
                          unsigned* counters, float* partials, hipStream_t stream);

}  // namespace w4a16
