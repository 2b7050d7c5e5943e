// Routing to experts: scores and the best k (moe_route), rows sorted by
// expert (moe_tables) and the weighted sum over a token's rows (moe_combine).
#include <type_traits>

#include "moe.hpp"
#include "product.hpp"
#include "tables_plan.hpp"
#include "w4a16_moe.h"

namespace w4a16 {
namespace {

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t at) {
  if (a.type == MOE_LOGITS_F32) return static_cast<const float*>(a.logits)[at];
  return scale16(static_cast<const uint16_t*>(a.logits)[at], a.type == MOE_LOGITS_BF16);
}

// ---------------------------------------------------------------------------
// choices
// ---------------------------------------------------------------------------
//
// What experts (and groups) are compared by, in three forms:
//   uint32_t  16-bit logits in their own order: 16 bits that order as the
//             logits do above 16 that fall with the index, so that one maximum
//             of whole numbers is the choice, ties included
//   float     FP32 logits in their own order, with the index beside them
//   double    c in 64 bits, so that rounding turns no order
// none<V>() is no choice; a lane's i-th value has the index lane + L i.

// Tokens from which 16 lanes take one.  Packed, 128 experts: 4.4 us with 64
// lanes and 4.6 with 16 at 4096 tokens, 9.7 and 5.9 at 16384.  Up to 16 experts
// they always do (8 experts: 2.7 and 2.3 us at 48 tokens).
constexpr int kNarrowFrom = 4096;

template <typename V>
__device__ __forceinline__ V none() {
  return -(V)__builtin_inf();
}
template <>
__device__ __forceinline__ uint32_t none<uint32_t>() {
  return 0;
}

// The packed form of a 16-bit logit that is neither NaN nor -infinity.
__device__ __forceinline__ uint32_t packed(uint16_t logit, int index) {
  uint32_t u = logit == 0x8000 ? 0 : logit;  // -0 is 0
  u = u & 0x8000 ? ~u & 0xffff : u | 0x8000;
  return u << 16 | (uint32_t)(0xffff - index);
}

// The value of another lane: CTRL a lane pattern within 16, d a distance.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, x)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint64_t lo = dpp<CTRL>((uint32_t)u), hi = dpp<CTRL>((uint32_t)(u >> 32));
  return __builtin_bit_cast(double, hi << 32 | lo);
}

// The pair (x of this lane's row or half, x of the other one's) in either order,
// rows of 16 lanes swapped for D = 16, halves of 32 for D = 32.
template <int D>
__device__ __forceinline__ void both_sides(uint32_t x, uint32_t& p, uint32_t& q) {
  if constexpr (D == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    p = r[0];
    q = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    p = r[0];
    q = r[1];
  }
}
template <int D>
__device__ __forceinline__ void both_sides(float x, float& p, float& q) {
  uint32_t a, b;
  both_sides<D>(__builtin_bit_cast(uint32_t, x), a, b);
  p = __builtin_bit_cast(float, a);
  q = __builtin_bit_cast(float, b);
}
template <int D>
__device__ __forceinline__ void both_sides(double x, double& p, double& q) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  uint32_t a, b, c, d;
  both_sides<D>((uint32_t)u, a, b);
  both_sides<D>((uint32_t)(u >> 32), c, d);
  p = __builtin_bit_cast(double, (uint64_t)c << 32 | a);
  q = __builtin_bit_cast(double, (uint64_t)d << 32 | b);
}

// x = join(x, y) over the L lanes of a token (16 or 64), the result in all of
// them: neighbours, pairs, mirrored halves of 8 and of 16; then rows.
template <int L, typename T, typename Join>
__device__ __forceinline__ T over_lanes(T x, Join join) {
  x = join(x, dpp<0xB1>(x));
  x = join(x, dpp<0x4E>(x));
  x = join(x, dpp<0x141>(x));
  x = join(x, dpp<0x140>(x));
  if constexpr (L == 64) {
    T p, q;
    both_sides<16>(x, p, q);
    x = join(p, q);
    both_sides<32>(x, p, q);
    x = join(p, q);
  }
  return x;
}

// The best of the lanes' (value, index): the larger value, at equal values the
// lower index.
template <typename V>
__device__ __forceinline__ void better_of(V& v, int& i, V ov, int oi) {
  const bool better = ov > v || (ov == v && oi < i);
  v = better ? ov : v;
  i = better ? oi : i;
}
// Whole numbers that order as floats do (no NaN, no -0), and as doubles do but
// for ties in their upper halves.
__device__ __forceinline__ uint32_t upper_key(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t upper_key(double v) {
  const uint32_t u = (uint32_t)(__builtin_bit_cast(uint64_t, v) >> 32);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_lane(float v, int l) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ double from_lane(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, hi << 32 | lo);
}

// A wave that has one token takes the largest key first; only where several
// indices have it the values and indices themselves are joined (48 tokens, 256
// experts in 8 groups: 10.4 us with every join of 64 bits,
// 7.4 so, with chosen scores kept and the bias loaded beside the logits).
template <int L, typename V>
__device__ __forceinline__ void best_over_lanes(V& v, int& i) {
  if constexpr (std::is_same<V, uint32_t>::value) {
    v = over_lanes<L>(v, [](uint32_t p, uint32_t q) { return q > p ? q : p; });
    i = 0xffff - (int)(v & 0xffff);
  } else {
    if constexpr (L == 64) {
      const uint32_t key = upper_key(v);
      const uint64_t on = __ballot(
          key == over_lanes<L>(key, [](uint32_t p, uint32_t q) { return q > p ? q : p; }));
      const int l = __builtin_ctzll(on), first = __builtin_amdgcn_readlane(i, l);
      if ((on & ~__ballot(i == first)) == 0) {
        v = from_lane(v, l);
        i = first;
        return;
      }
    }
    better_of(v, i, dpp<0xB1>(v), (int)dpp<0xB1>((uint32_t)i));
    better_of(v, i, dpp<0x4E>(v), (int)dpp<0x4E>((uint32_t)i));
    better_of(v, i, dpp<0x141>(v), (int)dpp<0x141>((uint32_t)i));
    better_of(v, i, dpp<0x140>(v), (int)dpp<0x140>((uint32_t)i));
    if constexpr (L == 64) {
      V w;
      uint32_t p, q;
      both_sides<16>((uint32_t)i, p, q);
      both_sides<16>(v, v, w);
      i = (int)p;
      better_of(v, i, w, (int)q);
      both_sides<32>((uint32_t)i, p, q);
      both_sides<32>(v, v, w);
      i = (int)p;
      better_of(v, i, w, (int)q);
    }
  }
}

template <typename T>
__device__ __forceinline__ T sum_of(T x, T y) {
  return x + y;
}

// The numerator of an eligible expert's score.  Sigmoid takes it in 64 bits
// only: in 32 the exponential of x < -88.7 overflows and the score is 0, also
// where all chosen ones are of that size and renorm divides them by their sum
// (without a bias, in 32 and 64 bits: 48 tokens, 256 experts 3.8 and 4.3 us;
// 16384 tokens, 128 experts 5.4 and 5.7).  A softmax that is taken in 32 bits
// has 1 among the chosen, so what is lost beside it is below 2^-126.
template <typename F>
__device__ __forceinline__ F numerator(const RouteArgs& a, float x, float top) {
  if constexpr (sizeof(F) == 8)
    if (a.score == MOE_SIGMOID) return 1.0 / (1.0 + exp(-(double)x));
  if (top == __builtin_inff()) return x == top ? (F)1 : (F)0;
  if constexpr (sizeof(F) == 8)
    return exp((double)x - (double)top);
  else
    return expf(x - top);
}

// L lanes a token (64 / L tokens a wave), lane l of them with experts l + L i.
// V: what choices are compared as; scores are 64 bits beside double.
//
// What bounds it: instructions; each of the k choices looks at the lane's
// experts again and joins the lanes.  16 lanes a token share the joining among
// four tokens, 64 find one token's choices sooner.
template <typename V, int L, int P>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a) {
  constexpr bool kPacked = std::is_same<V, uint32_t>::value;
  typedef typename std::conditional<std::is_same<V, double>::value, double, float>::type F;
  constexpr bool kKeep = std::is_same<V, double>::value;
  constexpr int TOKENS = 256 / L;
  __shared__ V marks[TOKENS][L * P];
  const int lane = threadIdx.x & (L - 1), slot = threadIdx.x / L;
  const int t = blockIdx.x * TOKENS + slot;
  const bool live = t < a.T;
  const int64_t row = (int64_t)(live ? t : a.T - 1) * a.row;
  const float inf = __builtin_inff();

  float x[P];
  V c[P];
  float b[std::is_same<V, double>::value ? P : 1];  // loaded with the logits: one trip
  float top = -inf;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + L * i;
    if constexpr (kPacked) {
      const uint16_t h = e < a.E ? static_cast<const uint16_t*>(a.logits)[row + e] : 0;
      x[i] = e < a.E ? scale16(h, a.type == MOE_LOGITS_BF16) : -inf;
      c[i] = x[i] > -inf ? packed(h, e) : none<V>();
    } else {
      x[i] = e < a.E ? load_logit(a, row + e) : -inf;
      if constexpr (sizeof(V) == 8) b[i] = a.bias && e < a.E ? a.bias[e] : 0.f;
    }
    top = x[i] > top ? x[i] : top;  // NaN: not above
  }
  top = over_lanes<L>(top, [](float p, float q) { return q > p ? q : p; });
  F sum = 1;  // softmax: the scores' denominator
  F s[kKeep ? P : 1];  // the scores' numerators
  const bool softmax = a.score == MOE_SOFTMAX;
  if constexpr (std::is_same<V, double>::value) {
    F own = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      s[i] = x[i] > -inf ? numerator<F>(a, x[i], top) : 0;
      own += s[i];
    }
    if (softmax) sum = over_lanes<L>(own, sum_of<F>);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const F v = (softmax ? s[i] / sum : s[i]) + (F)b[i];
      c[i] = x[i] > -inf && v > none<V>() ? v : none<V>();
    }
  } else {
    if (softmax && !a.renorm) {
      F own = 0;
#pragma unroll
      for (int i = 0; i < P; ++i) own += x[i] > -inf ? numerator<F>(a, x[i], top) : 0;
      sum = over_lanes<L>(own, sum_of<F>);
    }
    if constexpr (!kPacked)
#pragma unroll
      for (int i = 0; i < P; ++i) c[i] = x[i] > none<V>() ? x[i] + 0.f : none<V>();  // -0 is 0
  }

  if (a.groups > 1) {
    // marks by `share` lanes a group, then the best groups one by one
    const int size = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < P; ++i) marks[slot][lane + L * i] = c[i];
    __syncthreads();
    int share = 1;
    while (2 * share * a.groups <= L) share *= 2;
    constexpr int MOST = MOE_MAX_GROUPS / L;
    V mark[MOST];
    const int own = lane / share;  // this lane's group, and own + L m
#pragma unroll
    for (int m = 0; m < MOST; ++m) {
      const int g = own + L * m;
      V first = none<V>(), second = none<V>();
      if (g < a.groups)
#pragma unroll 4
        for (int j = lane & (share - 1); j < size; j += share) {
          const V v = marks[slot][g * size + j];
          second = v > first ? first : v > second ? v : second;
          first = v > first ? v : first;
        }
      // lanes join as in over_lanes: what was joined before is alike in them
      auto join = [&](V f, V s) {
        const V least = f > first ? first : f;
        second = s > second ? s : second;
        second = least > second ? least : second;
        first = f > first ? f : first;
      };
      if (share > 1) join(dpp<0xB1>(first), dpp<0xB1>(second));
      if (share > 2) join(dpp<0x4E>(first), dpp<0x4E>(second));
      if (share > 4) join(dpp<0x141>(first), dpp<0x141>(second));
      if (share > 8) join(dpp<0x140>(first), dpp<0x140>(second));
      if constexpr (L == 64) {
        V f, s;
        if (share > 16) {
          both_sides<16>(first, first, f);
          both_sides<16>(second, second, s);
          join(f, s);
        }
      }
      if constexpr (kPacked)
        mark[m] = first ? (first & 0xffff0000u) | (0xffffu - g) : 0;
      else
        mark[m] = a.group_best == 2 && second > none<V>() ? first + second : first;
    }
    uint64_t keep = 0;
    for (int n = 0; n < a.top_groups; ++n) {
      V best = mark[0];
      int at = own;
#pragma unroll
      for (int m = 1; m < MOST; ++m) {
        at = mark[m] > best ? own + L * m : at;
        best = mark[m] > best ? mark[m] : best;
      }
      best_over_lanes<L>(best, at);
      if (!(best > none<V>())) at = -1;
      if (at >= 0) keep |= 1ull << at;
#pragma unroll
      for (int m = 0; m < MOST; ++m) mark[m] = at == own + L * m ? none<V>() : mark[m];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane + L * i;
      c[i] = e < a.E && ((keep >> (e / size)) & 1) ? c[i] : none<V>();
    }
  }

  constexpr int MINE = MOE_MAX_TOP / L > 0 ? MOE_MAX_TOP / L : 1;
  int mine[MINE];  // lane l: choices l, l + L
  F kept = 0;      // kKeep, L = 64: the score of mine[0]
#pragma unroll
  for (int m = 0; m < MINE; ++m) mine[m] = -1;
  for (int j = 0; j < a.k; ++j) {
    V best = c[0];
    int at = lane;
#pragma unroll
    for (int i = 1; i < P; ++i) {
      at = c[i] > best ? lane + L * i : at;
      best = c[i] > best ? c[i] : best;
    }
    best_over_lanes<L>(best, at);
    if (!(best > none<V>())) at = -1;
#pragma unroll
    for (int m = 0; m < MINE; ++m) mine[m] = lane + L * m == j ? at : mine[m];
    if constexpr (kKeep && L == 64) {
      // its score from the lane that has it: cheaper than once more a trip for
      // the logit and an exponential
      const int chosen = __builtin_amdgcn_readfirstlane(at);
      F of = s[0];
#pragma unroll
      for (int i = 1; i < P; ++i) of = chosen / L == i ? s[i] : of;
      of = from_lane(of, chosen & (L - 1));
      kept = lane == j && chosen >= 0 ? of : kept;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] = at == lane + L * i ? none<V>() : c[i];
  }

  // S: what the weights are computed in
  auto finish = [&](auto zero) {
    typedef decltype(zero) S;
    S score[MINE], total = 0, denominator = (S)sum;
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      if constexpr (kKeep && L == 64)
        score[m] = kept;
      else
        score[m] = mine[m] >= 0 ? numerator<S>(a, load_logit(a, row + mine[m]), top) : (S)0;
      total += score[m];
    }
    if (a.renorm) denominator = over_lanes<L>(total, sum_of<S>);
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      const int j = lane + L * m;
      if (live && j < a.k) {
        a.ids[(int64_t)t * a.k + j] = mine[m];
        a.weights[(int64_t)t * a.k + j] =
            mine[m] < 0 || !(denominator > 0) ? 0.f : (float)(score[m] / denominator) * a.scale;
      }
    }
  };
  if (softmax)
    finish((F)0);
  else
    finish(0.0);
}

// ---------------------------------------------------------------------------
// tables
// ---------------------------------------------------------------------------
//
// A stable counting sort.  Up to kTablesOneLaunch choices every workgroup counts all
// choices of each expert, and those before its own chunk, for itself, so that
// none waits for another, and then places its chunk.  Beyond, counting
// everything in every workgroup costs more than launches (128 experts: 5.4 us
// against 8.3 at 8192 choices, 27 against 12 at 131072): the chunks' counts are
// made by one launch and kept in `order`, the second sums them and writes
// `where`, the third `order`.

constexpr int kTableWaves = kTableThreads / 64;
static_assert(MOE_MAX_EXPERTS <= kTableThreads, "one thread an expert");

// counts[e] of ids[begin .. end), by all threads; `early` those before `border`.
__device__ __forceinline__ void count_ids(const TablesArgs& a, int begin, int end, int* counts,
                                          int border, int* early) {
  constexpr int U = 4;
  for (int at = begin + (int)threadIdx.x; at < end; at += U * kTableThreads) {
    unsigned e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = at + u * kTableThreads;
      e[u] = i < end ? (unsigned)a.ids[i] : ~0u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e[u] < (unsigned)a.E) {
        atomicAdd(&counts[e[u]], 1);
        if (early && at + u * kTableThreads < border) atomicAdd(&early[e[u]], 1);
      }
  }
}

// Exclusive sum over the threads, and the whole sum.
__device__ __forceinline__ int sum_before(int n, int* wave_sum, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = n;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) wave_sum[wave] = x;
  __syncthreads();
  int base = 0, all = 0;
  for (int w = 0; w < kTableWaves; ++w) {
    base += w < wave ? wave_sum[w] : 0;
    all += wave_sum[w];
  }
  *total = all;
  return base + x - n;
}

// Places ids[begin .. end): ahead[e] is where the first of expert e goes.
template <bool ORDER>
__device__ __forceinline__ void place_ids(const TablesArgs& a, int begin, int end, int* ahead,
                                          int* in_wave) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int at = begin; at < end; at += kTableThreads) {
    __syncthreads();
    for (int i = tid; i < kTableWaves * a.E; i += kTableThreads) in_wave[i] = 0;
    __syncthreads();
    const int i = at + tid;
    unsigned e = i < end ? (unsigned)a.ids[i] : ~0u;
    if (e >= (unsigned)a.E) e = a.E;
    // lanes of the same expert
    uint64_t same = __ballot(e < (unsigned)a.E);
    for (int bit = 0; (1 << bit) <= a.E; ++bit) {
      const bool on = (e >> bit) & 1;
      const uint64_t with = __ballot(on);
      same &= on ? with : ~with;
    }
    const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
    if (e < (unsigned)a.E && rank == 0) in_wave[wave * a.E + e] = __builtin_popcountll(same);
    __syncthreads();
    if (i < end) {
      int pos = -1;
      if (e < (unsigned)a.E) {
        pos = ahead[e] + rank;
#pragma unroll
        for (int w = 0; w < kTableWaves - 1; ++w) pos += w < wave ? in_wave[w * a.E + e] : 0;
        if constexpr (ORDER) a.order[pos] = i;
      }
      a.where[i] = pos;
    }
    if (at + kTableThreads >= end) break;
    __syncthreads();
    if (tid < a.E)
      for (int w = 0; w < kTableWaves; ++w) ahead[tid] += in_wave[w * a.E + tid];
  }
}

__global__ __launch_bounds__(kTableThreads) void moe_tables_kernel(TablesArgs a, int chunk) {
  extern __shared__ int lds[];
  int* const all = lds;              // [E]: choices of the expert
  int* const ahead = all + a.E;      // [E]: those before this chunk
  int* const in_wave = ahead + a.E;  // [waves][E]
  __shared__ int wave_sum[kTableWaves];
  const int tid = threadIdx.x;
  const int begin = blockIdx.x * chunk, end = begin + chunk < a.n ? begin + chunk : a.n;
  for (int i = tid; i < 2 * a.E; i += kTableThreads) all[i] = 0;
  __syncthreads();
  count_ids(a, 0, a.n, all, begin, begin > 0 ? ahead : nullptr);
  __syncthreads();
  int total;
  const int base = sum_before(tid < a.E ? all[tid] : 0, wave_sum, &total);
  if (tid < a.E) {
    ahead[tid] += base;
    if (blockIdx.x == 0) {
      a.starts[tid] = base;
      if (tid == a.E - 1) a.starts[a.E] = total;
    }
  }
  // positions behind the last kept choice
  for (int i = begin + tid; i < end; i += kTableThreads)
    if (i >= total) a.order[i] = -1;
  place_ids<true>(a, begin, end, ahead, in_wave);
}

// counts [chunks][E]
__global__ __launch_bounds__(kTableThreads) void moe_count_kernel(TablesArgs a, int chunk,
                                                                  int* __restrict__ counts) {
  extern __shared__ int lds[];
  const int tid = threadIdx.x;
  const int begin = blockIdx.x * chunk, end = begin + chunk < a.n ? begin + chunk : a.n;
  for (int i = tid; i < a.E; i += kTableThreads) lds[i] = 0;
  __syncthreads();
  count_ids(a, begin, end, lds, 0, nullptr);
  __syncthreads();
  for (int i = tid; i < a.E; i += kTableThreads) counts[(int64_t)blockIdx.x * a.E + i] = lds[i];
}

__global__ __launch_bounds__(kTableThreads) void moe_where_kernel(TablesArgs a, int chunk,
                                                                  const int* __restrict__ counts) {
  extern __shared__ int lds[];
  int* const all = lds;
  int* const ahead = all + a.E;
  int* const in_wave = ahead + a.E;
  __shared__ int wave_sum[kTableWaves];
  const int tid = threadIdx.x;
  const int begin = blockIdx.x * chunk, end = begin + chunk < a.n ? begin + chunk : a.n;
  for (int i = tid; i < 2 * a.E; i += kTableThreads) all[i] = 0;
  __syncthreads();
  // several threads an expert, each a share of the chunks
  const int shares = kTableThreads / a.E;
  const int e = tid % a.E, share = tid / a.E;
  if (share < shares) {
    int n = 0, early = 0;
    constexpr int U = 8;  // loads at once
    for (int c0 = share; c0 < (int)gridDim.x; c0 += U * shares) {
      int v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * shares;
        v[u] = c < (int)gridDim.x ? counts[(int64_t)c * a.E + e] : 0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        n += v[u];
        early += c0 + u * shares < (int)blockIdx.x ? v[u] : 0;
      }
    }
    atomicAdd(&all[e], n);
    atomicAdd(&ahead[e], early);
  }
  __syncthreads();
  int total;
  const int base = sum_before(tid < a.E ? all[tid] : 0, wave_sum, &total);
  if (tid < a.E) {
    ahead[tid] += base;
    if (blockIdx.x == 0) {
      a.starts[tid] = base;
      if (tid == a.E - 1) a.starts[a.E] = total;
    }
  }
  place_ids<false>(a, begin, end, ahead, in_wave);
}

__global__ __launch_bounds__(256) void moe_order_kernel(TablesArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.n) return;
  const int p = a.where[i];
  if ((unsigned)p < (unsigned)a.n) a.order[p] = i;
  if (i >= a.starts[a.E]) a.order[i] = -1;
}

// Eight columns a thread; the rows of eight choices are loaded before any of
// them is added.
//
// What bounds it: bandwidth, the rows' way in; for few tokens the two trips,
// one for the positions and one for the rows.
template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_kernel(CombineArgs a) {
  const int t = blockIdx.y + blockIdx.z * gridDim.y;
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (t >= a.T || c >= a.N) return;
  constexpr int U = 8;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < a.k; j0 += U) {
    int at[U];
    float w[U];
    uint4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = (int64_t)t * a.k + (j0 + j < a.k ? j0 + j : a.k - 1);
      at[j] = a.where[i];
      w[j] = a.weights[i];
      if (j0 + j >= a.k) at[j] = -1;
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
      if ((unsigned)at[j] < (unsigned)a.rows)
        v[j] = *reinterpret_cast<const uint4*>(a.Y + (int64_t)at[j] * a.N + c);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if ((unsigned)at[j] >= (unsigned)a.rows) continue;
      const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = __builtin_fmaf(w[j], scale16((uint16_t)(u[i / 2] >> (16 * (i & 1))), BF16), x[i]);
    }
  }
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = round16(x[2 * i], BF16) | ((uint32_t)round16(x[2 * i + 1], BF16) << 16);
  *reinterpret_cast<uint4*>(a.out + (int64_t)t * a.N + c) = uint4{u[0], u[1], u[2], u[3]};
}

template <typename V>
hipError_t route(const RouteArgs& a, hipStream_t stream) {
  const dim3 block(256);
  const dim3 wide((a.T + 3) / 4), narrow((a.T + 15) / 16);
#define MOE_ROUTE(L, P, GRID)                                                        \
  do {                                                                               \
    hipLaunchKernelGGL((moe_route_kernel<V, L, P>), GRID, block, 0, stream, a);      \
    return hipGetLastError();                                                        \
  } while (0)
  if (a.E <= 16 && a.k <= 16) MOE_ROUTE(16, 1, narrow);
  if (a.T >= kNarrowFrom && a.E <= 256) {
    if (a.E <= 64) MOE_ROUTE(16, 4, narrow);
    if (a.E <= 128) MOE_ROUTE(16, 8, narrow);
    MOE_ROUTE(16, 16, narrow);
  }
  if (a.E <= 64) MOE_ROUTE(64, 1, wide);
  if (a.E <= 128) MOE_ROUTE(64, 2, wide);
  if (a.E <= 256) MOE_ROUTE(64, 4, wide);
  if (a.E <= 512) MOE_ROUTE(64, 8, wide);
  MOE_ROUTE(64, 16, wide);
#undef MOE_ROUTE
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  const bool by_logit = !a.bias && (a.groups == 1 || a.group_best == 1);
  if (!by_logit) return route<double>(a, stream);
  return a.type == MOE_LOGITS_F32 ? route<float>(a, stream) : route<uint32_t>(a, stream);
}

hipError_t launch_moe_tables(const TablesArgs& a, hipStream_t stream) {
  const bool one = a.n <= kTablesOneLaunch;
  const int chunk = table_chunk(a.n, a.E);
  const dim3 groups(table_groups(a.n, chunk)), block(kTableThreads);
  const size_t bytes = (size_t)(2 + kTableWaves) * a.E * sizeof(int);
  if (bytes > 60 * 1024) {
    const hipError_t e = hipFuncSetAttribute(
        one ? reinterpret_cast<const void*>(moe_tables_kernel)
            : reinterpret_cast<const void*>(moe_where_kernel),
        hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != hipSuccess) return e;
  }
  if (one) {
    hipLaunchKernelGGL(moe_tables_kernel, groups, block, bytes, stream, a, chunk);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(moe_count_kernel, groups, block, a.E * sizeof(int), stream, a, chunk, a.order);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_where_kernel, groups, block, bytes, stream, a, chunk, a.order);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_order_kernel, dim3((a.n + 255) / 256), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t stream) {
  const int y = a.T < 32768 ? a.T : 32768;
  const dim3 grid((a.N / 8 + 255) / 256, y, (a.T + y - 1) / y);
  if (a.dtype == W4A16_DTYPE_BF16)
    hipLaunchKernelGGL((moe_combine_kernel<true>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((moe_combine_kernel<false>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace w4a16
