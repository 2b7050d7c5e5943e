// Rotary positions (kv4_rope), the quantising append (kv4_append,
// kv4_rope_append) and the read-back (kv4_dequant_debug).
//
// One kernel does the first three.  A row (one token, one head) is D/8
// neighbouring lanes of a wave with eight channels each, one 16-byte load.
// A lane's partner channels of a rotation by halves sit rot/16 lanes away
// and come by lane exchange; minimum and maximum are reduced over the row's
// lanes; and a lane's eight codes are exactly one 32-bit word of the cache,
// so nothing is read back or merged.
//
// A workgroup takes `tokens` tokens and a range of their rows (query heads,
// then key heads, then value heads).  The angles of its tokens are computed
// once, in FP64 (a far position times a frequency needs more than FP32 to be
// reduced), and shared through LDS.
//
// What bounds it: HBM for prefills, the launch and one trip to memory for
// decode steps.  Rotation of 16384 x 32 rows of 128, 47 us (5.7 TB/s; 54 with
// temporal loads); 8192 tokens of 64 + 2 x 8 heads rotated and stored, 69 us (4.5);
// 4001 x 2 x 32 heads stored, 27 us (3.7: by the counters a wave issues 197
// vector instructions for its four rows, 49 thousand cycles per SIMD, 23 of
// the 27 us); 32 tokens, 4.0 us.
#include "../../include/w4a16_kv4.h"
#include "format.hpp"
#include "kv4.hpp"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokensLog = kKvAppendTokensLog, kMaxTokens = 1 << kMaxTokensLog;  // of a workgroup
constexpr float kFifteenth = 1.0f / 15.0f;
constexpr float kMaxHalf = 65504.0f;

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

template <bool BF16>
__device__ __forceinline__ float to_float(uint32_t bits16) {
  if constexpr (BF16) return __builtin_bit_cast(float, bits16 << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
}

template <bool BF16>
__device__ __forceinline__ uint32_t to_bits(float x) {
  if constexpr (BF16) {
    const __bf16 h = (__bf16)x;  // round half to even
    return __builtin_bit_cast(uint16_t, h);
  } else {
    const _Float16 h = (_Float16)x;
    return __builtin_bit_cast(uint16_t, h);
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4v& w, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = to_float<BF16>(w[i] & 0xffffu);
    x[2 * i + 1] = to_float<BF16>(w[i] >> 16);
  }
}

template <bool BF16>
__device__ __forceinline__ uint4v pack8(const float* x) {
  uint4v w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = to_bits<BF16>(x[2 * i]) | (to_bits<BF16>(x[2 * i + 1]) << 16);
  return w;
}

__device__ __forceinline__ bool finite(float x) {
  return (__builtin_bit_cast(uint32_t, x) & 0x7f800000u) != 0x7f800000u;
}

__device__ __forceinline__ int rope_axis(const RopeArgs& r, int i) {
  return (i >= r.n0) + (i >= r.n01);
}

// cos and sin of the angle of pair i at token t.  The angle is formed in
// radians, as the definition has it, and reduced in half turns; 1/pi as two
// numbers, so that the half turns of a far position keep their fraction.
__device__ __forceinline__ float2 rope_angle(const RopeArgs& r, int i, int t) {
  const double angle =
      (double)r.positions[rope_axis(r, i) * r.pos_stride + t] * r.inv_freq[i];
  constexpr double kInvPi = 0x1.45f306dc9c883p-2, kInvPiLow = -0x1.6b01ec5417056p-56;
  const double turns = angle * kInvPi;
  const double low = __builtin_fma(angle, kInvPi, -turns) + angle * kInvPiLow;
  double s, c;
  sincospi(turns - 2.0 * rint(0.5 * turns) + low, &s, &c);
  return make_float2((float)c, (float)s);
}

// Turns a lane's eight channels 8 j .. 8 j + 7 in place; cs holds the token's
// (cos, sin) by pair.  `w` are the lane's 16-bit inputs: the partner lane's
// are fetched as they are.
template <bool BF16>
__device__ __forceinline__ void rotate8(const RopeArgs& r, const float2* cs, int j,
                                        const uint4v& w, float* x) {
#pragma clang fp contract(off)
  const int rot8 = r.half / 4;  // lanes that turn
  if (r.pairs == KV4_ROPE_PAIRS) {
    if (j < rot8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = cs[4 * j + i];
        const float x1 = x[2 * i], x2 = x[2 * i + 1];
        x[2 * i] = x1 * a.x - x2 * a.y;
        x[2 * i + 1] = x2 * a.x + x1 * a.y;
      }
    }
    return;
  }
  const int half8 = rot8 / 2;
  const bool low = j < half8;
  const int lane = threadIdx.x & 63;
  const int partner = j >= rot8 ? lane : low ? lane + half8 : lane - half8;
  // x1 cos - x2 sin and x2 cos + x1 sin: the first's partner changes sign
  const uint32_t sign = low ? 0x80008000u : 0u;
  uint4v other;
#pragma unroll
  for (int i = 0; i < 4; ++i) other[i] = (uint32_t)__shfl((int)w[i], partner) ^ sign;
  if (j < rot8) {
    float y[8];
    unpack8<BF16>(other, y);
    const float2* a = cs + 8 * (low ? j : j - half8);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * a[i].x + y[i] * a[i].y;
  }
}

struct Quantised {
  uint32_t codes, params;
};

template <int CTRL>
__device__ __forceinline__ float other_lane(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// Reduction over a row's LANES lanes, all of which get the result.  Once
// lanes hold what their neighbours of a group of four hold, a mirrored lane
// is as good as an exchanged one.
template <int LANES, typename Op>
__device__ __forceinline__ float over_row(float x, Op op) {
  x = op(x, other_lane<0xb1>(x));   // quad_perm 1 0 3 2
  x = op(x, other_lane<0x4e>(x));   // quad_perm 2 3 0 1
  x = op(x, other_lane<0x141>(x));  // row_half_mirror: 8 lanes
  if constexpr (LANES >= 16) x = op(x, other_lane<0x140>(x));  // row_mirror: 16
  if constexpr (LANES >= 32) x = op(x, __shfl_xor(x, 16));
  return x;
}

// The stored form of a row, of which this lane holds eight channels.
template <int LANES>
__device__ __forceinline__ Quantised quantise8(const float* x) {
#pragma clang fp contract(off)
  // (these pass a NaN on, so that the row's ends tell of every channel)
  auto smaller = [](float a, float b) { return __builtin_elementwise_minimum(a, b); };
  auto larger = [](float a, float b) { return __builtin_elementwise_maximum(a, b); };
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = smaller(lo, x[i]);
    hi = larger(hi, x[i]);
  }
  lo = over_row<LANES>(lo, smaller);
  hi = over_row<LANES>(hi, larger);
  if (!finite(lo) || !finite(hi)) return {0x88888888u, 0x7e007e00u};  // code 8, NaN
  const _Float16 sh = (_Float16)fminf((hi - lo) * kFifteenth, kMaxHalf);
  const float s = (float)sh;
  const _Float16 zh = (_Float16)fminf(fmaxf(lo + 8.0f * s, -kMaxHalf), kMaxHalf);
  const float z = (float)zh;
  const float inv = s > 0.f ? 1.0f / s : 0.f;
  // Adding 1.5 2^23 rounds to an integer (half to even: the added number is
  // even, and so is 8) and leaves it in the low bits; what that number's own
  // bits add to the codes is one constant.
  constexpr float kRound = 12582912.0f + 8.0f;
  constexpr uint32_t kRoundBits = 0x4b400000u;
  uint32_t codes = 0u - kRoundBits * 0x11111111u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = __builtin_amdgcn_fmed3f((x[i] - z) * inv + kRound, kRound - 8.0f,
                                            kRound + 7.0f);
    codes += __builtin_bit_cast(uint32_t, q) << (4 * i);
  }
  return {codes, (uint32_t)__builtin_bit_cast(uint16_t, sh) |
                     (uint32_t)__builtin_bit_cast(uint16_t, zh) << 16};
}

// Grid: x = groups of 1 << tokens_log tokens, y = shares of the Hq + 2 H rows
// of a token.
template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppendArgs a, int tokens_log,
                                                             int page_log) {
  constexpr int LANES = D / 8, ROWS = kThreads / LANES;
  __shared__ float2 cs[kMaxTokens][D / 2];
  const int t0 = blockIdx.x << tokens_log;
  const int nt = a.T - t0 < 1 << tokens_log ? a.T - t0 : 1 << tokens_log;
  const int half = a.rope.half;
  const int j = threadIdx.x % LANES;
  // Rows in (head, token) order, so that neighbouring tokens of a head, whose
  // words lie side by side in the cache, are stored together.  Whole waves
  // leave the loop together and read a clamped row where there is none: the
  // lane exchanges need every lane.
  const int rows = (a.Hq + 2 * a.H) << tokens_log;
  struct Row {
    int head, tt, slot;
    uint4v w;
  };
  auto load = [&](int base) {
    Row r;
    int row = base + (int)threadIdx.x / LANES;
    row = row < rows ? row : rows - 1;
    r.head = row >> tokens_log;
    r.tt = row & ((1 << tokens_log) - 1);
    const int t = t0 + (r.tt < nt ? r.tt : nt - 1);
    const bool is_q = r.head < a.Hq, is_k = r.head < a.Hq + a.H;
    const Rows& src = is_q ? a.q : is_k ? a.k : a.v;
    const int h = r.head - (is_q ? 0 : is_k ? a.Hq : a.Hq + a.H);
    r.w = __builtin_nontemporal_load(  // read once
        reinterpret_cast<const uint4v*>(src.p + t * src.token + h * src.head + 8 * j));
    r.slot = is_q ? -1 : a.slots[t];
    return r;
  };
  int base = blockIdx.y * ROWS;
  if (base >= rows) return;
  Row next = load(base);  // under way while the angles are computed
  if (half) {
    for (int i = threadIdx.x; i < nt * half; i += kThreads)
      cs[i / half][i % half] = rope_angle(a.rope, i % half, t0 + i / half);
    __syncthreads();
  }
  for (; base < rows; base += gridDim.y * ROWS) {
    const Row r = next;
    next = load(base + gridDim.y * ROWS);
    const bool live = base + (int)threadIdx.x / LANES < rows && r.tt < nt;
    const bool is_q = r.head < a.Hq, is_k = !is_q && r.head < a.Hq + a.H;
    float x[8];
    unpack8<BF16>(r.w, x);
    if (half && __any(is_q || is_k)) {
      float turned[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) turned[i] = x[i];
      rotate8<BF16>(a.rope, cs[r.tt < nt ? r.tt : nt - 1], j, r.w, turned);
      if (is_q || is_k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = turned[i];
      }
    }
    if (live && is_q)
      *reinterpret_cast<uint4v*>(a.qo + (t0 + r.tt) * a.qo_token + r.head * a.qo_head + 8 * j) =
          pack8<BF16>(x);
    if (!__any(!is_q)) continue;
    const Quantised c = quantise8<LANES>(x);
    if (!live || is_q || r.slot < 0 || r.slot >= a.pages << page_log) continue;
    const int h = r.head - (is_k ? a.Hq : a.Hq + a.H);
    const int at = r.slot & (a.page - 1), u = at % kKvUnit;
    uint8_t* unit = a.cache + kv_unit_offset<D>(r.slot >> page_log, a.H, h, a.page, at);
    uint32_t* codes = reinterpret_cast<uint32_t*>(unit + (is_k ? 0 : KvUnit<D>::values));
    codes[is_k ? u * LANES + j : (u / 4 * LANES + j) * 4 + u % 4] = c.codes;
    if (j == 0)
      reinterpret_cast<uint32_t*>(
          unit + (is_k ? KvUnit<D>::key_params : KvUnit<D>::value_params))[u] = c.params;
  }
}

template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void kv_dequant_kernel(
    const int32_t* __restrict__ slots, const uint8_t* __restrict__ cache,
    uint16_t* __restrict__ K, uint16_t* __restrict__ V, int T, int H, int pages, int page) {
  constexpr int LANES = D / 8, ROWS = kThreads / LANES;
  const int j = threadIdx.x % LANES;
  const int64_t rows = 2 * (int64_t)T * H;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; row < rows;
       row += (int64_t)gridDim.x * ROWS) {
    const bool is_k = row < (int64_t)T * H;
    const int64_t th = is_k ? row : row - (int64_t)T * H;
    const int t = (int)(th / H), h = (int)(th % H);
    const int slot = slots[t];
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot >= 0 && slot < pages * page) {
      const int at = slot % page, r = at % kKvUnit;
      const uint8_t* unit = cache + kv_unit_offset<D>(slot / page, H, h, page, at);
      const uint32_t c = reinterpret_cast<const uint32_t*>(
          unit + (is_k ? 0 : KvUnit<D>::values))[is_k ? r * LANES + j
                                                      : (r / 4 * LANES + j) * 4 + r % 4];
      const uint32_t p = reinterpret_cast<const uint32_t*>(
          unit + (is_k ? KvUnit<D>::key_params : KvUnit<D>::value_params))[r];
      const float s = to_float<false>(p & 0xffffu), z = to_float<false>(p >> 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (float)((int)(c >> (4 * i) & 15u) - 8) * s + z;
    }
    *reinterpret_cast<uint4v*>((is_k ? K : V) + th * D + 8 * j) = pack8<BF16>(x);
  }
}

template <int D, bool BF16>
hipError_t append(const KvAppendArgs& a, hipStream_t stream) {
  constexpr int ROWS = kThreads / (D / 8);
  // Few tokens: one per workgroup, its rows shared out, so that every row
  // is under way at once; many: four per workgroup, which share no angles
  // but fill the threads that compute them.
  const int tokens_log = a.T >= 1024 ? kMaxTokensLog : 0;
  const int page_log = a.page > 0 ? 31 - __builtin_clz((unsigned)a.page) : 0;
  const int groups = (a.T + (1 << tokens_log) - 1) >> tokens_log;
  const int rows = (a.Hq + 2 * a.H) << tokens_log;
  int shares = (rows + ROWS - 1) / ROWS;
  const int enough = (2048 + groups - 1) / groups;
  if (shares > enough) shares = enough;
  if (shares > 65535) shares = 65535;
  hipLaunchKernelGGL((kv_append_kernel<D, BF16>), dim3(groups, shares), dim3(kThreads), 0, stream,
                     a, tokens_log, page_log);
  return hipGetLastError();
}

template <int D, bool BF16>
hipError_t dequant(const int32_t* slots, const uint8_t* cache, uint16_t* K, uint16_t* V, int T,
                   int H, int pages, int page, hipStream_t stream) {
  constexpr int ROWS = kThreads / (D / 8);
  int64_t groups = (2 * (int64_t)T * H + ROWS - 1) / ROWS;
  if (groups > 8192) groups = 8192;
  hipLaunchKernelGGL((kv_dequant_kernel<D, BF16>), dim3((unsigned)groups), dim3(kThreads), 0,
                     stream, slots, cache, K, V, T, H, pages, page);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, int D, int dtype, hipStream_t stream) {
  const bool bf = dtype == W4A16_DTYPE_BF16;
  switch (D) {
    case 64: return bf ? append<64, true>(a, stream) : append<64, false>(a, stream);
    case 128: return bf ? append<128, true>(a, stream) : append<128, false>(a, stream);
    default: return bf ? append<256, true>(a, stream) : append<256, false>(a, stream);
  }
}

hipError_t launch_kv_dequant(const int32_t* slots, const uint8_t* cache, uint16_t* K,
                             uint16_t* V, int T, int H, int D, int pages, int page, int dtype,
                             hipStream_t stream) {
  const bool bf = dtype == W4A16_DTYPE_BF16;
#define W4A16_DEQ(d)                                                                   \
  return bf ? dequant<d, true>(slots, cache, K, V, T, H, pages, page, stream)          \
            : dequant<d, false>(slots, cache, K, V, T, H, pages, page, stream)
  switch (D) {
    case 64: W4A16_DEQ(64);
    case 128: W4A16_DEQ(128);
    default: W4A16_DEQ(256);
  }
#undef W4A16_DEQ
}

}  // namespace w4a16
