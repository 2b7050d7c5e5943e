// Routing to experts: scores and the best k (moe_route), rows sorted by
// expert (moe_tables) and the weighted sum over a token's rows (moe_combine).
#include "moe.hpp"
#include "product.hpp"
#include "w4a16_moe.h"

namespace w4a16 {
namespace {

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t at) {
  if (a.type == MOE_LOGITS_F32) return static_cast<const float*>(a.logits)[at];
  return scale16(static_cast<const uint16_t*>(a.logits)[at], a.type == MOE_LOGITS_BF16);
}

__device__ __forceinline__ float lowest(float) { return -__builtin_inff(); }
__device__ __forceinline__ double lowest(double) { return -__builtin_inf(); }

// Whether (x, i) comes before (y, j): the larger value, at equal values the
// lower index.
template <typename V>
__device__ __forceinline__ bool before(V x, int i, V y, int j) {
  return x > y || (x == y && i < j);
}

// One wave a token; lane l has experts l + 64 i.  V: the type that choices
// are compared in -- the logits as FP32 where their order is that of c, else
// c in 64 bits, so that rounding turns no order.
template <typename V, int PER>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a) {
  __shared__ V choice[4][PER * 64];
  __shared__ uint64_t kept[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= a.T) return;
  const float inf = __builtin_inff();

  float x[PER];
  float top = -inf;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < a.E ? load_logit(a, t * a.row + e) : -inf;
    top = x[i] > top ? x[i] : top;  // NaN: not above
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const float o = __shfl_xor(top, d);
    top = o > top ? o : top;
  }
  // numerators of the scores; sum: their denominator (softmax)
  V s[PER];
  V sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!(x[i] > -inf)) {
      s[i] = 0;
    } else if (a.score == MOE_SIGMOID) {
      if constexpr (sizeof(V) == 8)
        s[i] = 1.0 / (1.0 + exp(-(double)x[i]));
      else
        s[i] = 1.f / (1.f + expf(-x[i]));
    } else if (top == inf) {
      s[i] = x[i] == inf ? 1 : 0;
    } else {
      if constexpr (sizeof(V) == 8)
        s[i] = exp((double)x[i] - (double)top);
      else
        s[i] = expf(x[i] - top);
    }
    sum += s[i];
  }
  if (a.score == MOE_SOFTMAX) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
  } else {
    sum = 1;
  }
  V c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    c[i] = lowest(V{});
    if (x[i] > -inf) {
      if constexpr (sizeof(V) == 8) {
        c[i] = s[i] / sum;
        if (a.bias) c[i] += (double)a.bias[e];
        if (!(c[i] > lowest(V{}))) c[i] = lowest(V{});
      } else {
        c[i] = x[i];
      }
    }
  }
  if (a.groups > 1) {
    // marks by one lane a group, then the best groups one by one
    const int size = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < PER; ++i) choice[wave][lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    V mark = lowest(V{});
    if (lane < a.groups) {
      V first = lowest(V{}), second = lowest(V{});
      for (int j = 0; j < size; ++j) {
        const V v = choice[wave][lane * size + j];
        if (v > first) {
          second = first;
          first = v;
        } else if (v > second) {
          second = v;
        }
      }
      mark = first;
      if (a.group_best == 2 && second > lowest(V{})) mark += second;
    }
    uint64_t keep = 0;
    for (int g = 0; g < a.top_groups; ++g) {
      V best = mark;
      int at = lane;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const V o = __shfl_xor(best, d);
        const int oi = __shfl_xor(at, d);
        if (before(o, oi, best, at)) {
          best = o;
          at = oi;
        }
      }
      if (!(best > lowest(V{}))) break;
      keep |= 1ull << at;
      if (lane == at) mark = lowest(V{});
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 64 * i;
      if (e < a.E && !((keep >> (e / size)) & 1)) c[i] = lowest(V{});
    }
  }
  (void)kept;
  int id = -1;       // lane j: the j-th choice
  V weight = 0;
  V total = 0;
  for (int j = 0; j < a.k; ++j) {
    V best = c[0], score = s[0];
    int at = lane;
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (c[i] > best) {
        best = c[i];
        score = s[i];
        at = lane + 64 * i;
      }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const V o = __shfl_xor(best, d), os = __shfl_xor(score, d);
      const int oi = __shfl_xor(at, d);
      if (before(o, oi, best, at)) {
        best = o;
        score = os;
        at = oi;
      }
    }
    if (!(best > lowest(V{}))) break;
    if (lane == j) {
      id = at;
      weight = score;
    }
    total += score;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (at == lane + 64 * i) c[i] = lowest(V{});
  }
  if (lane < a.k) {
    const V by = a.renorm ? total : sum;
    a.ids[(int64_t)t * a.k + lane] = id;
    a.weights[(int64_t)t * a.k + lane] =
        id < 0 || !(by > 0) ? 0.f : (float)(weight / by) * a.scale;
  }
}

// Every workgroup counts all choices of each expert, and those before its own
// chunk, for itself, so that none waits for another; then it places its chunk.
constexpr int kTableThreads = 1024;
constexpr int kTableWaves = kTableThreads / 64;

__global__ __launch_bounds__(kTableThreads) void moe_tables_kernel(TablesArgs a, int chunk) {
  extern __shared__ int lds[];
  int* const all = lds;                 // [E]: choices of the expert
  int* const ahead = all + a.E;         // [E]: those before this chunk
  int* const in_wave = ahead + a.E;     // [waves][E]
  __shared__ int wave_sum[kTableWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int begin = blockIdx.x * chunk;
  for (int i = tid; i < 2 * a.E; i += kTableThreads) all[i] = 0;
  __syncthreads();
  for (int i = tid; i < a.n; i += kTableThreads) {
    const unsigned e = (unsigned)a.ids[i];
    if (e < (unsigned)a.E) {
      atomicAdd(&all[e], 1);
      if (i < begin) atomicAdd(&ahead[e], 1);
    }
  }
  __syncthreads();
  // exclusive sums over the experts: MOE_MAX_EXPERTS threads, one each
  static_assert(MOE_MAX_EXPERTS <= kTableThreads, "one thread an expert");
  const int n = tid < a.E ? all[tid] : 0;
  int x = n;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) wave_sum[wave] = x;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < wave; ++w) base += wave_sum[w];
  int total = 0;
  for (int w = 0; w < kTableWaves; ++w) total += wave_sum[w];
  if (tid < a.E) {
    ahead[tid] += base + x - n;  // where the chunk's first of this expert goes
    if (blockIdx.x == 0) {
      a.starts[tid] = base + x - n;
      if (tid == a.E - 1) a.starts[a.E] = base + x;
    }
  }
  // positions behind the last kept choice
  for (int i = begin + tid; i < begin + chunk && i < a.n; i += kTableThreads)
    if (i >= total) a.order[i] = -1;
  const int end = begin + chunk < a.n ? begin + chunk : a.n;
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
        for (int w = 0; w < wave; ++w) pos += in_wave[w * a.E + e];
        a.order[pos] = i;
      }
      a.where[i] = pos;
    }
    __syncthreads();
    if (tid < a.E)
      for (int w = 0; w < kTableWaves; ++w) ahead[tid] += in_wave[w * a.E + tid];
  }
}

// Eight columns a thread.
template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_kernel(CombineArgs a) {
  const int t = blockIdx.y + blockIdx.z * gridDim.y;
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (t >= a.T || c >= a.N) return;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < a.k; ++j) {
    const int p = a.where[(int64_t)t * a.k + j];
    if ((unsigned)p >= (unsigned)a.rows) continue;
    const float w = a.weights[(int64_t)t * a.k + j];
    const uint4 v = *reinterpret_cast<const uint4*>(a.Y + (int64_t)p * a.N + c);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = __builtin_fmaf(w, scale16((uint16_t)(u[i / 2] >> (16 * (i & 1))), BF16), x[i]);
  }
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = round16(x[2 * i], BF16) | ((uint32_t)round16(x[2 * i + 1], BF16) << 16);
  *reinterpret_cast<uint4*>(a.out + (int64_t)t * a.N + c) = uint4{u[0], u[1], u[2], u[3]};
}

template <typename V>
hipError_t route(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid((a.T + 3) / 4), block(256);
  if (a.E <= 64)
    hipLaunchKernelGGL((moe_route_kernel<V, 1>), grid, block, 0, stream, a);
  else if (a.E <= 128)
    hipLaunchKernelGGL((moe_route_kernel<V, 2>), grid, block, 0, stream, a);
  else if (a.E <= 256)
    hipLaunchKernelGGL((moe_route_kernel<V, 4>), grid, block, 0, stream, a);
  else if (a.E <= 512)
    hipLaunchKernelGGL((moe_route_kernel<V, 8>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((moe_route_kernel<V, 16>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  const bool by_logit = !a.bias && (a.groups == 1 || a.group_best == 1);
  return by_logit ? route<float>(a, stream) : route<double>(a, stream);
}

hipError_t launch_moe_tables(const TablesArgs& a, hipStream_t stream) {
  // chunks of a multiple of the threads, at most 256 of them
  int chunk = kTableThreads;
  while ((int64_t)chunk * 256 < a.n) chunk *= 2;
  const int groups = a.n > 0 ? (a.n + chunk - 1) / chunk : 1;
  const size_t bytes = (size_t)(2 + kTableWaves) * a.E * sizeof(int);
  if (bytes > 60 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(moe_tables_kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(moe_tables_kernel, dim3(groups), dim3(kTableThreads), bytes, stream, a, chunk);
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
