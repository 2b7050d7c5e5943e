// Page tables, slots and positions from request lengths (kv4_tables).
//
// Three exclusive prefix sums over the requests (new tokens, pages taken,
// pages given back) place everything; the rest is independent per token and
// per page.  Free pages wait in a ring, taken at its head and given back at
// its tail, so what a call reads of it (head .. head + count) and what it
// writes (from head + count on) never meet, and workgroups need not wait for
// each other.  Every workgroup therefore makes the (small) prefix sums for
// itself in LDS, beside what it needs of each request, and then takes its
// share of the tokens and pages.  lens_out and state_out may be lens and
// state: then the last workgroup to finish, counted in state_out[3], writes
// them.
//
// What bounds it: latency alone.  The launch, the trip for the lengths, the
// scan, a binary search in LDS, the trip for the page, in place the arrival.
// 256 requests of one token: 4.3 us (5.1 in place); 1000 with 62 thousand tokens: 8.4 us (11.7
// with one kind of workgroup for tokens and pages, one after another, and an
// arrival whatever the outputs).
#include "../../include/w4a16_kv4.h"
#include "kv4.hpp"

namespace w4a16 {
namespace {

constexpr int kMaxGroups = 256;
constexpr size_t kDefaultLds = 60 * 1024;  // beyond that a launch has to ask
constexpr int kOver = (int)0x80000000;  // with a length: more pages wanted than fit

// Addition of non-negative numbers that stops at `most`: associative, so a
// scan of it does not depend on its shape, and no length overflows it.
__device__ __forceinline__ int add_up_to(int a, int b, int most) {
  const unsigned s = (unsigned)a + (unsigned)b;
  return s < (unsigned)most ? (int)s : most;
}

// Lengths of a request as they count, and whether it wants too many pages.
struct Request {
  int len, want;
  bool over;
};

__device__ __forceinline__ Request request(const KvTablesArgs& a, int len, int want) {
  Request r;
  const int64_t most = (int64_t)a.max_pages * a.page;
  len = len > 0 ? len : 0;
  r.len = len < most ? len : (int)most;
  r.want = want > 0 ? want : 0;
  r.over = r.want > most;
  return r;
}

// The last index b with sums[b] <= x, for x < sums[n].
__device__ __forceinline__ int owner(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Served requests are those whose pages are there: cumulative need within
// the free pages (requests that take none are always served).  The pages of a
// request refused for its tokens need no leaving out of later sums: those
// tokens leave no room for any request after it that grows.
__device__ __forceinline__ bool served(bool over, int need_before, int need_upto, int count) {
  return !over && (need_upto == need_before || need_upto <= count);
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void kv_tables_kernel(KvTablesArgs a) {
  constexpr int kMaxPerThread = KV4_MAX_REQUESTS / THREADS;
  // exclusive sums, [B + 1] each: new tokens, pages wanted, pages returned
  extern __shared__ int lds[];
  int* const tok = lds;
  int* const need = tok + a.B + 1;
  int* const back = need + a.B + 1;
  int* const held = back + a.B + 1;  // [B]: lengths, with kOver
  __shared__ int wave_sum[3][THREADS / 64];
  __shared__ int s_refused, s_taken, s_last;
  constexpr int kMost = 0x7fffffff;
  // new tokens are summed to one past what there is room for, which tells a
  // request that ends at the room's end from one that does not fit
  const int most_tokens = a.capacity + 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.B + THREADS - 1) / THREADS;
  const int shift = 31 - __builtin_clz((unsigned)a.page);
  auto pages_of = [&](int n) { return (int)(((int64_t)n + a.page - 1) >> shift); };
  const int b0 = tid * per < a.B ? tid * per : a.B;
  const int b1 = b0 + per < a.B ? b0 + per : a.B;
  if (tid == 0) s_refused = s_taken = 0;

  const unsigned P = a.pages;
  const unsigned head = (unsigned)a.state[0] % P;
  int count = a.state[1];
  count = count < 0 ? 0 : count > a.pages ? a.pages : count;

  // the loads of all of a thread's requests at once
  int lens[kMaxPerThread], want[kMaxPerThread];
#pragma unroll
  for (int k = 0; k < kMaxPerThread; ++k) {
    if (k >= per) break;
    const int b = b0 + k < a.B ? b0 + k : a.B - 1;
    lens[k] = a.lens[b];
    want[k] = a.want[b];
  }
  int sum[3] = {0, 0, 0};
#pragma unroll
  for (int k = 0; k < kMaxPerThread; ++k) {
    if (k >= per) break;
    const int b = b0 + k;
    if (b >= b1) break;
    const Request r = request(a, lens[k], want[k]);
    const int grown = r.want > r.len ? r.want - r.len : 0;
    const int diff = r.over ? 0 : pages_of(r.want) - pages_of(r.len);
    // kept per request; made exclusive below
    tok[b + 1] = grown;
    need[b + 1] = diff > 0 ? diff : 0;
    back[b + 1] = diff < 0 ? -diff : 0;
    held[b] = r.len | (r.over ? kOver : 0);
    sum[0] = add_up_to(sum[0], grown, most_tokens);
    sum[1] = add_up_to(sum[1], need[b + 1], kMost);
    sum[2] = add_up_to(sum[2], back[b + 1], kMost);
  }
  const int most[3] = {most_tokens, kMost, kMost};
  int before[3];
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    int x = sum[s];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(x, d);
      if (lane >= d) x = add_up_to(x, y, most[s]);
    }
    before[s] = __shfl_up(x, 1);
    if (lane == 0) before[s] = 0;
    if (lane == 63) wave_sum[s][wave] = x;
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    int base = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64 - 1; ++w)  // (all read at once)
      base = add_up_to(base, w < wave ? wave_sum[s][w] : 0, most[s]);
    int x = add_up_to(base, before[s], most[s]);
    int* const sums = s == 0 ? tok : s == 1 ? need : back;
    for (int b = b0; b < b1; ++b) {
      x = add_up_to(x, sums[b + 1], most[s]);
      sums[b + 1] = x;
    }
    if (tid == 0) sums[0] = 0;
  }
  __syncthreads();

  const int tokens = tok[a.B] < a.capacity ? tok[a.B] : a.capacity;
  const int wanted = need[a.B], returned = back[a.B];
  // whether the tokens of a request that grows all have room
  auto fits = [&](int b) { return tok[b + 1] <= a.capacity; };
  // A workgroup alone does everything (in place that spares the arrival); of
  // several the last ones do the pages, beside the tokens of the others.
  const int page_groups = gridDim.x - a.token_groups;
  const bool pages_only = (int)blockIdx.x >= a.token_groups;
  const bool tokens_only = page_groups > 0 && !pages_only;
  const int stride = (pages_only ? page_groups : a.token_groups) * THREADS;
  const int first = ((int)blockIdx.x - (pages_only ? a.token_groups : 0)) * THREADS + tid;

  // pages taken: request b's j-th new page is the ring's (need[b] + j)-th
  const int take = tokens_only ? 0 : wanted < count ? wanted : count;
  for (int i = first; i < take; i += stride) {
    const int b = owner(need, a.B, i);
    if (!fits(b) || !served(false, need[b], need[b + 1], count)) continue;  // over wants none
    const int col = pages_of(held[b]) + i - need[b];
    a.table[(int64_t)b * a.max_pages + col] = a.ring[(head + (unsigned)i) % P];
  }
  // pages given back, to the tail: the last of the request's row
  for (int i = first; i < (tokens_only ? 0 : returned); i += stride) {
    const int b = owner(back, a.B, i);
    const int col = pages_of(held[b]) - (back[b + 1] - i);
    a.ring[(head + (unsigned)count + (unsigned)i) % P] =
        a.table[(int64_t)b * a.max_pages + col];
  }
  for (int t = first; t < (pages_only ? 0 : a.capacity); t += stride) {
    int slot = -1, pos = 0;
    if (t < tokens) {
      const int b = owner(tok, a.B, t);
      const int len = held[b] & ~kOver;
      pos = len + t - tok[b];
      if (fits(b) && served(held[b] & kOver, need[b], need[b + 1], count)) {
        const int col = pos >> shift, old = pages_of(len);
        // a page of this call comes from the ring: the table's entry may
        // not be written yet
        const unsigned id = col >= old
                                ? a.ring[(head + (unsigned)(need[b] + col - old)) % P]
                                : a.table[(int64_t)b * a.max_pages + col];
        if (id < P) slot = (int)(id << shift) | (pos & (a.page - 1));
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  if (!tokens_only)
    for (int b = first; b <= a.B; b += stride)
      a.q_start[b] = tok[b] < a.capacity ? tok[b] : a.capacity;

  // In place, the last workgroup writes what others may still have been
  // reading; otherwise one writes at once.
  const bool in_place = a.lens_out == a.lens || a.state_out == a.state;
  if (!in_place) {
    if (blockIdx.x != gridDim.x - 1) return;
  } else if (gridDim.x > 1) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (tid == 0)
      s_last = __hip_atomic_fetch_add(reinterpret_cast<unsigned*>(a.state_out) + 3, 1u,
                                      __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
  }
#pragma unroll
  for (int k = 0; k < kMaxPerThread; ++k) {
    const int b = b0 + k;
    if (b >= b1) break;
    const Request r = request(a, lens[k], want[k]);
    const bool ok = (r.want <= r.len || fits(b)) && served(r.over, need[b], need[b + 1], count);
    a.lens_out[b] = ok ? r.want : r.len;
    if (!ok) atomicAdd(&s_refused, 1);
    else if (need[b + 1] > need[b]) atomicMax(&s_taken, need[b + 1]);
  }
  __syncthreads();
  if (tid == 0) {
    const int64_t left = (int64_t)count - s_taken + returned;
    a.state_out[0] = (int)((head + (unsigned)s_taken) % P);
    a.state_out[1] = left < a.pages ? (int)left : a.pages;
    a.state_out[2] = s_refused;
    a.state_out[3] = 0;
  }
}

template <int THREADS>
hipError_t launch(const KvTablesArgs& args, hipStream_t stream) {
  KvTablesArgs a = args;
  int64_t groups = ((int64_t)a.capacity + THREADS - 1) / THREADS;
  if (groups < 1) groups = 1;
  if (groups > kMaxGroups) groups = kMaxGroups;
  a.token_groups = (int)groups;
  if (groups > 1 || (a.lens_out != a.lens && a.state_out != a.state)) {
    // as many as there are pages to take, and one page a request to return
    int64_t pages = ((int64_t)a.capacity / a.page + 2 * a.B + THREADS - 1) / THREADS;
    groups += pages < 1 ? 1 : pages > kMaxGroups ? kMaxGroups : pages;
  }
  const size_t lds = (4 * (size_t)a.B + 3) * sizeof(int);
  if (lds > kDefaultLds) {
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void*>(kv_tables_kernel<THREADS>),
        hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kv_tables_kernel<THREADS>, dim3((unsigned)groups), dim3(THREADS), lds,
                     stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_tables(const KvTablesArgs& a, hipStream_t stream) {
  // A token per thread (pages are fewer).  Large workgroups scan many
  // requests in fewer steps, and fewer of them arrive at the end: 1000
  // requests with 62 thousand tokens took 11.7 us with 1024 threads each, 17
  // with 256.  A decode step of 256 requests fits one small workgroup.
  return a.B <= 256 && a.capacity <= 1024 ? launch<256>(a, stream) : launch<1024>(a, stream);
}

}  // namespace w4a16
