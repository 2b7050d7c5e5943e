// The paged 4-bit key/value cache (include/w4a16_kv4.h): its addresses, and
// the declarations its translation units share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace w4a16 {

// Tokens of a unit, the smallest run of a page that is contiguous for one
// head: one operand of the 16x16x32 matrix instruction has 16 rows.
constexpr int kKvUnit = 16;
constexpr int kKvMinPage = 16, kKvMaxPage = 1024;

// Workgroups of 256 threads that a launch takes: it has fewer than 2^32 threads.
constexpr int64_t kKvMaxGroups = (1 << 24) - 1;
// Tokens of a workgroup of the append kernel, where there are many, and so of
// a call.
constexpr int kKvAppendTokensLog = 2;
constexpr int64_t kKvMaxAppendTokens = kKvMaxGroups << kKvAppendTokensLog;

// Byte offsets inside a unit.
template <int D>
struct KvUnit {
  static constexpr int bytes = kKvUnit * (D + 8);
  static constexpr int values = 8 * D;          // value codes
  static constexpr int key_params = 16 * D;     // FP16 (scale, offset) pairs
  static constexpr int value_params = 16 * D + 64;
};

// The unit that holds token `at` of page `id` for `head`.
template <int D>
__host__ __device__ inline int64_t kv_unit_offset(int64_t id, int heads, int head, int page,
                                                  int at) {
  return ((id * heads + head) * (page / kKvUnit) + at / kKvUnit) * (int64_t)KvUnit<D>::bytes;
}

// One strided 16-bit tensor [T][heads][D].
struct Rows {
  const uint16_t* p;
  int64_t token, head;
};

// Rotary positions of a call; n[a] frequency pairs belong to axis a.
struct RopeArgs {
  const int32_t* positions;
  int64_t pos_stride;
  const double* inv_freq;
  int n0, n01;  // pairs of axis 0, of axes 0 and 1
  int half;     // all pairs
  int pairs;    // enum kv4_rope_pairs
};

struct KvAppendArgs {
  Rows q, k, v;
  uint16_t* qo;
  int64_t qo_token, qo_head;
  RopeArgs rope;  // half == 0: no rotation
  const int32_t* slots;
  uint8_t* cache;
  int T, Hq, H, pages, page;
};

struct KvTablesArgs {
  const int32_t *lens, *want;
  int32_t* table;
  int max_pages;
  int32_t* ring;
  int pages;
  const int32_t* state;
  int32_t *lens_out, *state_out, *q_start, *slots, *positions;
  int capacity, B, page;
  int token_groups;  // workgroups that take tokens; the others take pages
};

// Division of 0 <= n < 2^31 by a number the host knows: with 2^(s-1) < d <=
// 2^s and m = floor(2^32 (2^s - d) / d) + 1, floor(n / d) is
// (n + floor(n m / 2^32)) >> s (the round-up reciprocal).  A workgroup's start
// is a chain of divisions; by the instruction for reciprocals they take 1 us.
struct Divisor {
  uint32_t d, m;
  int s;
  Divisor() = default;
  explicit Divisor(int by) : d((uint32_t)by), m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)((((1ull << s) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ int of(int n) const {
    return (int)(((uint32_t)n + __umulhi((uint32_t)n, m)) >> s);
  }
  __device__ __forceinline__ int rest(int n) const { return n - of(n) * (int)d; }
};

struct KvAttentionArgs {
  Rows q;
  const uint8_t* cache;
  const int32_t* table;
  int max_pages;
  const int32_t *lens, *q_start;
  uint16_t* o;
  int64_t o_token, o_head;
  float* lse;
  int T, B, Hq, H, pages, page;
  float scale;
  int window, max_q;
  // of the plan: row tiles, token ranges, tokens of a range
  Divisor tiles, splits, chunk, group, heads;
};

// How a kv4_attention call is cut into work.
//  row_tile  query rows (query, head of the group) of a workgroup
//  rows   1: its waves take different ones and walk the same tokens;
//         0: they share them and divide the tokens
//  waves  waves per workgroup
//  tiles  row tiles per (request, head)
//  splits token ranges per row tile, one workgroup each, of `chunk` tokens
//         (longer where a request is longer than planned)
struct KvAttentionPlan {
  int row_tile, rows, waves, tiles, splits, chunk;
  size_t workspace_bytes;
};

KvAttentionPlan make_kv_attention_plan(int B, int Hq, int H, int D, int max_q, int max_len,
                                       int window, int cus);

hipError_t launch_kv_tables(const KvTablesArgs& a, hipStream_t stream);
hipError_t launch_kv_append(const KvAppendArgs& a, int D, int dtype, hipStream_t stream);
hipError_t launch_kv_dequant(const int32_t* slots, const uint8_t* cache, uint16_t* K,
                             uint16_t* V, int T, int H, int D, int pages, int page, int dtype,
                             hipStream_t stream);
hipError_t launch_kv_attention(const KvAttentionPlan& p, const KvAttentionArgs& a, int D,
                               int dtype, void* workspace, hipStream_t stream);

}  // namespace w4a16
