// The C interface of the 4-bit key/value cache (include/w4a16_kv4.h):
// argument checks and launches.  Nothing here allocates, prints or
// synchronises.
#include <hip/hip_runtime.h>

#include <cstdio>

#include "../../include/w4a16_kv4.h"
#include "internal.hpp"
#include "kv4.hpp"

namespace w4a16 {
namespace {

constexpr int kKvLayoutVersion = 1;
// Rows of one call's grid and lengths stay well inside 32-bit arithmetic.
constexpr int64_t kMaxTokens = 1 << 30;
constexpr int64_t kMaxStride = 1ll << 32;

bool aligned(const void* p, int to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

bool good_page(int page) {
  return page >= kKvMinPage && page <= kKvMaxPage && (page & (page - 1)) == 0;
}

// The sizes of a cache.
int check_cache(int pages, int heads, int D, int page) {
  if (D != 64 && D != 128 && D != 256) return W4A16_ERR_SHAPE;
  if (pages <= 0 || heads <= 0 || heads > 65535 || !good_page(page)) return W4A16_ERR_SHAPE;
  if ((int64_t)pages * page > 0x7fffffff) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

bool good_dtype(int dtype) { return dtype == W4A16_DTYPE_F16 || dtype == W4A16_DTYPE_BF16; }

// A strided [T][heads][D] tensor: 16-byte loads of its rows.
int check_rows(const void* p, int64_t token, int64_t head) {
  if (!p) return W4A16_ERR_NULL;
  if (token < 0 || head < 0 || token > kMaxStride || head > kMaxStride) return W4A16_ERR_SHAPE;
  if (!aligned(p, 16) || token % 8 || head % 8) return W4A16_ERR_ALIGN;
  return W4A16_OK;
}

// One that is written: its rows must not share elements.
int check_out(const void* p, int64_t token, int64_t head, int T, int heads, int D) {
  const int rc = check_rows(p, token, head);
  if (rc != W4A16_OK) return rc;
  if (heads > 1 && head < D) return W4A16_ERR_SHAPE;
  // tokens outside the heads or, tokens of a head together, inside them
  if (T > 1 && token < (heads - 1) * head + D &&
      !(token >= D && head >= (T - 1) * token + D))
    return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// Bytes from the first to the last element of such a tensor.
size_t extent(int64_t token, int64_t head, int T, int heads, int D) {
  return ((size_t)(T - 1) * token + (size_t)(heads - 1) * head + D) * 2;
}

// Whether two such tensors of T tokens share elements.  Exact where their
// strides are alike, as in parts of one buffer; otherwise told apart by where
// they lie, and by where their rows lie within equal token strides.
bool rows_overlap(const uint16_t* x, int64_t x_token, int64_t x_head, int x_heads,
                  const uint16_t* y, int64_t y_token, int64_t y_head, int y_heads, int T, int D) {
  if (!overlap(x, extent(x_token, x_head, T, x_heads, D), y,
               extent(y_token, y_head, T, y_heads, D)))
    return false;
  // strides of dimensions of one element mean nothing
  if (T == 1) x_token = y_token = 0;
  if (x_heads == 1) x_head = y_head;
  if (y_heads == 1) y_head = x_head;
  if (x_token != y_token) return true;
  const int64_t by =
      (int64_t)(reinterpret_cast<uintptr_t>(y) - reinterpret_cast<uintptr_t>(x)) / 2;
  const int64_t wx = (x_heads - 1) * x_head + D, wy = (y_heads - 1) * y_head + D;
  if (wx <= x_token && wy <= y_token) {
    int64_t at = by % x_token;
    if (at < 0) at += x_token;
    if (at >= wx && at + wy <= x_token) return false;
  }
  if (x_head != y_head) return true;
  // Two rows are by + h heads + t tokens apart; for every h the nearest t.
  for (int64_t h = -(int64_t)(x_heads - 1); h < y_heads; ++h) {
    const int64_t off = by + h * x_head;
    int64_t t = x_token > 0 ? -off / x_token : 0;  // towards zero: the other
    for (int i = 0; i < 2; ++i) {                  // neighbour is further from it
      const int64_t at = t < -(int64_t)(T - 1) ? -(int64_t)(T - 1) : t < T - 1 ? t : T - 1;
      const int64_t apart = off + at * x_token;
      if (apart > -D && apart < D) return true;
      t += off < 0 ? 1 : -1;
    }
  }
  return false;
}

// Fills *r; positions and inv_freq must be there.
int check_rope(const int32_t* positions, int64_t pos_stride, const double* inv_freq,
               const int* sections, int axes, int pairs, int D, RopeArgs* r) {
  if (axes < 1 || axes > 3) return W4A16_ERR_SHAPE;
  if (!sections) return W4A16_ERR_NULL;
  if (pairs != KV4_ROPE_HALVES && pairs != KV4_ROPE_PAIRS) return W4A16_ERR_SHAPE;
  int64_t half = 0;
  for (int a = 0; a < axes; ++a) {
    if (sections[a] < 0) return W4A16_ERR_SHAPE;
    half += sections[a];
  }
  if (half <= 0 || 2 * half > D || (2 * half) % 16) return W4A16_ERR_SHAPE;
  if (!positions || !inv_freq) return W4A16_ERR_NULL;
  if (!aligned(positions, 4) || !aligned(inv_freq, 8)) return W4A16_ERR_ALIGN;
  if (axes > 1 && pos_stride < 0) return W4A16_ERR_SHAPE;
  r->positions = positions;
  r->pos_stride = axes > 1 ? pos_stride : 0;
  r->inv_freq = inv_freq;
  r->half = (int)half;
  r->n0 = sections[0];
  r->n01 = axes > 1 ? sections[0] + sections[1] : (int)half;
  r->pairs = pairs;
  return W4A16_OK;
}

// Whether the n bytes at p hold a position or frequency of a call of T tokens.
bool over_rope(const void* p, size_t n, const RopeArgs& r, int axes, int T) {
  for (int a = 0; a < axes; ++a)
    if (overlap(p, n, r.positions + a * r.pos_stride, (size_t)T * 4)) return true;
  return overlap(p, n, r.inv_freq, (size_t)r.half * 8);
}

int done(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_LAUNCH; }

// The cache half of the append entry points.
int check_append(const uint16_t* K, int64_t k_token, int64_t k_head, const uint16_t* V,
                 int64_t v_token, int64_t v_head, const int32_t* slots, uint8_t* cache, int T,
                 int H, int D, int pages, int page) {
  int rc = check_rows(K, k_token, k_head);
  if (rc == W4A16_OK) rc = check_rows(V, v_token, v_head);
  if (rc != W4A16_OK) return rc;
  if (!slots || !cache) return W4A16_ERR_NULL;
  if (!aligned(slots, 4) || !aligned(cache, 16)) return W4A16_ERR_ALIGN;
  const size_t bytes = kv4_cache_bytes(pages, H, D, page);
  if (overlap(cache, bytes, K, extent(k_token, k_head, T, H, D)) ||
      overlap(cache, bytes, V, extent(v_token, v_head, T, H, D)) ||
      overlap(cache, bytes, slots, (size_t)T * 4))
    return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// Sizes of an attention call that do not depend on pointers.
int check_attention(int B, int Hq, int H, int D, int max_q, int max_len, int window) {
  if (D != 64 && D != 128 && D != 256) return W4A16_ERR_SHAPE;
  if (B < 0 || H <= 0 || Hq <= 0 || Hq > 65535 || Hq % H) return W4A16_ERR_SHAPE;
  if (max_q < 0 || max_len < 0 || window < 0) return W4A16_ERR_SHAPE;
  if (max_q > kMaxTokens || max_len > kMaxTokens) return W4A16_ERR_SHAPE;
  // query rows of a request, and what a plan may count
  if ((int64_t)(Hq / H) * max_q > kMaxTokens) return W4A16_ERR_SHAPE;
  if ((int64_t)B * Hq * ((max_q + 15) / 16 + 1) > kMaxTokens) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// The plan of such a call; false if no launch takes its workgroups.
bool plan_attention(int B, int Hq, int H, int D, int max_q, int max_len, int window, int cus,
                    KvAttentionPlan* p) {
  *p = make_kv_attention_plan(B, Hq, H, D, max_q, max_len, window, cus);
  return (int64_t)B * H * p->tiles * p->splits <= kKvMaxGroups;
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int kv4_layout_version(void) { return kKvLayoutVersion; }

size_t kv4_cache_bytes(int pages, int heads, int D, int page) {
  if (check_cache(pages, heads, D, page) != W4A16_OK) return 0;
  return (size_t)pages * heads * page * (D + 8);
}

int kv4_tables(const int32_t* lens, const int32_t* want, int32_t* table, int max_pages,
               int32_t* ring, int pages, const int32_t* state, int32_t* lens_out,
               int32_t* state_out, int32_t* q_start, int32_t* slots, int32_t* positions,
               int capacity, int B, int page, void* stream) {
  if (B < 0 || B > KV4_MAX_REQUESTS || capacity < 0 || capacity > kMaxTokens) return W4A16_ERR_SHAPE;
  if (pages <= 0 || max_pages <= 0 || !good_page(page)) return W4A16_ERR_SHAPE;
  if ((int64_t)pages * page > 0x7fffffff || (int64_t)max_pages * page > kMaxTokens)
    return W4A16_ERR_SHAPE;
  if (!ring || !state || !state_out || !q_start) return W4A16_ERR_NULL;
  if (B > 0 && (!lens || !want || !table || !lens_out)) return W4A16_ERR_NULL;
  if (capacity > 0 && (!slots || !positions)) return W4A16_ERR_NULL;
  const void* all[] = {lens, want, table, ring, state, lens_out, state_out, q_start, slots, positions};
  for (const void* p : all)
    if (!aligned(p, 4)) return W4A16_ERR_ALIGN;
  // Every written buffer apart from every other one, save the two pairs
  // that may be the same.
  const size_t n = (size_t)B * 4;
  const struct { const void* p; size_t bytes; } buf[] = {
      {table, n * max_pages}, {ring, (size_t)pages * 4}, {lens_out, n}, {state_out, 16},
      {q_start, n + 4}, {slots, (size_t)capacity * 4}, {positions, (size_t)capacity * 4},
      {lens, n}, {want, n}, {state, 16}};
  for (int i = 0; i < 7; ++i)
    for (int j = i + 1; j < 10; ++j) {
      if ((i == 2 && j == 7 && buf[i].p == buf[j].p) ||
          (i == 3 && j == 9 && buf[i].p == buf[j].p))
        continue;
      if (buf[i].bytes && buf[j].bytes && overlap(buf[i].p, buf[i].bytes, buf[j].p, buf[j].bytes))
        return W4A16_ERR_SHAPE;
    }
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  KvTablesArgs a{lens, want, table, max_pages, ring, pages, state, lens_out, state_out, q_start,
                 slots, positions, capacity, B, page, 0};
  return done(launch_kv_tables(a, static_cast<hipStream_t>(stream)));
}

int kv4_rope(const uint16_t* X, int64_t x_token, int64_t x_head, uint16_t* Y, int64_t y_token,
             int64_t y_head, const int32_t* positions, int64_t pos_stride,
             const double* inv_freq, const int* sections, int axes, int pairs, int T, int H,
             int D, int dtype, void* stream) {
  if (!good_dtype(dtype)) return W4A16_ERR_DTYPE;
  if (T < 0 || T > kKvMaxAppendTokens || H < 0 || H > 65535) return W4A16_ERR_SHAPE;
  if (D != 64 && D != 128 && D != 256) return W4A16_ERR_SHAPE;
  if (T == 0 || H == 0) return W4A16_OK;
  KvAppendArgs a{};
  int rc = check_rope(positions, pos_stride, inv_freq, sections, axes, pairs, D, &a.rope);
  if (rc == W4A16_OK) rc = check_rows(X, x_token, x_head);
  if (rc == W4A16_OK) rc = check_out(Y, y_token, y_head, T, H, D);
  if (rc != W4A16_OK) return rc;
  if (!(X == Y && x_token == y_token && x_head == y_head) &&
      rows_overlap(X, x_token, x_head, H, Y, y_token, y_head, H, T, D))
    return W4A16_ERR_SHAPE;
  if (over_rope(Y, extent(y_token, y_head, T, H, D), a.rope, axes, T)) return W4A16_ERR_SHAPE;
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  a.q = Rows{X, x_token, x_head};
  a.k = a.v = a.q;
  a.qo = Y;
  a.qo_token = y_token;
  a.qo_head = y_head;
  a.T = T;
  a.Hq = H;
  return done(launch_kv_append(a, D, dtype, static_cast<hipStream_t>(stream)));
}

int kv4_append(const uint16_t* K, int64_t k_token, int64_t k_head, const uint16_t* V,
               int64_t v_token, int64_t v_head, const int32_t* slots, uint8_t* cache, int T,
               int H, int D, int pages, int page, int dtype, void* stream) {
  if (!good_dtype(dtype)) return W4A16_ERR_DTYPE;
  if (T < 0 || T > kKvMaxAppendTokens) return W4A16_ERR_SHAPE;
  int rc = check_cache(pages, H, D, page);
  if (rc != W4A16_OK) return rc;
  if (T == 0) return W4A16_OK;
  rc = check_append(K, k_token, k_head, V, v_token, v_head, slots, cache, T, H, D, pages, page);
  if (rc != W4A16_OK) return rc;
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  KvAppendArgs a{};
  a.k = Rows{K, k_token, k_head};
  a.v = Rows{V, v_token, v_head};
  a.q = a.k;
  a.slots = slots;
  a.cache = cache;
  a.T = T;
  a.H = H;
  a.pages = pages;
  a.page = page;
  return done(launch_kv_append(a, D, dtype, static_cast<hipStream_t>(stream)));
}

int kv4_rope_append(const uint16_t* Q, int64_t q_token, int64_t q_head, const uint16_t* K,
                    int64_t k_token, int64_t k_head, const uint16_t* V, int64_t v_token,
                    int64_t v_head, uint16_t* Qout, int64_t qo_token, int64_t qo_head,
                    const int32_t* positions, int64_t pos_stride, const double* inv_freq,
                    const int* sections, int axes, int pairs, const int32_t* slots,
                    uint8_t* cache, int T, int Hq, int H, int D, int pages, int page, int dtype,
                    void* stream) {
  if (!good_dtype(dtype)) return W4A16_ERR_DTYPE;
  if (T < 0 || T > kKvMaxAppendTokens || Hq < 0 || Hq > 65535) return W4A16_ERR_SHAPE;
  int rc = check_cache(pages, H, D, page);
  if (rc != W4A16_OK) return rc;
  if (T == 0) return W4A16_OK;
  KvAppendArgs a{};
  rc = check_rope(positions, pos_stride, inv_freq, sections, axes, pairs, D, &a.rope);
  if (rc == W4A16_OK)
    rc = check_append(K, k_token, k_head, V, v_token, v_head, slots, cache, T, H, D, pages, page);
  if (rc == W4A16_OK && Hq > 0) {
    rc = check_rows(Q, q_token, q_head);
    if (rc == W4A16_OK) rc = check_out(Qout, qo_token, qo_head, T, Hq, D);
  }
  if (rc != W4A16_OK) return rc;
  const size_t bytes = kv4_cache_bytes(pages, H, D, page);
  if (over_rope(cache, bytes, a.rope, axes, T)) return W4A16_ERR_SHAPE;
  if (Hq > 0) {
    if (!(Q == Qout && q_token == qo_token && q_head == qo_head) &&
        rows_overlap(Q, q_token, q_head, Hq, Qout, qo_token, qo_head, Hq, T, D))
      return W4A16_ERR_SHAPE;
    if (rows_overlap(K, k_token, k_head, H, Qout, qo_token, qo_head, Hq, T, D) ||
        rows_overlap(V, v_token, v_head, H, Qout, qo_token, qo_head, Hq, T, D))
      return W4A16_ERR_SHAPE;
    const size_t out = extent(qo_token, qo_head, T, Hq, D);
    if (over_rope(Qout, out, a.rope, axes, T) || overlap(Qout, out, slots, (size_t)T * 4) ||
        overlap(cache, bytes, Qout, out) ||
        overlap(cache, bytes, Q, extent(q_token, q_head, T, Hq, D)))
      return W4A16_ERR_SHAPE;
  }
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  a.k = Rows{K, k_token, k_head};
  a.v = Rows{V, v_token, v_head};
  a.q = Hq > 0 ? Rows{Q, q_token, q_head} : a.k;
  a.qo = Qout;
  a.qo_token = qo_token;
  a.qo_head = qo_head;
  a.slots = slots;
  a.cache = cache;
  a.T = T;
  a.Hq = Hq;
  a.H = H;
  a.pages = pages;
  a.page = page;
  return done(launch_kv_append(a, D, dtype, static_cast<hipStream_t>(stream)));
}

int kv4_dequant_debug(const int32_t* slots, const uint8_t* cache, uint16_t* K, uint16_t* V,
                      int T, int H, int D, int pages, int page, int dtype, void* stream) {
  if (!good_dtype(dtype)) return W4A16_ERR_DTYPE;
  if (T < 0 || T > kMaxTokens) return W4A16_ERR_SHAPE;
  const int rc = check_cache(pages, H, D, page);
  if (rc != W4A16_OK) return rc;
  if (T == 0) return W4A16_OK;
  if (!slots || !cache || !K || !V) return W4A16_ERR_NULL;
  if (!aligned(slots, 4) || !aligned(cache, 16) || !aligned(K, 16) || !aligned(V, 16))
    return W4A16_ERR_ALIGN;
  const size_t bytes = kv4_cache_bytes(pages, H, D, page), out = (size_t)T * H * D * 2;
  if (overlap(cache, bytes, K, out) || overlap(cache, bytes, V, out) || overlap(K, out, V, out) ||
      overlap(slots, (size_t)T * 4, K, out) || overlap(slots, (size_t)T * 4, V, out))
    return W4A16_ERR_SHAPE;
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  return done(launch_kv_dequant(slots, cache, K, V, T, H, D, pages, page, dtype,
                                static_cast<hipStream_t>(stream)));
}

size_t kv4_attention_workspace_bytes(int B, int Hq, int H, int D, int max_q, int max_len,
                                     int window) {
  if (check_attention(B, Hq, H, D, max_q, max_len, window) != W4A16_OK) return 0;
  if (B == 0 || max_q == 0) return 0;
  const int cus = current_cus(nullptr);
  if (cus <= 0) return 0;
  KvAttentionPlan p;
  return plan_attention(B, Hq, H, D, max_q, max_len, window, cus, &p) ? p.workspace_bytes : 0;
}

int kv4_attention_describe(int B, int Hq, int H, int D, int max_q, int max_len, int window,
                           int cus, char* buf, size_t len) {
  if (!buf || len == 0) return W4A16_ERR_NULL;
  buf[0] = 0;
  const int rc = check_attention(B, Hq, H, D, max_q, max_len, window);
  if (rc != W4A16_OK) return rc;
  if (B == 0 || max_q == 0 || cus < 0) return W4A16_ERR_SHAPE;
  if (cus == 0) cus = current_cus(nullptr);
  if (cus <= 0) return W4A16_ERR_DEVICE;
  KvAttentionPlan p;
  if (!plan_attention(B, Hq, H, D, max_q, max_len, window, cus, &p)) return W4A16_ERR_SHAPE;
  snprintf(buf, len, "kv_attention<%d,%d,%s> grid=%lld block=%d tiles=%d splits=%d chunk=%d workspace=%zu",
           D, p.row_tile, p.rows ? "rows" : "tokens", (long long)B * H * p.tiles * p.splits,
           64 * p.waves, p.tiles, p.splits, p.chunk, p.workspace_bytes);
  return W4A16_OK;
}

int kv4_attention(const uint16_t* Q, int64_t q_token, int64_t q_head, const uint8_t* cache,
                  const int32_t* table, int max_pages, const int32_t* lens,
                  const int32_t* q_start, uint16_t* O, int64_t o_token, int64_t o_head,
                  float* lse, int T, int B, int Hq, int H, int D, int pages, int page,
                  float scale, int window, int max_q, int max_len, int dtype, void* workspace,
                  void* stream) {
  if (!good_dtype(dtype)) return W4A16_ERR_DTYPE;
  int rc = check_attention(B, Hq, H, D, max_q, max_len, window);
  if (rc == W4A16_OK) rc = check_cache(pages, H, D, page);
  if (rc != W4A16_OK) return rc;
  if (T < 0 || T > kMaxTokens || max_pages <= 0 || (int64_t)max_pages * page > kMaxTokens)
    return W4A16_ERR_SHAPE;
  if (!(scale > 0.f) || scale > 3e38f) return W4A16_ERR_SHAPE;
  if (T == 0 || B == 0 || max_q == 0) return W4A16_OK;
  rc = check_rows(Q, q_token, q_head);
  if (rc == W4A16_OK) rc = check_out(O, o_token, o_head, T, Hq, D);
  if (rc != W4A16_OK) return rc;
  if (!cache || !table || !lens) return W4A16_ERR_NULL;
  if (!aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(q_start, 4) ||
      !aligned(lse, 4))
    return W4A16_ERR_ALIGN;
  const size_t bytes = kv4_cache_bytes(pages, H, D, page);
  const size_t out = extent(o_token, o_head, T, Hq, D), in = extent(q_token, q_head, T, Hq, D);
  const size_t lse_bytes = (size_t)T * Hq * 4;
  const struct { const void* p; size_t bytes; } read[] = {
      {Q, in}, {cache, bytes}, {table, (size_t)B * max_pages * 4}, {lens, (size_t)B * 4},
      {q_start, q_start ? (size_t)(B + 1) * 4 : 0}};
  for (const auto& r : read) {
    if (&r != read && r.bytes && overlap(O, out, r.p, r.bytes)) return W4A16_ERR_SHAPE;
    if (lse && r.bytes && overlap(lse, lse_bytes, r.p, r.bytes)) return W4A16_ERR_SHAPE;
  }
  if (rows_overlap(Q, q_token, q_head, Hq, O, o_token, o_head, Hq, T, D)) return W4A16_ERR_SHAPE;
  if (lse && overlap(O, out, lse, lse_bytes)) return W4A16_ERR_SHAPE;
  const int cus = current_cus(nullptr);
  if (cus <= 0) return W4A16_ERR_DEVICE;
  KvAttentionPlan p;
  if (!plan_attention(B, Hq, H, D, max_q, max_len, window, cus, &p)) return W4A16_ERR_SHAPE;
  if (p.workspace_bytes > 0) {
    if (!workspace) return W4A16_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return W4A16_ERR_ALIGN;
    for (const auto& r : read)
      if (r.bytes && overlap(workspace, p.workspace_bytes, r.p, r.bytes)) return W4A16_ERR_SHAPE;
    if (overlap(workspace, p.workspace_bytes, O, out) ||
        (lse && overlap(workspace, p.workspace_bytes, lse, lse_bytes)))
      return W4A16_ERR_SHAPE;
  }
  KvAttentionArgs a{Rows{Q, q_token, q_head}, cache, table, max_pages, lens, q_start, O, o_token,
                    o_head, lse, T, B, Hq, H, pages, page, scale, window, max_q};
  return done(launch_kv_attention(p, a, D, dtype, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
