// The C interface of the expert layers and of products in 8-bit floating
// point (include/w4a16_moe.h, include/w8a8.h): argument checks, plans and
// launches.  Nothing here allocates, prints or synchronises.
#include <hip/hip_runtime.h>

#include <cstdio>

#include "internal.hpp"
#include "moe.hpp"
#include "product.hpp"
#include "w4a16_moe.h"
#include "w8a8.h"

namespace w4a16 {
namespace {

constexpr int kW8a8LayoutVersion = 1;
constexpr int kMaxRows = 1 << 24;        // rows of one call
constexpr int kMaxColumns = 1 << 24;
constexpr int64_t kMaxStride = 1ll << 32;

bool aligned(const void* p, int to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

struct Part {
  const void* p;
  size_t bytes;
};

// Whether one of the `written` first parts shares memory with another part.
bool share(const Part* part, int written, int n) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(part[i].p),
                      y = reinterpret_cast<uintptr_t>(part[j].p);
      if (part[i].bytes && part[j].bytes && x < y + part[j].bytes && y < x + part[i].bytes)
        return true;
    }
  return false;
}

bool good_dtype(int dtype) { return dtype == W4A16_DTYPE_F16 || dtype == W4A16_DTYPE_BF16; }

// Sizes of weights: K and the columns W of one matrix.  Offsets in the
// kernels are 32 bits from a wave's first column block (K) and over the scales
// of one matrix.
bool good_weights(int K, int64_t W) {
  return K > 0 && K % kBlockK == 0 && K <= (1 << 20) && W > 0 && W % kBlockN == 0 &&
         W <= (1ll << 36) / K && W <= kMaxColumns;
}

int done(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_LAUNCH; }

int check_product(int rows, int K, int N, int E, bool gate, bool f8) {
  if (rows < 0 || rows > kMaxRows || N < 0 || E < 1 || E > MOE_MAX_EXPERTS) return W4A16_ERR_SHAPE;
  if (N % (gate && f8 ? 32 : 16)) return W4A16_ERR_SHAPE;
  if (!good_weights(K, N > 0 ? (int64_t)N * (gate ? 2 : 1) : 16)) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

bool good_plan(const ProductPlan& p) {
  // threads of one launch dimension; the tile counts themselves fit in int
  return (int64_t)p.tiles_m * p.tiles_n * 64 * p.waves < (1ll << 32);
}

int describe(int format, int rows, int K, int N, int E, bool gate, int cus, char* buf,
             size_t len) {
  if (!buf || len == 0) return W4A16_ERR_NULL;
  buf[0] = 0;
  if (rows == 0 || N == 0) return W4A16_ERR_SHAPE;
  const int rc = check_product(rows, K, N, E > 0 ? E : 1, gate, format == kProdF8);
  if (rc != W4A16_OK) return rc;
  if (cus == 0) cus = current_cus(nullptr);
  if (cus <= 0) return W4A16_ERR_DEVICE;
  const ProductPlan p = make_product_plan(format, rows, K, N, E, gate, cus);
  if (!good_plan(p)) return W4A16_ERR_SHAPE;
  std::snprintf(buf, len, "%s<%d,%d,%d,%d> tile=%dx%d grid=%dx%d splits=%d workspace=%zu",
                p.tile ? "product_tile_kernel" : "product_stream_kernel", p.mb, p.nb, p.waves,
                p.depth, p.tm, p.tn, p.tiles_m, p.tiles_n, p.splits, p.workspace_bytes);
  return W4A16_OK;
}

// The expert products' shared part: everything but the operands' types.
int check_experts(const void* A, int a_rows, const int32_t* order, int k, const int32_t* starts,
                  const void* Bpacked, const void* scales, const uint16_t* C, int rows, int K,
                  int N, int E, int activation, int dtype, bool f8) {
  if (!good_dtype(dtype)) return W4A16_ERR_DTYPE;
  if (activation != MOE_ACT_NONE && activation != MOE_ACT_SILU_GATE) return W4A16_ERR_EPILOGUE;
  const int rc = check_product(rows, K, N, E, activation == MOE_ACT_SILU_GATE, f8);
  if (rc != W4A16_OK) return rc;
  if (rows == 0 || N == 0) return W4A16_OK;
  if (k < 1 || a_rows < (order ? 1 : rows) || a_rows > kMaxRows) return W4A16_ERR_SHAPE;
  if (!A || !starts || !Bpacked || !scales || !C) return W4A16_ERR_NULL;
  if (!aligned(A, 16) || !aligned(Bpacked, 16) || !aligned(scales, 16) || !aligned(C, 16) ||
      !aligned(starts, 4) || !aligned(order, 4))
    return W4A16_ERR_ALIGN;
  return W4A16_OK;
}

}  // namespace

namespace {

// A compiled shape of the tile kernel, and what a matrix product in it takes,
// measured at 4096 and 11008 x 4096 and 4096 x 22016 with 16 to 2048 rows:
// `alone` microseconds a K block for a workgroup that has its compute unit to
// itself, `shared` for each of several, `once` for the rest of a workgroup.
struct Tile {
  int mb, nb;
  float alone, shared, once;
};
constexpr Tile kTilesF8[] = {{2, 1, 0.30f, 0.19f, 1.5f}, {4, 1, 0.36f, 0.26f, 1.5f},
                             {4, 2, 0.49f, 0.37f, 2.f},  {8, 2, 0.62f, 0.56f, 7.f},
                             {8, 4, 1.33f, 0.90f, 12.f}};

ProductPlan stream_plan(int mb, int nb, int waves, int depth) {
  ProductPlan p{};
  p.mb = mb;
  p.nb = nb;
  p.waves = waves;
  p.depth = depth;
  p.tm = 16 * mb;
  p.tn = 16 * nb;
  p.splits = 1;
  return p;
}

ProductPlan tile_plan(int mb, int nb) {
  ProductPlan p{};
  p.tile = 1;
  p.mb = mb;
  p.nb = nb;
  p.waves = 4;
  p.depth = 4;
  p.tm = 16 * mb;
  p.tn = 16 * nb * p.waves;
  p.splits = 1;
  return p;
}

// A matrix product.  Up to 16 rows the streaming kernel, with one column block
// a workgroup while two of them a compute unit cover the columns (4096 x 4096,
// 16 rows: 6.1 us against 8.1 in tiles; 4096 x 12288: 16.6, but 13.7 with two
// blocks).  Up to 32 rows too while K is short (2048 x 4096: 5.8 against 6.4;
// 11008 x 4096: 18.6 against 15.3).  Beyond, the tile and the number of K
// ranges whose predicted time is least: a compute unit takes its workgroups'
// K blocks one after another, a join of s ranges takes s trips of the tile's
// sums (64 x 64, 11008 x 4096 at 64 rows: 32.5, 21.2 and 17.8 us in 1, 2 and 4
// ranges).
ProductPlan plan_matrix(int M, int K, int N, int cus) {
  const int KB = K / kBlockK;
  if (M <= 16 || (M <= 32 && KB <= 24 && N / 16 <= 2 * cus)) {
    if (M > 16) return stream_plan(2, 1, 8, 3);
    return N / 16 <= 2 * cus ? stream_plan(1, 1, 8, 4) : stream_plan(1, 2, 4, 4);
  }
  ProductPlan best{};
  float least = 0.f;
  for (const Tile& t : kTilesF8) {
    ProductPlan p = tile_plan(t.mb, t.nb);
    const int64_t tiles = (int64_t)((M + p.tm - 1) / p.tm) * ((N + p.tn - 1) / p.tn);
    for (int s = 1; s <= 8; s *= 2) {
      if (s > 1 && (KB < 8 * s || tiles * s > 2 * cus || tiles > kMaxSplitTiles)) break;
      const int64_t each = (tiles * s + cus - 1) / cus;
      const float block = each * t.shared > t.alone ? each * t.shared : t.alone;
      const float join = s == 1 ? 0.f : s * (1.9f + 0.5f * p.tm * p.tn / 4096.f);
      const float us = t.once + (KB + s - 1) / s * block + join;
      if (best.tm == 0 || us < least) {
        least = us;
        best = p;
        best.splits = s;
      }
    }
  }
  return best;
}

// Rows of experts.  With few rows each, by their mean, the streaming kernel
// (mean 4: 59.7 us against 59.0 in tiles of 32 rows for 64 experts of
// 2048 x 2816 in e4m3, 74.6 against 84.9 for 8 of 4096 x 22016 in 4 bits; 8:
// 89.8 and 83.7), unless K is too short for its waves and the columns are many
// (5 rows each of 60 experts of K x 17664: 256 105 in e4m3 and 65.2 in 4 bits
// against 72.7 and 46.7 in tiles; 1024 x 8192 100 and 69.0 against 102 and
// 68.1).  Beyond, the shape whose predicted time is least, from the
// sum of tiles (half a tile an expert for unlike loads) as in plan_matrix: with
// many tiles by the rate of each shape, with few by what one takes alone.
// Constants measured at the first three of, in us:
//                                           streaming  32 x 128  64 x *  128 x 256
//   4 bits, 8 x 4096 x 22016, 16 rows each  112        89.5
//     48                                               129       129
//     96                                               228       169
//   e4m3, 64 x 2048 x 2816, 16 rows each    82.2       65.5
//     32                                               74.3      69.4
//     96                                                         100     96.3
//     192                                                        162     120
//   e4m3, 16 x 8960 x 256, 36 rows each     25.5       35.3      40.9
//     4 x 8192 x 256, 1024                  75.9       40.9      42.8    80.8
//   4 bits, 8 x 8192 x 512, 32 rows each    20.6       35.1      73.0
//     64 x 4864 x 320, 54 (BF16)            54.0       34.2      60.8
//     4 x 8192 x 256, 1024                  66.6       50.1      74.6
// (64 x *: 64 x 128 in e4m3, 64 x 256 in 4 bits.)
// Choices that the tables leave out count in `rows`, since how many there are
// is known on the device only; with half of them left out the mean is twice the
// true one.  Planned by all rows and by the kept ones, in us: 4 bits, 8 experts of
// 4096 x 22016, 2 to 512 kept rows each, 77.5 : 72.5 at 6, 103 : 84.8 at 32, the
// rest within 7%; e4m3, 64 experts of 2048 x 2816, 2 to 256 rows, 64.3 : 60.2 at 4,
// 80.9 : 74.5 at 64, the rest within 6%.
// 4 bits stream four column blocks a workgroup: 16 tokens through 8 experts of
// 4096 x 22016 93.2 us with two, 74.6 with four; with fewer workgroups than
// compute units two, and eight waves (one token, 11008 x 4096: 25.6 and 19.4).
constexpr Tile kExpertsF8[] = {
    {2, 2, 0.48f, 0.28f, 1.5f}, {4, 2, 0.56f, 0.37f, 2.f}, {8, 4, 1.20f, 0.90f, 12.f}};
constexpr Tile kExpertsI4[] = {{2, 2, 0.70f, 0.38f, 1.5f}, {4, 4, 1.20f, 1.10f, 8.f}};
constexpr Tile kStreamF8 = {1, 2, 0.28f, 0.145f, 4.f}, kStreamI4 = {1, 4, 0.27f, 0.24f, 4.f};

ProductPlan plan_experts(bool f8, int rows, int used, int K, int W, int cus) {
  const int mean = (rows + used - 1) / used;
  if (mean <= (f8 ? 6 : 7)) {
    if (K < 8 * kBlockK && (int64_t)used * (W / 64) > 4 * (int64_t)cus) return tile_plan(2, 2);
    if (f8) return stream_plan(1, 2, 4, 4);
    return (int64_t)used * (W / 64) >= cus ? stream_plan(1, 4, 4, 3) : stream_plan(1, 2, 8, 3);
  }
  auto us = [&](const Tile& t, const ProductPlan& p) {
    const float down = (float)mean / p.tm + 0.5f, across = (float)((W + p.tn - 1) / p.tn);
    const float each = used * (down > 1.f ? down : 1.f) * across / cus;
    const float block = each * t.shared > t.alone ? each * t.shared : t.alone;
    return t.once + K / kBlockK * block;
  };
  ProductPlan best = f8 ? stream_plan(1, 2, 4, 4) : stream_plan(1, 4, 4, 3);
  float least = us(f8 ? kStreamF8 : kStreamI4, best);
  auto consider = [&](const Tile& t) {
    const ProductPlan p = tile_plan(t.mb, t.nb);
    const float time = us(t, p);
    if (time < least) {
      least = time;
      best = p;
    }
  };
  if (f8)
    for (const Tile& t : kExpertsF8) consider(t);
  else
    for (const Tile& t : kExpertsI4) consider(t);
  return best;
}

}  // namespace

ProductPlan make_product_plan(int format, int rows, int K, int N, int E, bool gate, int cus) {
  const int experts = E > 0 ? E : 1;
  const int used = rows < experts ? rows : experts;
  ProductPlan p = E == 0 ? plan_matrix(rows, K, N, cus)
                         : plan_experts(format == kProdF8, rows, used, K, gate ? 2 * N : N, cus);
  if (gate) p.tn /= 2;
  p.tiles_n = (N + p.tn - 1) / p.tn;
  // the most that the used experts' rows can make: sum of ceil(rows / tm)
  p.tiles_m = (int)(((int64_t)rows + (int64_t)used * (p.tm - 1)) / p.tm);
  if (p.splits > 1)
    p.workspace_bytes = kCounterHeaderBytes +
                        (size_t)p.tiles_m * p.tiles_n * p.splits * p.tm * p.tn * 4;
  return p;
}

}  // namespace w4a16

using namespace w4a16;

extern "C" {

int w8a8_layout_version(void) { return kW8a8LayoutVersion; }

size_t w8a8_packed_bytes(int K, int N) { return good_weights(K, N) ? (size_t)K * N : 0; }

int w8a8_repack(const uint8_t* B, uint8_t* Bpacked, int K, int N, void* stream) {
  if (!good_weights(K, N)) return W4A16_ERR_SHAPE;
  if (!B || !Bpacked) return W4A16_ERR_NULL;
  if (!aligned(B, 16) || !aligned(Bpacked, 16)) return W4A16_ERR_ALIGN;
  const size_t n = (size_t)K * N;
  const Part part[] = {{Bpacked, n}, {B, n}};
  if (share(part, 1, 2)) return W4A16_ERR_SHAPE;
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  return done(launch_w8a8_repack(B, Bpacked, K, N, static_cast<hipStream_t>(stream)));
}

int w8a8_quantize(const uint16_t* X, int64_t x_row, uint8_t* Xq, float* Xs, int T, int K,
                  int dtype, void* stream) {
  if (!good_dtype(dtype)) return W4A16_ERR_DTYPE;
  if (T < 0 || T > kMaxRows || K <= 0 || K % kBlockK) return W4A16_ERR_SHAPE;
  if (T == 0) return W4A16_OK;
  if (T > 1 && (x_row < K || x_row > kMaxStride)) return W4A16_ERR_SHAPE;
  if (!X || !Xq || !Xs) return W4A16_ERR_NULL;
  if (!aligned(X, 16) || !aligned(Xq, 16) || !aligned(Xs, 16)) return W4A16_ERR_ALIGN;
  if (T > 1 && x_row % 8) return W4A16_ERR_ALIGN;
  if (T == 1) x_row = K;
  const Part part[] = {{Xq, (size_t)T * K}, {Xs, (size_t)T * (K / kBlockK) * 4},
                       {X, ((size_t)(T - 1) * x_row + K) * 2}};
  if (share(part, 2, 3)) return W4A16_ERR_SHAPE;
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  return done(
      launch_w8a8_quantize(X, x_row, Xq, Xs, T, K, dtype, static_cast<hipStream_t>(stream)));
}

size_t w8a8_workspace_bytes(int M, int K, int N) {
  if (M <= 0 || N <= 0 || check_product(M, K, N, 1, false, true) != W4A16_OK) return 0;
  const int cus = current_cus(nullptr);
  if (cus <= 0) return 0;
  return make_product_plan(kProdF8, M, K, N, 0, false, cus).workspace_bytes;
}

int w8a8_describe(int M, int K, int N, int cus, char* buf, size_t len) {
  return describe(kProdF8, M, K, N, 0, false, cus, buf, len);
}

int w8a8_gemm(const uint8_t* A, const float* As, const uint8_t* Bpacked, const float* Bs,
              uint16_t* C, int M, int K, int N, int dtype, void* workspace, void* stream) {
  if (!good_dtype(dtype)) return W4A16_ERR_DTYPE;
  const int rc = check_product(M, K, N, 1, false, true);
  if (rc != W4A16_OK) return rc;
  if (M == 0 || N == 0) return W4A16_OK;
  if (!A || !As || !Bpacked || !Bs || !C) return W4A16_ERR_NULL;
  const void* all[] = {A, As, Bpacked, Bs, C, workspace};
  for (const void* q : all)
    if (!aligned(q, 16)) return W4A16_ERR_ALIGN;
  const size_t KB = K / kBlockK;
  Part part[] = {{C, (size_t)M * N * 2}, {workspace, 0}, {A, (size_t)M * K},
                 {As, (size_t)M * KB * 4}, {Bpacked, (size_t)K * N},
                 {Bs, ((size_t)N + 127) / 128 * KB * 4}};
  if (share(part, 2, 6)) return W4A16_ERR_SHAPE;
  const int cus = current_cus(nullptr);
  if (cus <= 0) return W4A16_ERR_DEVICE;
  const ProductPlan plan = make_product_plan(kProdF8, M, K, N, 0, false, cus);
  if (!good_plan(plan)) return W4A16_ERR_SHAPE;
  if (plan.workspace_bytes) {
    if (!workspace) return W4A16_ERR_WORKSPACE;
    part[1].bytes = plan.workspace_bytes;
    if (share(part, 2, 6)) return W4A16_ERR_SHAPE;
  }
  ProductArgs a{};
  a.A = A;
  a.As = As;
  a.B = Bpacked;
  a.S = Bs;
  a.C = C;
  a.a_rows = a.rows = M;
  a.k = 1;
  a.E = 1;
  a.K = K;
  a.N = a.W = N;
  a.dtype = dtype;
  a.tiles_n = plan.tiles_n;
  a.splits = plan.splits;
  if (plan.splits > 1) {
    a.counters = static_cast<unsigned*>(workspace);
    a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterHeaderBytes);
  }
  return done(launch_product_f8(plan, a, false, static_cast<hipStream_t>(stream)));
}

int moe_route(const void* logits, int64_t row, int logits_type, const float* bias, int32_t* ids,
              float* weights, int T, int E, int k, int score, int groups, int top_groups,
              int group_best, int renorm, float scale, void* stream) {
  if (logits_type != MOE_LOGITS_F16 && logits_type != MOE_LOGITS_BF16 &&
      logits_type != MOE_LOGITS_F32)
    return W4A16_ERR_DTYPE;
  if (score != MOE_SOFTMAX && score != MOE_SIGMOID) return W4A16_ERR_SHAPE;
  if (T < 0 || T > kMaxRows || E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_TOP || k > E)
    return W4A16_ERR_SHAPE;
  if (groups < 1 || groups > MOE_MAX_GROUPS || E % groups || top_groups < 1 ||
      top_groups > groups || group_best < 1 || group_best > 2)
    return W4A16_ERR_SHAPE;
  if (T == 0) return W4A16_OK;
  if (T > 1 && (row < E || row > kMaxStride)) return W4A16_ERR_SHAPE;
  if (!logits || !ids || !weights) return W4A16_ERR_NULL;
  const int size = logits_type == MOE_LOGITS_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return W4A16_ERR_ALIGN;
  if (T == 1) row = E;
  const size_t out = (size_t)T * k * 4;
  const Part part[] = {{ids, out}, {weights, out}, {logits, ((size_t)(T - 1) * row + E) * size},
                       {bias, bias ? (size_t)E * 4 : 0}};
  if (share(part, 2, 4)) return W4A16_ERR_SHAPE;
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  const RouteArgs a{logits, row, logits_type, bias, ids, weights, T, E, k, score,
                    groups, top_groups, group_best, renorm, scale};
  return done(launch_moe_route(a, static_cast<hipStream_t>(stream)));
}

int moe_tables(const int32_t* ids, int32_t* starts, int32_t* order, int32_t* where, int T, int k,
               int E, void* stream) {
  if (T < 0 || k < 1 || E < 1 || E > MOE_MAX_EXPERTS || (int64_t)T * k > kMaxRows)
    return W4A16_ERR_SHAPE;
  const size_t n = (size_t)T * k * 4;
  if (!starts || (n && (!ids || !order || !where))) return W4A16_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(starts, 4) || !aligned(order, 4) || !aligned(where, 4))
    return W4A16_ERR_ALIGN;
  const Part part[] = {{starts, (size_t)(E + 1) * 4}, {order, n}, {where, n}, {ids, n}};
  if (share(part, 3, 4)) return W4A16_ERR_SHAPE;
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  const TablesArgs a{ids, starts, order, where, T * k, E};
  return done(launch_moe_tables(a, static_cast<hipStream_t>(stream)));
}

int w4a16_moe_gemm(const uint16_t* A, int a_rows, const int32_t* order, int k,
                   const int32_t* starts, const uint32_t* Bpacked, const uint16_t* scales,
                   uint16_t* C, int rows, int K, int N, int group, int E, int activation,
                   int dtype, void* stream) {
  int rc = check_experts(A, a_rows, order, k, starts, Bpacked, scales, C, rows, K, N, E,
                         activation, dtype, false);
  if (rc != W4A16_OK) return rc;
  if (group <= 0 || group % kBlockK || K % group) return W4A16_ERR_GROUP;
  if (rows == 0 || N == 0) return W4A16_OK;
  const bool gate = activation == MOE_ACT_SILU_GATE;
  const int W = N * (gate ? 2 : 1);
  const size_t weights = (size_t)K * W / 2, scale_count = (size_t)(K / group) * W;
  const Part part[] = {{C, (size_t)rows * N * 2}, {A, (size_t)a_rows * K * 2},
                       {order, order ? (size_t)rows * 4 : 0}, {starts, (size_t)(E + 1) * 4},
                       {Bpacked, weights * E}, {scales, scale_count * E * 2}};
  if (share(part, 1, 6)) return W4A16_ERR_SHAPE;
  const int cus = current_cus(nullptr);
  if (cus <= 0) return W4A16_ERR_DEVICE;
  const int format = dtype == W4A16_DTYPE_BF16 ? kProdI4Bf16 : kProdI4F16;
  const ProductPlan plan = make_product_plan(format, rows, K, N, E, gate, cus);
  if (!good_plan(plan)) return W4A16_ERR_SHAPE;
  ProductArgs a{};
  a.A = reinterpret_cast<const uint8_t*>(A);
  a.order = order;
  a.starts = starts;
  a.B = reinterpret_cast<const uint8_t*>(Bpacked);
  a.S = scales;
  a.C = C;
  a.b_expert = (int64_t)weights;
  a.s_expert = (int64_t)scale_count;
  a.a_rows = a_rows;
  a.k = k;
  a.E = E;
  a.rows = rows;
  a.K = K;
  a.N = N;
  a.W = W;
  a.dtype = dtype;
  const uint32_t per = (uint32_t)(group / kBlockK);
  a.gmagic = ((1ull << 32) + per - 1) / per;
  a.tiles_n = plan.tiles_n;
  a.splits = 1;
  return done(launch_product_i4(plan, a, gate, static_cast<hipStream_t>(stream)));
}

int w8a8_moe_gemm(const uint8_t* A, const float* As, int a_rows, const int32_t* order, int k,
                  const int32_t* starts, const uint8_t* Bpacked, const float* Bs, uint16_t* C,
                  int rows, int K, int N, int E, int activation, int dtype, void* stream) {
  int rc = check_experts(A, a_rows, order, k, starts, Bpacked, Bs, C, rows, K, N, E, activation,
                         dtype, true);
  if (rc != W4A16_OK || rows == 0 || N == 0) return rc;
  if (!As) return W4A16_ERR_NULL;
  if (!aligned(As, 16)) return W4A16_ERR_ALIGN;
  const bool gate = activation == MOE_ACT_SILU_GATE;
  const int W = N * (gate ? 2 : 1);
  const size_t KB = K / kBlockK, scale_count = ((size_t)W + 127) / 128 * KB;
  const Part part[] = {{C, (size_t)rows * N * 2}, {A, (size_t)a_rows * K},
                       {As, (size_t)a_rows * KB * 4}, {order, order ? (size_t)rows * 4 : 0},
                       {starts, (size_t)(E + 1) * 4}, {Bpacked, (size_t)K * W * E},
                       {Bs, scale_count * E * 4}};
  if (share(part, 1, 7)) return W4A16_ERR_SHAPE;
  const int cus = current_cus(nullptr);
  if (cus <= 0) return W4A16_ERR_DEVICE;
  const ProductPlan plan = make_product_plan(kProdF8, rows, K, N, E, gate, cus);
  if (!good_plan(plan)) return W4A16_ERR_SHAPE;
  ProductArgs a{};
  a.A = A;
  a.As = As;
  a.order = order;
  a.starts = starts;
  a.B = Bpacked;
  a.S = Bs;
  a.C = C;
  a.b_expert = (int64_t)K * W;
  a.s_expert = (int64_t)scale_count;
  a.a_rows = a_rows;
  a.k = k;
  a.E = E;
  a.rows = rows;
  a.K = K;
  a.N = N;
  a.W = W;
  a.dtype = dtype;
  a.tiles_n = plan.tiles_n;
  a.splits = 1;
  return done(launch_product_f8(plan, a, gate, static_cast<hipStream_t>(stream)));
}

int moe_gemm_describe(int form, int rows, int K, int N, int E, int activation, int cus, char* buf,
                      size_t len) {
  if (form != 4 && form != 8) return W4A16_ERR_SHAPE;
  if (activation != MOE_ACT_NONE && activation != MOE_ACT_SILU_GATE) return W4A16_ERR_EPILOGUE;
  if (E < 1) return W4A16_ERR_SHAPE;
  return describe(form == 4 ? kProdI4F16 : kProdF8, rows, K, N, E,
                  activation == MOE_ACT_SILU_GATE, cus, buf, len);
}

int moe_combine(const uint16_t* Y, int rows, const int32_t* where, const float* weights,
                uint16_t* out, int T, int k, int N, int dtype, void* stream) {
  if (!good_dtype(dtype)) return W4A16_ERR_DTYPE;
  if (T < 0 || T > kMaxRows || k < 1 || k > MOE_MAX_TOP || N < 0 || N % 8 || N > kMaxColumns ||
      rows < 0 || rows > kMaxRows)
    return W4A16_ERR_SHAPE;
  if (T == 0 || N == 0) return W4A16_OK;
  if ((!Y && rows > 0) || !where || !weights || !out) return W4A16_ERR_NULL;
  if (!aligned(Y, 16) || !aligned(out, 16) || !aligned(where, 4) || !aligned(weights, 4))
    return W4A16_ERR_ALIGN;
  const size_t n = (size_t)T * k * 4;
  const Part part[] = {{out, (size_t)T * N * 2}, {Y, (size_t)rows * N * 2}, {where, n},
                       {weights, n}};
  if (share(part, 1, 4)) return W4A16_ERR_SHAPE;
  if (current_cus(nullptr) <= 0) return W4A16_ERR_DEVICE;
  const CombineArgs a{Y, where, weights, out, rows, T, k, N, dtype};
  return done(launch_moe_combine(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
