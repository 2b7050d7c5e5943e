// Declarations of the expert layers and 8-bit products (include/w4a16_moe.h,
// include/w8a8.h) shared by their translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace w4a16 {

struct ProductArgs;

// How one product is cut into work.
//  tile     0: the streaming kernel, 1: the tile kernel
//  mb, nb   16-row and 16-column blocks of a wave
//  waves    tile kernel: along columns; streaming kernel: that divide K
//  tm, tn   rows of a workgroup and its output columns
//  tiles_m  the most row tiles; splits: K ranges of a tile (tile kernel)
struct ProductPlan {
  int tile, mb, nb, waves, depth;
  int tm, tn, tiles_m, tiles_n, splits;
  size_t workspace_bytes;
};

// format: kProdF8 ... (product.hpp); E = 0: a matrix product of `rows` rows
// (which may split K), else the rows of E experts.
ProductPlan make_product_plan(int format, int rows, int K, int N, int E, bool gate, int cus);

hipError_t launch_product_f8(const ProductPlan& plan, const ProductArgs& a, bool gate,
                             hipStream_t stream);
hipError_t launch_product_i4(const ProductPlan& plan, const ProductArgs& a, bool gate,
                             hipStream_t stream);

hipError_t launch_w8a8_repack(const uint8_t* B, uint8_t* Bp, int K, int N, hipStream_t stream);
hipError_t launch_w8a8_quantize(const uint16_t* X, int64_t x_row, uint8_t* Xq, float* Xs, int T,
                                int K, int dtype, hipStream_t stream);

struct RouteArgs {
  const void* logits;
  int64_t row;
  int type;
  const float* bias;
  int32_t* ids;
  float* weights;
  int T, E, k, score, groups, top_groups, group_best, renorm;
  float scale;
};
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream);

struct TablesArgs {
  const int32_t* ids;
  int32_t *starts, *order, *where;
  int n, E;
};
hipError_t launch_moe_tables(const TablesArgs& a, hipStream_t stream);

struct CombineArgs {
  const uint16_t* Y;
  const int32_t* where;
  const float* weights;
  uint16_t* out;
  int rows, T, k, N, dtype;
};
hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t stream);

}  // namespace w4a16
