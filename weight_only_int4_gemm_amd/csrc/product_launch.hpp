// The compiled variants of product.hpp's kernels and their launch.
#pragma once

#include "moe.hpp"
#include "product.hpp"

namespace w4a16 {

// Streaming kernel: (MB, NB, WAVES, DEPTH); NB is even where gate and up
// columns share a workgroup.  e4m3, 4 bits (experts only).
#define W4A16_STREAM_F8(X) X(1, 1, 8, 4) X(1, 2, 4, 4) X(2, 1, 8, 3)
#define W4A16_STREAM_I4(X) X(1, 2, 8, 3) X(1, 4, 4, 3)
// Tile kernel: (MB, NB, WAVES, whether experts take it, with the gate too).
#define W4A16_TILE_F8(X) \
  X(2, 1, 4, 0) X(2, 2, 4, 1) X(4, 1, 4, 0) X(4, 2, 4, 1) X(8, 2, 4, 0) X(8, 4, 4, 1)
#define W4A16_TILE_I4(X) X(2, 2, 4, 1) X(4, 4, 4, 1)

template <int F>
hipError_t launch_product(const ProductPlan& plan, const ProductArgs& a, bool gate,
                          hipStream_t stream) {
  if (plan.tile == 0) {
    const dim3 grid((unsigned)((int64_t)plan.tiles_m * plan.tiles_n)), block(64 * plan.waves);
#define W4A16_CASE(MB_, NB_, WAVES_, DEPTH_)                                                      \
  if (plan.mb == MB_ && plan.nb == NB_ && plan.waves == WAVES_ && plan.depth == DEPTH_) {            \
    if (gate) {                                                                                   \
      if constexpr (NB_ % 2 == 0)                                                                 \
        hipLaunchKernelGGL((product_stream_kernel<F, MB_, NB_, WAVES_, DEPTH_, true>), grid,      \
                           block, 0, stream, a);                                                  \
      else                                                                                        \
        return hipErrorInvalidValue;                                                              \
    } else                                                                                        \
      hipLaunchKernelGGL((product_stream_kernel<F, MB_, NB_, WAVES_, DEPTH_, false>), grid,       \
                         block, 0, stream, a);                                                    \
    return hipGetLastError();                                                                     \
  }
    if constexpr (F == kProdF8) {
      W4A16_STREAM_F8(W4A16_CASE)
    } else {
      W4A16_STREAM_I4(W4A16_CASE)
    }
#undef W4A16_CASE
    return hipErrorInvalidValue;
  }
  const dim3 grid((unsigned)((int64_t)plan.tiles_m * plan.tiles_n), (unsigned)plan.splits);
  const dim3 block(64 * plan.waves);
#define W4A16_CASE(MB_, NB_, WAVES_, GATE_)                                                     \
  if (plan.mb == MB_ && plan.nb == NB_ && plan.waves == WAVES_) {                               \
    if (gate) {                                                                                 \
      if constexpr (GATE_)                                                                      \
        hipLaunchKernelGGL((product_tile_kernel<F, MB_, NB_, WAVES_, true>), grid, block, 0,    \
                           stream, a);                                                          \
      else                                                                                      \
        return hipErrorInvalidValue;                                                            \
    } else                                                                                      \
      hipLaunchKernelGGL((product_tile_kernel<F, MB_, NB_, WAVES_, false>), grid, block, 0,     \
                         stream, a);                                                            \
    return hipGetLastError();                                                                   \
  }
  if constexpr (F == kProdF8) {
    W4A16_TILE_F8(W4A16_CASE)
  } else {
    W4A16_TILE_I4(W4A16_CASE)
  }
#undef W4A16_CASE
  return hipErrorInvalidValue;
}

}  // namespace w4a16
