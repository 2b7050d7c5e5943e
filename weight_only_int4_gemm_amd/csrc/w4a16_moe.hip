// Products of rows with their own expert's 4-bit weights: the compiled
// variants of the kernels of product.hpp for FP16 and BF16.
#include "moe.hpp"
#include "product.hpp"
#include "product_launch.hpp"

namespace w4a16 {

hipError_t launch_product_i4(const ProductPlan& plan, const ProductArgs& a, bool gate,
                             hipStream_t stream) {
  return a.dtype == W4A16_DTYPE_BF16 ? launch_product<kProdI4Bf16>(plan, a, gate, stream)
                                     : launch_product<kProdI4F16>(plan, a, gate, stream);
}

}  // namespace w4a16
