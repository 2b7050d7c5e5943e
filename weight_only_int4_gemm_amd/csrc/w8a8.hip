// Products in 8-bit floating point: the compiled variants of the kernels of
// product.hpp for e4m3 operands, the quantisation of activations and the
// offline permutation of weights.
#include "moe.hpp"
#include "product.hpp"
#include "product_launch.hpp"

namespace w4a16 {

hipError_t launch_product_f8(const ProductPlan& plan, const ProductArgs& a, bool gate,
                             hipStream_t stream) {
  return launch_product<kProdF8>(plan, a, gate, stream);
}

namespace {

// A thread moves 16 codes at a time: 16-byte piece i of the permuted matrix.
__global__ __launch_bounds__(256) void w8a8_repack_kernel(const uint8_t* __restrict__ B,
                                                          uint8_t* __restrict__ Bp, int K,
                                                          int64_t pieces) {
  const int KB = K / kBlockK;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces;
       i += (int64_t)gridDim.x * 256) {
    const int lane = (int)(i & 63), half = (int)(i >> 6) & 1;
    const int64_t block = i >> 7;
    const int64_t n16 = block / KB, kb = block - n16 * KB;
    const int64_t from =
        (n16 * 16 + (lane & 15)) * K + kb * kBlockK + half * 64 + (lane >> 4) * 16;
    reinterpret_cast<uint4*>(Bp)[i] = *reinterpret_cast<const uint4*>(B + from);
  }
}

// 16 lanes hold one block of 128 values, eight each.  The largest magnitude
// is found on the bit patterns: as whole numbers they order finite values,
// infinity and NaN as wanted.
//
// What bounds it: bandwidth (3 bytes a value).
template <bool BF16>
__global__ __launch_bounds__(256) void w8a8_quantize_kernel(const uint16_t* __restrict__ X,
                                                            int64_t x_row,
                                                            uint8_t* __restrict__ Xq,
                                                            float* __restrict__ Xs, int KB,
                                                            int64_t blocks) {
  const int sub = threadIdx.x & 15;
  const int64_t step = (int64_t)gridDim.x * 16;
  for (int64_t b = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); b < blocks; b += step) {
    const int64_t t = b / KB, kb = b - t * KB;
    const uint4 v = *reinterpret_cast<const uint4*>(X + t * x_row + kb * kBlockK + sub * 8);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[8];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t h = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
      x[i] = scale16(h, BF16);
      const uint32_t m = __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu;
      most = m > most ? m : most;
    }
#pragma unroll
    for (int d = 1; d < 16; d *= 2) {
      const uint32_t o = __shfl_xor(most, d);
      most = o > most ? o : most;
    }
    const bool finite = most < 0x7f800000u;
    float scale = __builtin_bit_cast(float, most) / 448.f;
    scale = scale > 0x1p-126f ? scale : 0x1p-126f;
    const float inv = 1.f / scale;
    int q[2] = {0, 0};
    if (finite) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i] * inv, x[4 * i + 1] * inv, q[i], false);
        q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2] * inv, x[4 * i + 3] * inv, q[i], true);
      }
    }
    *reinterpret_cast<int2*>(Xq + b * kBlockK + sub * 8) = int2{q[0], q[1]};
    if (sub == 0) Xs[b] = finite ? scale : __builtin_nanf("");
  }
}

}  // namespace

hipError_t launch_w8a8_repack(const uint8_t* B, uint8_t* Bp, int K, int N, hipStream_t stream) {
  const int64_t pieces = (int64_t)K * N / 16;
  const int64_t groups = (pieces + 255) / 256;
  hipLaunchKernelGGL(w8a8_repack_kernel, dim3((unsigned)(groups < 65536 ? groups : 65536)),
                     dim3(256), 0, stream, B, Bp, K, pieces);
  return hipGetLastError();
}

hipError_t launch_w8a8_quantize(const uint16_t* X, int64_t x_row, uint8_t* Xq, float* Xs, int T,
                                int K, int dtype, hipStream_t stream) {
  const int64_t blocks = (int64_t)T * (K / kBlockK);
  const int64_t groups = (blocks + 15) / 16;
  const dim3 grid((unsigned)(groups < 16384 ? groups : 16384));
  if (dtype == W4A16_DTYPE_BF16)
    hipLaunchKernelGGL((w8a8_quantize_kernel<true>), grid, dim3(256), 0, stream, X, x_row, Xq, Xs,
                       K / kBlockK, blocks);
  else
    hipLaunchKernelGGL((w8a8_quantize_kernel<false>), grid, dim3(256), 0, stream, X, x_row, Xq, Xs,
                       K / kBlockK, blocks);
  return hipGetLastError();
}

}  // namespace w4a16
