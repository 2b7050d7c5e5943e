/*
 * w8a8.h -- products in 8-bit floating point of libw4a16 (gfx950): the
 * quantisation of 16-bit activations, the offline permutation of weights and
 *
 *   C[m][n] = sum_kb As[m][kb] * Bs[n/128][kb] * sum_{k in block kb} A[m][k] * B[n][k]
 *
 * A [M][K] and B [N][K] hold e4m3 codes (OCP 8-bit floating point: 4 exponent
 * bits, 3 fraction bits, largest value 448, no infinities, 0x7f and 0xff are
 * NaN), block kb is in-features 128 kb .. 128 kb + 127, As one FP32 scale for
 * each row and block, Bs one for each 128 x 128 block of weights.
 *
 * The conventions of w4a16.h hold for every entry point: 16-bit values travel
 * as uint16_t, codes as uint8_t, `stream` is a hipStream_t, pointers marked
 * "device" are memory of the current HIP device, arguments are checked before
 * anything is launched, nothing is allocated, synchronised or printed, and
 * every call can be captured into a HIP graph.  Status codes are those of
 * enum w4a16_status.  `dtype` is W4A16_DTYPE_F16 or W4A16_DTYPE_BF16.
 * Pointers are 16-byte aligned, buffers of one call do not overlap.
 */
#ifndef W8A8_H
#define W8A8_H

#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of the permuted layout written by w8a8_repack. */
int w8a8_layout_version(void);

/* Bytes of the permuted weights for an N x K matrix: K * N (0 for sizes that
 * w8a8_repack refuses). */
size_t w8a8_packed_bytes(int K, int N);

/*
 * w8a8_repack -- offline permutation of e4m3 weights into the order in which
 * the matrix instruction's lanes take them.
 *
 * B       (device, read)  e4m3 [N][K] row-major (out-features x in-features).
 * Bpacked (device, write) K * N bytes, layout version 1: code (n, k) is byte
 *                           ((n/16 * K/128 + k/128) * 2 + k%128/64) * 1024
 *                           + (n%16 + 16 * (k%64/16)) * 16 + k%16.
 * K       positive multiple of 128, at most 2^20.   N  positive multiple of 16,
 *         at most 2^24.   K * N at most 2^36.
 * Errors: W4A16_ERR_NULL, _SHAPE (sizes, or B and Bpacked overlapping),
 *         _ALIGN, _DEVICE, _LAUNCH.
 */
int w8a8_repack(const uint8_t* B, uint8_t* Bpacked, int K, int N, void* stream);

/*
 * w8a8_quantize -- 16-bit rows to e4m3 codes with one scale per 128.
 *
 * In FP32, each operation rounded to nearest even:
 *   scale = max(max |x| / 448, 2^-126)     over the 128 values of a block
 *   code  = e4m3(x * (1 / scale))          to nearest even
 * A block that holds an infinity or a NaN gets the scale NaN and codes 0: it
 * stands for NaN throughout.
 *
 * X  (device, read)  `dtype` [T] rows of K values, x_row elements apart
 *                    (a multiple of 8, at least K where T > 1).
 * Xq (device, write) e4m3 [T][K].
 * Xs (device, write) FP32 [T][K/128].
 * T  >= 0 (0: nothing is launched).  K  positive multiple of 128.
 * Errors: W4A16_ERR_NULL, _SHAPE, _ALIGN, _DTYPE, _DEVICE, _LAUNCH.
 */
int w8a8_quantize(const uint16_t* X, int64_t x_row, uint8_t* Xq, float* Xs, int T, int K,
                  int dtype, void* stream);

/*
 * w8a8_workspace_bytes -- bytes of workspace w8a8_gemm needs for this shape
 * on the current device; 0 where it needs none or refuses the shape.  The
 * contract is that of w4a16_workspace_bytes: zero-filled once after
 * allocating, then it serves calls of any shape it covers, one at a time.
 */
size_t w8a8_workspace_bytes(int M, int K, int N);

/* The plan of w8a8_gemm for this shape, as w4a16_describe.  cus: compute
 * units of the device it is for; 0 asks the current device. */
int w8a8_describe(int M, int K, int N, int cus, char* buf, size_t len);

/*
 * w8a8_gemm -- the product above.
 *
 * A         (device, read)  e4m3 [M][K].   As (device, read)  FP32 [M][K/128].
 * Bpacked   (device, read)  output of w8a8_repack for (K, N).
 * Bs        (device, read)  FP32 [ceil(N/128)][K/128].
 * C         (device, write) `dtype` [M][N].
 * M         >= 0, N >= 0 a multiple of 16 (0 of either: nothing is launched),
 *           K a positive multiple of 128; K and N as w8a8_repack takes them, M at
 *           most 2^24.
 * workspace (device, read/write) see w8a8_workspace_bytes; may be NULL only
 *           where that returns 0.
 * Numerics: the products of a block are summed by the matrix instruction in
 *           FP32, its sum is scaled and added in FP32, C is rounded once (to
 *           nearest even; overflow gives infinity).  The order of the
 *           summation depends on the shape alone: equal inputs give
 *           bit-identical C.
 * Errors:   W4A16_ERR_NULL, _SHAPE, _ALIGN, _DTYPE, _WORKSPACE, _DEVICE,
 *           _LAUNCH.
 */
int w8a8_gemm(const uint8_t* A, const float* As, const uint8_t* Bpacked, const float* Bs,
              uint16_t* C, int M, int K, int N, int dtype, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_H */
