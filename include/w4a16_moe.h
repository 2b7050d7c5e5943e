/*
 * w4a16_moe.h -- layers of experts of libw4a16 (gfx950): routing, row tables,
 * the products of each row with its own expert's 4-bit or 8-bit weights, and
 * the weighted sum over a token's experts.
 *
 *   moe_route        router logits -> ids and weights of each token's k experts
 *   moe_tables       ids -> rows sorted by expert
 *   w4a16_moe_gemm   (or w8a8_moe_gemm) with MOE_ACT_SILU_GATE: tokens -> the
 *                    experts' inner rows, gathered on the way in
 *   w4a16_moe_gemm   (or w8a8_quantize and w8a8_moe_gemm) -> output rows
 *   moe_combine      output rows -> tokens
 *
 * The conventions of w4a16.h hold for every entry point: 16-bit values travel
 * as uint16_t, `stream` is a hipStream_t, pointers marked "device" are memory
 * of the current HIP device, arguments are checked before anything is
 * launched, nothing is allocated, synchronised or printed, and every call can
 * be captured into a HIP graph (how many rows an expert has is read on the
 * device).  Status codes are those of enum w4a16_status.  Buffers of one call
 * do not overlap.  Index tensors are read with bounds: whatever they hold, no
 * call touches memory outside its tensors.
 */
#ifndef W4A16_MOE_H
#define W4A16_MOE_H

#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"
#include "w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_TOP 32
#define MOE_MAX_GROUPS 64

/* How a logit becomes a score. */
enum moe_score {
    MOE_SOFTMAX = 0, /* softmax over the token's experts                      */
    MOE_SIGMOID = 1  /* 1 / (1 + exp(-x)) of each                             */
};

/* Types of the logits. */
enum moe_logits {
    MOE_LOGITS_F16 = 0,
    MOE_LOGITS_BF16 = 1,
    MOE_LOGITS_F32 = 2
};

/* What w4a16_moe_gemm and w8a8_moe_gemm do to a row's sums. */
enum moe_activation {
    MOE_ACT_NONE = 0,     /* y[n] = x[n]                                      */
    MOE_ACT_SILU_GATE = 1 /* y[n] = x[n] / (1 + exp(-x[n])) * x[N + n]        */
};

/*
 * moe_route -- the experts of each token and their weights.
 *
 * For each token, over its E experts:
 *   s = score of the logits,  c = s + bias
 *   an expert is eligible unless its logit is -infinity or NaN, or c is
 *   -infinity or NaN (where every logit that counts is +infinity, softmax
 *   shares 1 among these);
 *   with groups > 1 the experts are `groups` runs of E / groups; a group's
 *   mark is the sum of its group_best highest eligible c (fewer, if it has
 *   fewer); the top_groups groups of the highest marks keep their experts,
 *   the others' are not eligible (ties keep the lower group);
 *   ids     = the k eligible experts of the highest c, highest first, ties
 *             to the lowest id;
 *   weights = s of these; with renorm divided by their sum (0 if that is 0);
 *             times scale.
 * Where fewer than k experts are eligible the rest of the row is id -1 and
 * weight 0, which every other call here leaves out.
 *
 * Without bias, and without marks of two summed, experts are compared by
 * their logits, whose order is that of the scores; otherwise marks and c are
 * 64-bit numbers.  So are the scores of a sigmoid, which are 0 for logits
 * below -709, and with bias or marks of two those of a softmax too; else a
 * softmax is in FP32.  Weights are FP32.
 *
 * logits  (device, read)  [T] rows of E values of type logits_type (enum
 *         moe_logits), `row` elements apart (at least E where T > 1), aligned
 *         to their size.
 * bias    (device, read)  FP32 [E], or NULL for none.
 * ids     (device, write) int32 [T][k].   weights (device, write) FP32 [T][k].
 * T       >= 0 (0: nothing is launched).
 * E       1..MOE_MAX_EXPERTS.   k  1..MOE_MAX_TOP, at most E.
 * groups  1..MOE_MAX_GROUPS, a divisor of E.   top_groups  1..groups.
 * group_best  1 or 2.
 * Errors: W4A16_ERR_NULL, _SHAPE (sizes, enums and overlaps), _DTYPE
 *         (logits_type), _ALIGN, _DEVICE, _LAUNCH.
 */
int moe_route(const void* logits, int64_t row, int logits_type, const float* bias, int32_t* ids,
              float* weights, int T, int E, int k, int score, int groups, int top_groups,
              int group_best, int renorm, float scale, void* stream);

/*
 * moe_tables -- the T * k choices of a routing sorted by expert.
 *
 * Choice i = t * k + j is entry j of token t.  Choices of one expert stay in
 * their order; choices whose id is not in 0..E-1 (none, or an expert of
 * another device) are left out.
 *
 * ids    (device, read)  int32 [T][k].
 * starts (device, write) int32 [E + 1]: expert e has the sorted positions
 *        starts[e] .. starts[e + 1] - 1; starts[E] choices are kept.
 * order  (device, write) int32 [T * k]: the choice at each sorted position;
 *        positions from starts[E] on are set to -1.
 * where  (device, write) int32 [T][k]: the sorted position of each choice, -1
 *        for those left out.
 * T      >= 0, T * k at most 2^24 (T = 0 sets starts to zeros).
 * Errors: W4A16_ERR_NULL, _SHAPE, _ALIGN (4 bytes), _DEVICE, _LAUNCH.
 */
int moe_tables(const int32_t* ids, int32_t* starts, int32_t* order, int32_t* where, int T, int k,
               int E, void* stream);

/*
 * w4a16_moe_gemm -- each sorted row times its expert's 4-bit weights.
 *
 *   C[p] = act(A[row(p)] . dequant(expert e)),  starts[e] <= p < starts[e + 1]
 *   row(p) = order[p] / k, or p where order is NULL
 *
 * A       (device, read)  `dtype` [a_rows][K]; a_rows >= rows without order.
 * order   (device, read)  int32 [rows] from moe_tables, or NULL.  An entry
 *         outside 0 .. a_rows * k - 1 stands for row 0.
 * starts  (device, read)  int32 [E + 1]; values are taken within 0 .. rows.
 * Bpacked (device, read)  E matrices, one after the other, each the output of
 *         w4a16_repack for (K, W); W = N, or 2 N with MOE_ACT_SILU_GATE: the
 *         N gate columns, then the N up columns.
 * scales  (device, read)  `dtype` [E][K/group][W].
 * C       (device, write) `dtype` [rows][N]; rows outside every expert's
 *         range keep what they hold.
 * rows    >= 0, K a positive multiple of 128, N >= 0 a multiple of 16 (0 rows
 *         or columns: nothing is launched), group a multiple of 128 that
 *         divides K, E 1..MOE_MAX_EXPERTS, k >= 1, a_rows >= 1.  At most 2^24
 *         rows and a_rows, K 2^20, W 2^24, K * W 2^36.
 * Numerics: products accumulate in FP32; the exact (q - 8) are multiplied and
 *         the scales go onto the FP32 sums of 128; the activation is in FP32,
 *         C rounded once.  BF16 codes enter as 128 + q, 136 times the row's
 *         sum taken off: a row of A that holds an infinity gives NaN where
 *         the product would be infinite too, and one with values of 2^112
 *         and more may.
 * Errors: W4A16_ERR_NULL, _SHAPE (sizes, overlaps), _GROUP, _ALIGN (16 bytes;
 *         order and starts 4), _DTYPE, _EPILOGUE (activation), _DEVICE,
 *         _LAUNCH.
 */
int w4a16_moe_gemm(const uint16_t* A, int a_rows, const int32_t* order, int k,
                   const int32_t* starts, const uint32_t* Bpacked, const uint16_t* scales,
                   uint16_t* C, int rows, int K, int N, int group, int E, int activation,
                   int dtype, void* stream);

/*
 * w8a8_moe_gemm -- the same with e4m3 activations and weights (w8a8.h).
 *
 * A       (device, read)  e4m3 [a_rows][K].  As (device, read) FP32 [a_rows][K/128].
 * Bpacked (device, read)  E outputs of w8a8_repack for (K, W).
 * Bs      (device, read)  FP32 [E][ceil(W/128)][K/128].
 * With MOE_ACT_SILU_GATE N is a multiple of 32.  Everything else as
 * w4a16_moe_gemm and w8a8_gemm.
 */
int w8a8_moe_gemm(const uint8_t* A, const float* As, int a_rows, const int32_t* order, int k,
                  const int32_t* starts, const uint8_t* Bpacked, const float* Bs, uint16_t* C,
                  int rows, int K, int N, int E, int activation, int dtype, void* stream);

/* How w4a16_moe_gemm (form 4) or w8a8_moe_gemm (form 8) would run these
 * sizes, as w4a16_describe.  cus: compute units of the device it is for; 0
 * asks the current device.  W4A16_ERR_SHAPE also for another form. */
int moe_gemm_describe(int form, int rows, int K, int N, int E, int activation, int cus, char* buf,
                      size_t len);

/*
 * moe_combine -- the weighted sum of a token's rows.
 *
 *   out[t][n] = sum_j weights[t][j] * Y[where[t][j]][n]
 *
 * in FP32, in the order of j, rounded once; entries of `where` outside
 * 0 .. rows - 1 are left out, whatever their weight (a token with no entry
 * gets zeros).
 *
 * Y       (device, read)  `dtype` [rows][N].
 * where   (device, read)  int32 [T][k].   weights (device, read) FP32 [T][k].
 * out     (device, write) `dtype` [T][N].
 * T       >= 0, N 0..2^24 a multiple of 8 (0 of either: nothing is launched),
 *         k 1..MOE_MAX_TOP, rows >= 0 (Y may be NULL for 0).
 * Errors: W4A16_ERR_NULL, _SHAPE, _ALIGN (16 bytes; where and weights 4),
 *         _DTYPE, _DEVICE, _LAUNCH.
 */
int moe_combine(const uint16_t* Y, int rows, const int32_t* where, const float* weights,
                uint16_t* out, int T, int k, int N, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_MOE_H */
