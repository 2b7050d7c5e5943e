/*
 * w4a16_kv4.h -- the paged 4-bit key/value cache of libw4a16 (gfx950): page
 * tables from request lengths, rotary positions, the quantising append, and
 * attention over the cache.  It stands between the qkv and the output
 * product of a layer whose weights w4a16_gemm multiplies.
 *
 * The conventions of w4a16.h hold for every entry point: 16-bit values
 * travel as uint16_t, `stream` is a hipStream_t, pointers marked "device"
 * are memory of the current HIP device, arguments are checked before
 * anything is launched, nothing is allocated, synchronised or printed, and
 * every call can be captured into a HIP graph.  Status codes are those of
 * enum w4a16_status.  `dtype` is W4A16_DTYPE_F16 or W4A16_DTYPE_BF16 and
 * covers every 16-bit tensor of a call; the cache does not depend on it.
 * What a call writes shares no element with what else it reads or writes,
 * save where an argument "may be" another; strided tensors may be parts of
 * one buffer, side by side or interleaved by head or token (with strides
 * alike, or rows apart within equal token strides).
 *
 * The stored form.  One token's keys (or values) of one head are a row
 * x[0..D).  With all arithmetic in FP32, round half to even, no contraction:
 *
 *   scale  = fp16((max x - min x) * fp32(1/15))          at most 65504
 *   offset = fp16(min x + 8 * scale)                     within +-65504
 *   q      = clamp(rint((x - offset) * (1 / scale)) + 8, 0, 15)
 *            (8 where scale is 0)
 *   value  = (q - 8) * scale + offset
 *
 * A row that holds an infinity or a NaN is stored with scale = offset = NaN
 * and reads back as NaN throughout.
 *
 * The cache of one layer: bytes [pages][heads][page][D + 8], D in {64, 128,
 * 256}, page (tokens of a page) a power of two in 16..1024, pages * page at
 * most 2^31 - 1.  A (page, head) is page / 16 units of 16 tokens, each
 * 16 D + 128 bytes:
 *
 *   8 D   key codes, uint32 [16 tokens][D/8]
 *   8 D   value codes, uint32 [4][D/8][4]: token 4 g + j of the unit, word w
 *         at [g][w][j]
 *   64    key FP16 pairs (scale, offset) [16]
 *   64    value FP16 pairs (scale, offset) [16]
 *
 * Word w of a row holds channels 8 w .. 8 w + 7, the lowest in the lowest
 * four bits.  The keys of 16 tokens and the values of four tokens by four
 * lanes are then exactly one 16-byte load per lane for the 16x16x32 matrix
 * instruction, and one token's append writes whole words only.
 *
 * A slot is page_id * page + token_in_page; slot -1 means "nowhere".
 */
#ifndef W4A16_KV4_H
#define W4A16_KV4_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the channels of a rotation are paired. */
enum kv4_rope_pairs {
    KV4_ROPE_HALVES = 0,  /* pair i = channels (i, i + rot/2)                */
    KV4_ROPE_PAIRS = 1    /* pair i = channels (2 i, 2 i + 1)                */
};

/* The most requests of one kv4_tables call. */
#define KV4_MAX_REQUESTS 4096

/* Version of the stored form above. */
int kv4_layout_version(void);

/* Bytes of a cache: pages * heads * page * (D + 8); 0 for sizes that no
 * cache has. */
size_t kv4_cache_bytes(int pages, int heads, int D, int page);

/*
 * kv4_tables -- page tables, slots and positions of a scheduler step, from
 * the lengths the requests have and the lengths they shall have.
 *
 * Free pages wait in a first-in-first-out ring: state = {head, count,
 * refused, 0}, the free pages are ring[(head + i) % pages], i < count.  With
 * old/new the pages that lens/want tokens take, the requests in order:
 *  - want > lens: takes new - old pages from the head of the ring, in
 *    request order, and writes them to table[b][old .. new).  If the pages
 *    wanted up to and including this request exceed `count`, new exceeds
 *    max_pages, or its new tokens do not all lie below `capacity` (see
 *    q_start), the request is refused: it keeps its length and pages.
 *  - want < lens: pages new .. old of its row go to the tail of the ring
 *    (available to the next call); the row's entries beyond new stay as
 *    they are and mean nothing.
 * lens_out[b] is want[b], or lens[b] if refused.  state_out is the new
 * {head, count, number refused, 0}.  q_start[b] counts the new tokens
 * (max(0, want - lens), refused or not) of the requests before b, limited
 * to `capacity`; new token i of request b is token t = q_start[b] + i:
 * positions[t] = lens[b] + i and slots[t] is its place in the cache, -1 if
 * refused or if its page id is outside the cache.  Entries from q_start[B]
 * to capacity get slot -1, position 0.  So every token below lens_out[b] has
 * a slot, now or from an earlier call.  The rows of a refused request still
 * count in q_start: its tokens are not stored, and kv4_attention computes its
 * queries over the tokens it holds (the last at position lens_out[b] - 1),
 * results that mean nothing.
 *
 * lens, want (device, read) int32 [B]; lengths below 0 count as 0, lens
 * above max_pages * page as that.  table (device, read and written) int32
 * [B][max_pages]; ring (device, read and written) int32 [pages]; state
 * (device, read) int32 [4]; lens_out (device, write) int32 [B], may be lens;
 * state_out (device, write) int32 [4], may be state, element 3 zero on
 * entry (it is a work counter that every call leaves at zero); q_start
 * (device, write) int32 [B + 1]; slots, positions (device, write) int32
 * [capacity].  4-byte alignment.  0 <= B <= KV4_MAX_REQUESTS.
 */
int kv4_tables(const int32_t* lens, const int32_t* want, int32_t* table, int max_pages,
               int32_t* ring, int pages, const int32_t* state, int32_t* lens_out,
               int32_t* state_out, int32_t* q_start, int32_t* slots, int32_t* positions,
               int capacity, int B, int page, void* stream);

/*
 * kv4_rope -- rotary positions over one to three axes.
 *
 * The first rot = 2 * (sections[0] + ... + sections[axes - 1]) channels of
 * every row of X turn pairwise; the others are copied.  Pair i belongs to
 * the axis a whose section holds i (the first sections[0] pairs to axis 0,
 * and so on) and turns by positions[a][t] * inv_freq[i] radians:
 *   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin).
 * Angles are formed and reduced in FP64, cos and sin rounded to FP32, the
 * products and the sum FP32 without contraction, the result rounded once.
 *
 * X (device, read), Y (device, write): 16-bit [T][H][D] with token and head
 * strides in elements, multiples of 8, and contiguous channels; 16-byte
 * aligned.  Y may be X (the same strides).  positions (device, read) int32
 * [axes][T], row a at positions + a * pos_stride.  inv_freq (device, read)
 * FP64 [rot/2].  sections: host array of `axes` counts.  rot a positive
 * multiple of 16, at most D.  T at most 2^26 - 4, here and in both appends.
 */
int kv4_rope(const uint16_t* X, int64_t x_token, int64_t x_head, uint16_t* Y, int64_t y_token,
             int64_t y_head, const int32_t* positions, int64_t pos_stride,
             const double* inv_freq, const int* sections, int axes, int pairs, int T, int H,
             int D, int dtype, void* stream);

/*
 * kv4_append -- quantise keys and values and store them at their slots.
 *
 * K, V (device, read) 16-bit [T][H][D], strides and alignment as in
 * kv4_rope.  slots (device, read) int32 [T]; a token whose slot is outside
 * [0, pages * page) is skipped; two tokens of a call must not share a slot.
 * cache (device, write), 16-byte aligned.
 */
int kv4_append(const uint16_t* K, int64_t k_token, int64_t k_head, const uint16_t* V,
               int64_t v_token, int64_t v_head, const int32_t* slots, uint8_t* cache, int T,
               int H, int D, int pages, int page, int dtype, void* stream);

/*
 * kv4_rope_append -- kv4_rope of Q into Qout and kv4_append in one launch,
 * the keys rotated on the way (and not rounded to 16 bits in between).
 *
 * Q, Qout [T][Hq][D], K, V [T][H][D]; Qout may be Q.  Hq may be 0 (Q and
 * Qout NULL).  Other arguments as in kv4_rope and kv4_append.  Queries are
 * rotated whatever the token's slot is.
 */
int kv4_rope_append(const uint16_t* Q, int64_t q_token, int64_t q_head, const uint16_t* K,
                    int64_t k_token, int64_t k_head, const uint16_t* V, int64_t v_token,
                    int64_t v_head, uint16_t* Qout, int64_t qo_token, int64_t qo_head,
                    const int32_t* positions, int64_t pos_stride, const double* inv_freq,
                    const int* sections, int axes, int pairs, const int32_t* slots,
                    uint8_t* cache, int T, int Hq, int H, int D, int pages, int page, int dtype,
                    void* stream);

/*
 * kv4_dequant_debug -- the values the cache holds at `slots`, rounded to 16
 * bits: K, V (device, write) [T][H][D] contiguous, 16-byte aligned.  Tokens
 * without a slot read as zeros.
 */
int kv4_dequant_debug(const int32_t* slots, const uint8_t* cache, uint16_t* K, uint16_t* V,
                      int T, int H, int D, int pages, int page, int dtype, void* stream);

/*
 * kv4_attention -- causal attention of new queries over the cache.
 *
 * Request b holds lens[b] tokens, token j at page table[b][j / page].  Its
 * queries are rows q_start[b] .. q_start[b + 1] of Q (q_start NULL: one
 * query per request, row b); the last is at position lens[b] - 1, and the
 * query at position p sees the keys j with p - window < j <= p (window 0:
 * all j <= p).  Query head h reads key/value head h / (Hq / H).
 *
 *   O = sum_j softmax_j(scale * q . k_j) v_j,   lse = log sum_j exp(scale * q . k_j)
 *
 * A query that sees no key gets O = 0, lse = -inf.  Tokens whose table
 * entry is outside [0, pages) count as not seen.  Nothing that the masked
 * parts of the cache hold reaches a result.  Codes multiply exactly and
 * sums are FP32; the only roundings to 16 bits are the probability times
 * the value's scale (to FP16; for FP16 calls the remainder is carried too)
 * and the output.  A query's size costs other queries no precision; logits
 * beyond FP32's integers (2^24) are told apart as far as FP32 does, and the
 * largest keeps its weight.  A logit (base 2) beyond FP32's range counts as
 * that infinity: no weight below it, a NaN above.
 *
 * Q (device, read), O (device, write): 16-bit [T][Hq][D], token and head
 * strides in elements, multiples of 8, contiguous channels, 16-byte
 * aligned; rows that no request has are not written.  lse (device, write)
 * FP32 [T][Hq] or NULL.  table int32 [B][max_pages], lens int32 [B]
 * (below 0 counts as 0, above max_pages * page as that), q_start int32
 * [B + 1], ascending, within [0, T]; device, read.  scale > 0.
 *
 * max_q: no request has more queries (rows beyond are not computed).  Sizes
 * that come to 2^24 or more workgroups (requests times key/value heads times
 * tiles of 128 query rows of max_q, of 16 or 8 where those are few) are
 * refused.
 * max_len: the length the work is planned for; longer requests are right
 * too, only slower.  workspace as in w4a16_workspace_bytes: at least
 * kv4_attention_workspace_bytes, zero-filled once, left ready for the next
 * call, may be shared with the GEMMs of the same stream; NULL if 0 bytes.
 */
int kv4_attention(const uint16_t* Q, int64_t q_token, int64_t q_head, const uint8_t* cache,
                  const int32_t* table, int max_pages, const int32_t* lens,
                  const int32_t* q_start, uint16_t* O, int64_t o_token, int64_t o_head,
                  float* lse, int T, int B, int Hq, int H, int D, int pages, int page,
                  float scale, int window, int max_q, int max_len, int dtype, void* workspace,
                  void* stream);

/* Workspace bytes of kv4_attention on the current device, at most 192 MiB;
 * 0 if the call needs none (or rejects the sizes). */
size_t kv4_attention_workspace_bytes(int B, int Hq, int H, int D, int max_q, int max_len,
                                     int window);

/* One line on how kv4_attention would run, as w4a16_describe, for a device
 * with `cus` compute units (0: the current device). */
int kv4_attention_describe(int B, int Hq, int H, int D, int max_q, int max_len, int window,
                           int cus, char* buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_KV4_H */
