/*
 * moe_decode.h -- the entry points of libmoe.so for decoding: weights in 4
 * bits with group scales, a linear layer on them, and the whole expert layer
 * of moe.h (A1 to A7) for a few tokens in two kernels, with the experts'
 * weights in bf16 or in 4 bits.  The conventions of moe.h hold: device
 * pointers owned by the caller and 16-byte aligned unless said otherwise, no
 * allocation, no synchronisation, asynchronous on `stream`, arguments checked
 * on the host.  Every result is the same on every call.
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Weights in 4 bits with one float32 scale per group of `group` (32, 64 or
 * 128) consecutive values of a row; a row's last group is shorter when cols is
 * no multiple of it.  Per group: m = max |w|, scale = m / 7 in float32,
 * code = 7 w / m rounded to the nearest integer, ties to even (the exact
 * quotient), in [-7, 7]; the value held is scale * code.  A group of zeros has
 * scale 0 and codes 0.  A group that holds an infinity or a NaN has scale NaN
 * and codes 0, so that what is computed from it is NaN.
 *   Eight codes k .. k + 7 (k a multiple of 8) share a 32-bit word (4 bytes,
 * the low byte first): code k + i, plus 8, lies in its bits 4 (i / 2 + 4 (i % 2))
 * to 3 above, so that a pair of neighbours lies 16 bits apart.  The products
 * below read any nibble, 0 (code -8) to 15 (code 7).
 *   w [rows][cols] (MOE_BF16 or MOE_F32 as `dtype`), rows ldw >= cols elements
 *   apart; q [rows][cols/2] bytes, rows ldq >= cols/2 bytes apart, ldq a
 *   multiple of 4 (the bytes past cols/2 of a row are left alone); scale
 *   [rows][ceil(cols/group)] float32, rows lds >= ceil(cols/group) elements
 *   apart, 4-byte aligned.  cols a multiple of 8; rows may be 0.  Errors:
 *   MOE_ERR_INVALID_ARG for a NULL or misaligned pointer or sizes outside
 *   these rules; MOE_ERR_UNSUPPORTED for another dtype or group, or more than
 *   2^28 cols. */
int moe_i4_quantize(const void* w, int dtype, int64_t rows, int64_t cols, int64_t ldw, int group, uint8_t* q,
                    int64_t ldq, float* scale, int64_t lds, void* stream);

/* The inverse: w [rows][cols] = scale * code (MOE_F32: the float32 product;
 * MOE_BF16: that rounded once more, to nearest even), e.g. to run a long
 * prompt on the bf16 products.  Layouts and errors as moe_i4_quantize. */
int moe_i4_dequantize(const uint8_t* q, int64_t ldq, const float* scale, int64_t lds, int64_t rows, int64_t cols,
                      int group, void* w, int dtype, int64_t ldw, void* stream);

/* A linear layer on 4-bit weights (e.g. a dense projection beside the
 * experts), for few rows: y[m][n] = sum over groups of scale[n][g] (sum over k
 * of group g of x[m][k] code[n][k]) + bias[n], float32 sums, one rounding to
 * y's type.
 *   x [M][K] bf16, rows ldx >= K elements apart, ldx a multiple of 8; wq
 *   [N][K/2] and ws as moe_i4_quantize writes them, rows ldw bytes (a multiple
 *   of 16) and lds elements apart; bias [N] float32 or NULL; y [M][N] MOE_BF16
 *   or MOE_F32 as `dtype`, rows ldy >= N elements apart.  K a multiple of 8;
 *   any M >= 0 (each 16 rows read the weights anew: for hundreds of rows
 *   dequantise them and use a bf16 product).  The matrix cores get the codes
 *   plus 24, and 24 times the sum of x is taken off again: the rounding error of
 *   a group's sum is relative to up to (24 + 31) sum |x|.  No sum on the way is
 *   above 31 sum |x|; a row of x for which that leaves float32 may give NaN, and
 *   one that holds an infinity or NaN does.  The nibbles and scales of a row's
 *   last 16 bytes past K are never used.
 *   Errors: MOE_ERR_INVALID_ARG for a NULL or misaligned pointer (ws 4-byte,
 *   the others 16-byte aligned) or sizes outside these rules;
 *   MOE_ERR_UNSUPPORTED for another dtype or group, K above 2^20, ldx, ldw or
 *   lds above 2^21, or M or N of 2^31 - 256 or more. */
int moe_i4_linear(int64_t M, int64_t N, int64_t K, int group, const void* x, int64_t ldx, const uint8_t* wq,
                  int64_t ldw, const float* ws, int64_t lds, const float* bias, void* y, int64_t ldy, int dtype,
                  void* stream);

/* The most tokens of the calls below. */
#define MOE_DECODE_MAX_T 64

/* Bytes of device workspace that moe_decode and moe_decode_i4 need for desc.
 * MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED as those calls. */
int moe_decode_workspace_size(const moe_desc* desc, size_t* bytes);

/* A1 to A7 for a decode step of T <= MOE_DECODE_MAX_T tokens: router logits,
 * selection (as moe_route, or moe_route_grouped with n_groups > 1), the local
 * experts' gate/up, SwiGLU and down, and the weighted sum, in two kernels.
 * An expert's weights are read once for up to 4 to 16 of its tokens (by type and
 * T; both tokens of two).
 *   x [T][d] bf16, Wr [E][d] bf16, bias [E] float32 or NULL; W1, W3 [NL][f][d]
 *   and W2 [NL][d][f] bf16; topk_idx [T][k] int32 and topk_w [T][k] float32,
 *   written (slots in falling order of the logits, ties to the lower expert);
 *   y [T][d] bf16, 0 for a token without a local slot.
 *   Wr NULL (then bias must be NULL and n_groups 1): topk_idx and topk_w are
 *   read instead, any routing: an expert outside the local ones counts for
 *   nothing, and an expert that a token names twice has the sum of the two
 *   weights.
 *   Sums are float32; h is rounded to bf16 between the products as in
 *   moe_grouped_ffn, y once at the end.  A token whose logits are not finite
 *   may get any selection; what does not depend on it is right.
 *   ws: moe_decode_workspace_size() bytes; calls that share one must not
 *   overlap (same stream, or ordered by events; where they do, y is undefined, and
 *   NaN if a call gives up, after seconds, on flags that the other has cleared).
 *   It needs no preparation and holds nothing from call to call.  tile_schedule
 *   and wgrad_dtype are of no consequence.
 *   Errors: MOE_ERR_INVALID_ARG for a NULL or misaligned pointer or a bad
 *   descriptor or n_groups (as moe_route_grouped); MOE_ERR_WORKSPACE for too
 *   small or a misaligned workspace; MOE_ERR_UNSUPPORTED for more tokens,
 *   another dtype than MOE_BF16, d or f above 2^20, or T k f of 2^30 or more. */
int moe_decode(const moe_desc* desc, int n_groups, const void* x, const void* Wr, const float* bias, const void* W1,
               const void* W3, const void* W2, int32_t* topk_idx, float* topk_w, void* y, void* ws, size_t ws_bytes,
               void* stream);

/* moe_decode with the experts' weights in 4 bits: W1q, W3q [NL][f][d/2], W2q
 * [NL][d][f/2] bytes with scales W1s, W3s [NL][f][ceil(d/group)], W2s
 * [NL][d][ceil(f/group)], as moe_i4_quantize writes them (rows without gaps).
 * The products are of bf16 activations with whole-number codes, summed in
 * float32 per group and scaled, as in moe_i4_linear.  MOE_ERR_UNSUPPORTED also for a group other
 * than 32, 64 or 128. */
int moe_decode_i4(const moe_desc* desc, int group, int n_groups, const void* x, const void* Wr, const float* bias,
                  const uint8_t* W1q, const float* W1s, const uint8_t* W3q, const float* W3s, const uint8_t* W2q,
                  const float* W2s, int32_t* topk_idx, float* topk_w, void* y, void* ws, size_t ws_bytes,
                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DECODE_H */
