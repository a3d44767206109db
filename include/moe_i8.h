/*
 * moe_i8.h -- the INT8 entry points of libmoe.so: the row quantiser, the
 * expert products A5 and A6 of moe.h on INT8 codes, and a plain linear layer
 * on INT8 codes.  The conventions of moe.h hold: device pointers owned by the
 * caller and 16-byte aligned unless said otherwise, no allocation, no
 * synchronisation, asynchronous on `stream`, arguments checked on the host.
 * Every result is the same on every call (32-bit integer sums, then a fixed
 * order of float32 operations), and no call needs a workspace.
 */
#ifndef MOE_I8_H
#define MOE_I8_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* INT8 with one scale per row (per token for activations, per output channel
 * for the weights of a linear layer): the codes and scales that the INT8
 * products below read.  Per row: m = max |w|, scale = m / 127 in float32,
 * code = 127 w / m rounded to the nearest integer, ties to even (the exact
 * quotient, not one in float32).  A row of zeros has scale 0 and codes 0.  A
 * row that holds an infinity or a NaN has scale NaN and codes 0, so that what
 * is computed from it is NaN.
 *   w [rows][cols] (MOE_BF16 or MOE_F32 as `dtype`), rows ldw >= cols elements
 *   apart; q [rows][cols] int8, rows ldq bytes apart, ldq >= cols and a
 *   multiple of 16 (the bytes past cols of a row are left alone); scale [rows]
 *   float32.  nrows (device int32, or NULL): rows at or past *nrows are left
 *   alone (e.g. offsets + NL: the routed rows of a [R_cap] buffer).  rows may
 *   be 0.  Errors: MOE_ERR_INVALID_ARG for a NULL pointer, w or q not 16-byte
 *   aligned, scale or nrows not 4-byte aligned, or sizes outside these rules;
 *   MOE_ERR_UNSUPPORTED for another dtype or more than 2^28 cols. */
int moe_i8_quantize_rows(const void* w, int dtype, int64_t rows, int64_t cols, int64_t ldw,
                         const int32_t* nrows, int8_t* q, int64_t ldq, float* scale, void* stream);

/* A linear layer on INT8 codes (e.g. a dense projection beside the experts):
 *   y[m][n] = xs[m] ws[n] (sum over k of xq[m][k] wq[n][k]) + bias[n]
 *   with the sum in 32-bit integers (exact), then, in float32 and in this order,
 *   times xs, times ws, plus the bias, each rounded (no fused operation), and one
 *   rounding to y's type: a row's values do not depend on the rows beside it.
 *   xq [M][K] codes, rows ldx bytes apart, xs [M]; wq [N][K] codes, rows ldw
 *   bytes apart, ws [N]; bias [N] float32 or NULL; y [M][N] MOE_BF16 or
 *   MOE_F32 as `dtype`, rows ldy >= N elements apart.  Any M >= 0, N >= 1 and
 *   1 <= K <= 131072; ldx, ldw >= K and multiples of 16 (of a row's last 16
 *   bytes, those past K may hold anything).  Codes lie in [-127, 127].
 *   Errors: MOE_ERR_INVALID_ARG for a NULL or misaligned pointer or sizes
 *   outside these rules; MOE_ERR_UNSUPPORTED for another dtype, a larger K,
 *   ldx or ldw above 4194304, or M or N of 2^31 - 256 or more. */
int moe_i8_linear(int64_t M, int64_t N, int64_t K, const int8_t* xq, int64_t ldx, const float* xs,
                  const int8_t* wq, int64_t ldw, const float* ws, const float* bias, void* y, int64_t ldy,
                  int dtype, void* stream);

/* A5 in INT8: gate/up with the SwiGLU epilogue, x read through row_token (as
 * moe_expert_gate_up_gather) as codes with one scale per token, W1 and W3 as
 * codes with one scale per channel:
 *   G[r][n] = xs[t] W1s[g][n] (sum over k of xq[t][k] W1q[g][n][k]),
 *   t = row_token[r], U likewise with W3, h = silu(G) * U; the sums in 32-bit
 *   integers, the rest in float32, each output rounded once to bf16.
 *   xq [T][d], xs [T] (moe_i8_quantize_rows of x); W1q, W3q [NL][f][d], W1s,
 *   W3s [NL][f] (of W1 and W3 as NL f rows); gu [R_cap][2f] (or NULL) and h
 *   [R_cap][f] bf16.  MOE_ERR_UNSUPPORTED unless dtype is MOE_BF16,
 *   d <= 131072 and T * d < 2^31. */
int moe_expert_gate_up_i8(const moe_desc* desc, const int32_t* offsets, const int32_t* row_token,
                          const int8_t* xq, const float* xs, const int8_t* W1q, const float* W1s,
                          const int8_t* W3q, const float* W3s, void* gu, void* h, void* stream);

/* A6 in INT8: y_perm[r][n] = hs[r] W2s[g][n] (sum over k of hq[r][k]
 * W2q[g][n][k]) for row r of expert g's segment.
 *   hq [R_cap][f], hs [R_cap] (moe_i8_quantize_rows of h with nrows =
 *   offsets + NL); W2q [NL][d][f], W2s [NL][d]; y_perm [R_cap][d] bf16.
 *   MOE_ERR_UNSUPPORTED unless dtype is MOE_BF16 and f <= 131072. */
int moe_expert_down_i8(const moe_desc* desc, const int32_t* offsets, const int8_t* hq, const float* hs,
                       const int8_t* W2q, const float* W2s, void* y_perm, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_I8_H */
