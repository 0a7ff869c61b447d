/*
 * pwq_serve.h -- C ABI of libpwq, second part: running a quantized layer.
 *
 * pwq.h turns a linear layer W into integer codes, steps and zero points.
 * The functions here pack those codes into 4 bits and multiply by them, and
 * normalise the hidden state that such a layer reads:
 *
 *   pwq_pack_codes, pwq_pack_overflow   codes -> packed layer
 *   pwq_rms_norm                        hidden state (+ residual) -> layer input
 *   pwq_packed_linear                   layer input -> layer output
 *
 * The conventions of pwq.h hold (row-major; caller-owned DEVICE pointers; no
 * allocation; work enqueued on `stream` without synchronising; argument
 * errors before anything is enqueued; bitwise-identical results for the same
 * arguments).  Hidden states are token-major: ntok x n, one row per token.
 *
 * The packed layer.  The weight of row r and column k is
 *     W^[r, k] = s[r, k / G] * (c[r, k] - z[r, k / G]),
 * c the stored code of a SYM (z = 0) or ASYM grid of at most 4 bits.  The
 * sweep does not clip [GEOM 2.3], so c may be any integer; it is held as
 *   qweight  : m x ldq bytes, ldq = pwq_packed_row_bytes(n) (a multiple of
 *              16).  Byte j of a row holds columns 2j (low half) and 2j + 1
 *              (high half) of clip(c): SYM -8 .. 7 as two's complement, ASYM
 *              0 .. 15.  Halves of columns >= n are ignored.
 *   scales   : m x (n / G) float32, as written by pwq_quant_layer.
 *   zeros    : m x (n / G) uint8 (0 .. 127), NULL for SYM.
 *   overflow : the codes outside the half's range, as a list sorted by tile
 *              of 16 rows x 128 columns (tiles row-major, pwq_pack_tiles(m, n)
 *              of them), then row, then column.  Entry = (c - clip(c)) * 65536
 *              + (row % 16) * 128 + column % 128 (with steps as below, c -
 *              clip(c) lies in -127 .. 239).  outlier_off[t] is the first
 *              entry of tile t, outlier_off[tiles] their number.  The SSQR
 *              outliers of pwq_overflow_entries [GEOM 3] are such codes; here
 *              they stay integers, so the product of the packed layer is that
 *              of the layer that was quantized.
 * Every lattice step c - z must lie in -127 .. 127.
 */
#ifndef PWQ_SERVE_H
#define PWQ_SERVE_H

#include "pwq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of 8-bit integers (beside pwq_dtype). */
enum { PWQ_I8 = 3 };

/* Bytes of one packed row of n columns; tiles of the overflow list. */
int64_t pwq_packed_row_bytes(int64_t n);
int64_t pwq_pack_tiles(int64_t m, int64_t n);

/* ---------------------------------------------------------------------- *
 * Packs codes (as written by pwq_quant_layer or pwq_babai_sweep).
 *   codes   : m x n int32, row stride ldc >= n.
 *   grid    : SYM or ASYM with bits in [2, 4] (else PWQ_ERR_UNSUPPORTED).
 *   zeros   : ASYM: m x (n / G) int32; ignored for SYM.
 *   qweight : out, m x pwq_packed_row_bytes(n), 16-byte aligned; padding is
 *             written 0.
 *   zeros8  : ASYM: out, m x (n / G) uint8.
 *   outlier_off : out, pwq_pack_tiles(m, n) + 1 int32.
 *   info    : out, 2 int32: the codes whose lattice step lies outside
 *             -127 .. 127, and the zero points outside 0 .. 127.  Where either
 *             is not 0 the packed layer does not stand for the codes.
 * pwq_pack_overflow then writes the outlier_off[tiles] entries (the caller
 * reads their number to allocate them; max_out bounds what is written).
 * ---------------------------------------------------------------------- */
pwq_status pwq_pack_codes(const int32_t* codes, int64_t m, int64_t n, int64_t ldc,
                          const pwq_grid* grid, const int32_t* zeros, uint8_t* qweight,
                          uint8_t* zeros8, int32_t* outlier_off, int32_t* info, void* stream);
pwq_status pwq_pack_overflow(const int32_t* codes, int64_t m, int64_t n, int64_t ldc,
                             const pwq_grid* grid, const int32_t* outlier_off,
                             int32_t* outliers, int64_t max_out, void* stream);

/* ---------------------------------------------------------------------- *
 * Root-mean-square norm with the residual's addition:
 *     h = x + residual,  y = h / sqrt(mean(h^2) + eps) * weight  per token,
 * all in float32; y and the sum h are rounded once, when they are written.
 *   x        : ntok x n, xdtype PWQ_F32 or PWQ_BF16, row stride ldx >= n.
 *   residual : NULL, or ntok x n of the same type, row stride ldr >= n.
 *   weight   : n values, wdtype PWQ_F32 or PWQ_BF16.
 *   eps      : 0 <= eps < 1e30, rounded to float32.
 *   sum      : NULL, or out: h in x's type, row stride lds >= n; may be the
 *              memory of x or of residual with the same stride, and else
 *              overlaps neither.
 *   y        : out, row stride ldy >= n, ydtype PWQ_F32, PWQ_BF16 or PWQ_I8;
 *              overlaps no other argument.
 *   scales   : PWQ_I8: out, ntok float32: the step max|y| / 127 of each token
 *              (1 where that is 0); y = rint(value / step), within -127 ..
 *              127.  A token whose y holds a NaN or an infinity gets that as
 *              its step, and the codes 0.  Unused otherwise.
 * Squares and their sum are float32: beyond its range (|h| above 1e19) they give
 * 0, and below it (|h| under 1e-22 with eps = 0) an infinity.
 * ---------------------------------------------------------------------- */
pwq_status pwq_rms_norm(const void* x, int32_t xdtype, int64_t ntok, int64_t n, int64_t ldx,
                        const void* residual, int64_t ldr, const void* weight, int32_t wdtype,
                        double eps, void* sum, int64_t lds, void* y, int32_t ydtype,
                        int64_t ldy, float* scales, void* stream);

/* ---------------------------------------------------------------------- *
 * y = x W^^T of a packed layer:
 *     y[t, r] = x_scale[t] * sum_k x[t, k] * s[r, k / G] * (c - z)[r, k].
 *   x         : ntok x n, row stride ldx >= n, xdtype PWQ_F32, PWQ_BF16 or
 *               PWQ_I8 (signed).  ntok may be 0.
 *   x_scales  : ntok float32 for PWQ_I8 (required), NULL otherwise.
 *   qweight, scales, zeros, outlier_off, outliers : the packed layer; zeros
 *               NULL for SYM; outlier_off and outliers NULL (n_out 0) when no
 *               code overflows.  n_out = outlier_off[tiles].
 *   group     : G, 0 for one step per row; divides n.
 *   y         : out, ntok x m, row stride ldy >= m, ydtype PWQ_F32 or PWQ_BF16;
 *               must not overlap x (rows of the two may lie side by side in a
 *               wider matrix).
 *   ws        : pwq_packed_linear_workspace_size bytes, for this x, sizes,
 *               group and n_out (0 for few tokens whose rows of x are 16-byte aligned).
 * Steps c - z multiply x as integers.  With groups of a multiple of 32 columns,
 * or one per row, the sum of a group, or of 32 or more of its columns, is
 * multiplied by the group's step; that sum is float32, and exact for PWQ_I8
 * (int32, or float32 below 2^24) but in rows of one group of more than 2^17
 * columns.  Groups of other sizes multiply each product.  Sums beyond that are
 * float32, and all of them in a fixed order; which kernel serves a token, and
 * so the last bits of its result, depends on ntok.  A token with an infinity or
 * NaN, or sums beyond float32's range, gives values that are not finite; other
 * tokens are unaffected.
 * ---------------------------------------------------------------------- */
size_t pwq_packed_linear_workspace_size(const void* x, int32_t xdtype, int64_t ntok, int64_t ldx,
                                        int64_t m, int64_t n, int32_t group, int64_t n_out);
pwq_status pwq_packed_linear(const void* x, int32_t xdtype, int64_t ntok, int64_t ldx,
                             const float* x_scales, const uint8_t* qweight, int64_t m, int64_t n,
                             const float* scales, const uint8_t* zeros, int32_t group,
                             const int32_t* outlier_off, const int32_t* outliers, int64_t n_out,
                             void* y, int32_t ydtype, int64_t ldy, void* ws, size_t ws_bytes,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PWQ_SERVE_H */
