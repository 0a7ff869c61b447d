/*
 * pwq_cache.h -- C ABI of libpwq, third part: the key-value cache between
 * quantized layers.
 *
 * The k, v and q projections of pwq_packed_linear give keys, values and
 * queries; the functions here keep keys and values in 8 or 4 bits and attend
 * to them:
 *
 *   pwq_cache_write         keys, values of new tokens -> cache
 *   pwq_cache_read          cache -> keys, values
 *   pwq_cached_attention    queries -> attention's output, over the cache, with
 *                           a prefix that all sequences share, or without
 *
 * The conventions of pwq.h hold (caller-owned DEVICE pointers; no allocation;
 * work enqueued on `stream` without synchronising; argument errors before
 * anything is enqueued; bitwise-identical results for the same arguments).
 *
 * What is stored.  A token's head of keys, or of values, x[0 .. D-1], becomes
 * codes c of b bits with a step s and a zero point z:
 *     lo = min(0, min x),  hi = max(0, max x),
 *     s = (hi - lo) / (2^b - 1), in float32, then rounded to 16 significant bits
 *         (halves upwards; to a multiple of 2^-141 where that is coarser),
 *     z = min(rint(-lo / s), 2^b - 1),  c = min(max(rint(x / s) + z, 0), 2^b - 1),
 * both quotients of the exact numbers, ties to even; z = c = 0 where s = 0.
 * It stands for s * (c - z), which is exact in float32.  Where x holds a NaN or
 * an infinity, or hi - lo is beyond float32, s is a NaN and c = z = 0: all of
 * that head reads as NaN.  The word of the head is s with z in its lowest 8
 * bits (the float32's lowest 8, which rounding has cleared).
 *
 * Records.  records : pages x kv_heads x (page / 32) records of
 * pwq_cache_record_bytes(head_dim, bits) bytes, 16-byte aligned.  A record holds
 * 32 consecutive tokens of one head: key codes, value codes (4 D b bytes each),
 * 32 key words, 32 value words (uint32).  Codes lie as the matrix cores take
 * them.  64 lanes share the keys' or values' codes; lane L's bytes go in pieces
 * of 16, piece P at 1024 P + 16 L:
 *   key codes   : token 16 t + a, channel 32 j + 8 g + e is of lane 16 g + a, in
 *                 the order (t, j, e); 4 bits: e at bit 4 (e / 2) + 16 (e % 2) of
 *                 the four bytes of a (t, j).
 *   value codes : token 16 t + 4 g + i, channel 16 n + a is of lane 16 g + a, in
 *                 the order (n, t, i); 4 bits: an even n is the low half and
 *                 n + 1 the high half of a byte, in the order (n / 2, t, i).
 *
 * Batches.  nseq sequences, of which sequence i has rows starts[i] ..
 * starts[i + 1] - 1 of the call's tensors (starts: nseq + 1 int32, ascending).
 * Those are its last tokens: lengths[i] (int32) counts all of its tokens, these
 * rows included.  Token p is in page table[i * ldt + p / page], at p % page.
 * Rows before starts[0] and from starts[nseq] on belong to no sequence: nothing
 * is read from them, and outputs keep what was there.  All of these are read on
 * the device, so that a captured call can be replayed with other batches.
 *   A table entry outside 0 .. pages - 1, and a token at or past width * page,
 * is a hole: writes there are dropped, reads give 0, and attention leaves its
 * keys out.  Values of starts outside 0 .. ntok are taken as 0 or ntok, and
 * lengths below 0 as 0; with starts that descend the outputs are unspecified.
 * Pages that a call writes may be shared by sequences only where they write
 * different tokens of the page (else either's bytes may stay).
 */
#ifndef PWQ_CACHE_H
#define PWQ_CACHE_H

#include "pwq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pwq_cache {
  void* records;
  int64_t pages;      /* >= 0; pages * kv_heads * (page / 32) <= 2^40 */
  int32_t kv_heads;   /* >= 1 */
  int32_t head_dim;   /* D: 64, 128 or 256 */
  int32_t bits;       /* b: 8 or 4 */
  int32_t page;       /* tokens of a page: a power of two, 32 .. 4096 */
} pwq_cache;

typedef struct pwq_batch {
  const int32_t* starts;
  const int32_t* lengths;
  const int32_t* table;
  int64_t ldt;        /* >= width */
  int32_t nseq;       /* >= 0 */
  int32_t width;      /* >= 0 */
} pwq_batch;

/* Bytes of a record; 0 for another head_dim or bits than above. */
int64_t pwq_cache_record_bytes(int32_t head_dim, int32_t bits);

/* ---------------------------------------------------------------------- *
 * Quantizes the rows of a batch into the cache.
 *   k, v : ntok x kv_heads x D, dtype PWQ_F32 or PWQ_BF16; element (t, h, d) at
 *          t * tstride + h * hstride + d (strides >= 0, in elements; those of
 *          several tokens or heads times their number at most 2^56).
 *          ntok * kv_heads < 2^30 (and ntok * heads below).
 * ---------------------------------------------------------------------- */
pwq_status pwq_cache_write(const pwq_cache* cache, const pwq_batch* batch, const void* k,
                           int64_t k_tstride, int64_t k_hstride, const void* v, int64_t v_tstride,
                           int64_t v_hstride, int32_t dtype, int64_t ntok, void* stream);

/* ---------------------------------------------------------------------- *
 * The values that the cache holds for the rows of a batch (for all tokens of a
 * sequence: as many rows as its length).
 *   k, v : out, as for pwq_cache_write, dtype PWQ_F32 (exact) or PWQ_BF16
 *          (rounded once); no two elements in one place; overlap nothing.
 * ---------------------------------------------------------------------- */
pwq_status pwq_cache_read(const pwq_cache* cache, const pwq_batch* batch, void* k,
                          int64_t k_tstride, int64_t k_hstride, void* v, int64_t v_tstride,
                          int64_t v_hstride, int32_t dtype, int64_t ntok, void* stream);

/* ---------------------------------------------------------------------- *
 * Attention of a batch's rows to what is cached, the rows' own tokens included
 * (written before, on the same stream):
 *     out[t, h] = sum_p w_p V[p, h'],  w = softmax_p(scale * q[t, h] . K[p, h']),
 * h' = h / (heads / kv_heads), over tokens p of t's sequence: all of them, or
 * (causal) those up to t's own.  A row without any token gives 0.
 *   prefix : NULL, or a batch of one sequence, nseq 1, whose starts are not
 *            read (may be NULL): lengths[0] tokens in pages table[0 .. width - 1]
 *            that come before every sequence of the batch.  Their keys and values
 *            are read once for all rows, not once for every sequence.
 *   q, out : ntok x heads x D, both PWQ_F32 or both PWQ_BF16, strides as above;
 *            heads is a multiple of kv_heads.  out overlaps neither q nor the
 *            cache and has no two elements in one place.
 *   scale  : 1e-30 .. 1e30.
 *   ws     : pwq_cached_attention_workspace_size bytes, 256-byte aligned.
 * Keys multiply as their codes, exactly, and values too but where said.  Rows of a
 * sequence are taken 16 together, or 128 or 256 where there are many.  A power of two
 * scales a row's queries so that the largest element fits float16 (128 or 256 together:
 * all of them alike, where no row's largest, but of rows of zeros, is more than 2^8
 * below another's):
 *   PWQ_BF16 : an element is exact where it is above 2^-22 of the row's largest, else
 *              off by 2^-30 of it.  A token's weight times its step is rounded to
 *              float16 once (2^-11).  Where rows are taken 128 or 256 together weight,
 *              step and step times code are each rounded (3 times 2^-11).
 *   PWQ_F32  : two float16 parts, for elements as for weights: within 2^-22, or 2^-30
 *              of the row's largest element.
 * A weight is off by 2^-33 of the largest so far at least (2^-25 where scores pass
 * 2^25), and a step (128 or 256 together, PWQ_BF16) by 2^-30 of the largest of the steps
 * that the row sees, or 2^-22 of itself.  Neither other rows nor tokens that a row does
 * not see make it less exact.  Sums, maxima and totals are float32, in a fixed order; how
 * a sequence is split, and so the last bits of its rows, depends on the sizes and starts
 * and lengths of the whole batch.  A row of q with an infinity or NaN, or with a token
 * it sees that reads as NaN, gives NaN; other rows are unaffected.  Scores, scale times
 * an element of q, and steps times 2^44 have to stay within float32.
 * ---------------------------------------------------------------------- */
size_t pwq_cached_attention_workspace_size(const pwq_cache* cache, const pwq_batch* batch,
                                           const pwq_batch* prefix, int32_t heads, int32_t dtype,
                                           int64_t ntok);
pwq_status pwq_cached_attention(const pwq_cache* cache, const pwq_batch* batch,
                                const pwq_batch* prefix, const void* q, int64_t q_tstride,
                                int64_t q_hstride, void* out, int64_t out_tstride,
                                int64_t out_hstride, int32_t heads, int32_t dtype, int64_t ntok,
                                double scale, int32_t causal, void* ws, size_t ws_bytes,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PWQ_CACHE_H */
