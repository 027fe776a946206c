/*
 * sgdn_serve.h - C ABI of libsgdn.so, third part: what stands around the paged
 * cache of sgdn_attn.h in a served softmax attention layer, on AMD Instinct
 * MI355X.
 *
 * One serving step of such a layer is
 *   sgdn_rope or sgdn_norm_rope   rotary positions of queries and keys, with a
 *                                 norm of every head in the same pass or without
 *   sgdn_paged_write              the keys and values into the cache
 *   sgdn_paged_attend_chunk       attention of the step's tokens, any number of
 *                                 each request, over its whole cached sequence
 * with sgdn_paged_plan once ahead of all layers.  sgdn_norm_rope without a
 * rotation also makes the L2-normalised queries and keys that sgdn.h expects.
 * Inference only: no entry point has a gradient.
 *
 * Conventions on ownership, streams, status codes and reentrancy are those of
 * sgdn.h: arrays are DEVICE memory of the caller's, nothing is allocated, kept
 * or synchronised, invalid arguments are refused before anything is enqueued,
 * and every call can be captured in a HIP graph.
 */
#ifndef SGDN_SERVE_H
#define SGDN_SERVE_H

#include "sgdn_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Rotary positions ------------------------------------------------ */

/* How frequencies are scaled for contexts longer than those of training.
 * With f_i = base^(-2 i / rot), i = 0 .. rot/2 - 1, radians per token:
 *   SGDN_ROPE_PLAIN       f_i
 *   SGDN_ROPE_LINEAR      f_i / factor (positions are divided by it)
 *   SGDN_ROPE_BASE        f_i of the base  base factor^(rot / (rot - 2)), so that
 *                         the slowest pair is slowed by the factor and the
 *                         fastest is not (rot >= 4)
 *   SGDN_ROPE_BY_PAIR     with p(n) = rot ln(original / (2 pi n)) / (2 ln base),
 *                         the pair that turns n times in `original` tokens,
 *                         a = max(floor(p(high)), 0), b = min(ceil(p(low)), rot - 1)
 *                         (b = a + 0.001 where they are equal) and
 *                         s = clamp((i - a) / (b - a), 0, 1):
 *                         f_i (1 - s) + f_i s / factor;
 *                         the magnitude is 1 + 0.1 ln(factor) for factor > 1
 *   SGDN_ROPE_BY_TURNS    with n_i = f_i original / (2 pi) turns in `original`
 *                         tokens and s = clamp((n_i - low) / (high - low), 0, 1):
 *                         f_i s + f_i (1 - s) / factor
 * The magnitude is 1 unless said otherwise. */
enum {
  SGDN_ROPE_PLAIN = 0, SGDN_ROPE_LINEAR = 1, SGDN_ROPE_BASE = 2, SGDN_ROPE_BY_PAIR = 3,
  SGDN_ROPE_BY_TURNS = 4
};

/* Frequencies for sgdn_rope, made on the host: freqs [rot / 2] and magnitude
 * [1] are HOST memory here (the caller copies the frequencies to the device,
 * once for a model).  rot >= 2 and even, at most 256; base > 1; factor >= 1
 * (read by all scalings but PLAIN); original > 0 and 0 < low < high (read by
 * BY_PAIR and BY_TURNS); SGDN_EINVAL otherwise. */
int sgdn_rope_freqs(int32_t rot, int32_t scaling, double base, double factor, double original,
                    double low, double high, double* freqs, double* magnitude);

/* Pairs of a rotation. */
enum {
  SGDN_ROPE_HALF = 0,         /* elements i and i + rot / 2                   */
  SGDN_ROPE_INTERLEAVED = 1   /* elements 2 i and 2 i + 1                     */
};

/* Strides in elements of [rows, heads, d]; the elements of a head follow each
 * other.  Heads may lie apart (views of a joint projection's output, or of one
 * that holds a gate beside each head), rows inside of heads; neither may
 * overlap.  At most 2^36; those of a single row or head are not looked at. */
typedef struct {
  int64_t row;       /* from one row to the next                              */
  int64_t head;      /* from one head to the next                             */
} sgdn_strides;

/* Shape of a call.  Supported: d <= 256 with rows of a multiple of 16 bytes
 * (d a multiple of 8, or of 4 in fp32), rot even and 0 <= rot <= d,
 * n_q + n_k < 2^16, rows < 2^26 - 3 (SGDN_EUNSUPPORTED otherwise; negative values
 * and d = 0 are SGDN_EINVAL; no rows, or no heads at all, do nothing). */
typedef struct {
  int32_t rows;
  int32_t n_q, n_k;  /* query and key heads; 0 for none                       */
  int32_t d;
  int32_t rot;       /* elements rotated: the first of each head; the rest passes */
  int32_t layout;    /* SGDN_ROPE_HALF or SGDN_ROPE_INTERLEAVED               */
  int32_t dtype;     /* sgdn_dtype of q, k and their outputs                  */
  int32_t w_dtype;   /* sgdn_dtype of the weights (sgdn_norm_rope)            */
  sgdn_strides q, k, q_out, k_out;
} sgdn_rope_shape;

/* Turns each pair (x, y) of every head of row r by the angle t = p freqs[i],
 * p = pos[r] + pos_offset:  magnitude (x cos t - y sin t, y cos t + x sin t).
 *   q, k         [rows, heads, d] inputs (NULL without heads); q_out, k_out
 *                outputs: either the inputs themselves (the same data and
 *                strides; SGDN_EINVAL for other strides) or without any overlap
 *   pos          [rows]; a row with p < 0 is left out: nothing of it is read or
 *                written.  (pos = row_len of sgdn_paged_plan, pos_offset = -1:
 *                each new token's place, and nothing for padding rows.)
 *   freqs        [rot / 2] fp64, radians per token (sgdn_rope_freqs, or any)
 *   magnitude    finite
 * Angles are formed and reduced in fp64, exact to 2^-53 of themselves: a
 * position of 10^6 errs by 10^-10.  (Beyond 2^52 nothing of an angle is known
 * modulo a turn: pairs are turned by some angle.)  Values are turned in fp32 and rounded
 * once.  Elements behind rot are copied.
 * Alignment: q, k and their outputs start at 16 bytes, strides are multiples of
 * 16 bytes, freqs starts at 8; SGDN_EINVAL otherwise. */
int sgdn_rope(const sgdn_rope_shape* p, const void* q, const void* k, const int32_t* pos,
              int32_t pos_offset, const double* freqs, double magnitude, void* q_out, void* k_out,
              void* stream);

/* The same of normed heads:  x / sqrt(mean of x^2 over the d elements + eps)
 * (w + w_offset), then the rotation.
 *   wq, wk       [d] w_dtype, 16-byte aligned, or NULL: zeros.  (w_offset = 1 for
 *                weights stored around 0; NULL weights, w_offset = 1/sqrt(d) and
 *                eps / d give the L2 norm.)
 *   eps          finite, >= 0.  (With 0, a head of zeros is 0/0.)
 * Sums of squares are held in fp64: heads of any magnitude that the type holds
 * are normed.  The rest is fp32, rounded once at the end. */
int sgdn_norm_rope(const sgdn_rope_shape* p, const void* q, const void* k, const void* wq,
                   const void* wk, float w_offset, float eps, const int32_t* pos,
                   int32_t pos_offset, const double* freqs, double magnitude, void* q_out,
                   void* k_out, void* stream);

/* ---- Attention of chunks over the paged cache ------------------------- */

/* Device workspace of sgdn_paged_attend_chunk; 0 for an invalid shape.  Up to
 * 68 MB for parts of work (34 MB for heads of 64) and 32 bytes for each request
 * and each tile of rows (128 (row, query head of one key head) pairs, 64 in
 * fp32).  What it holds does not matter. */
size_t sgdn_paged_chunk_workspace_bytes(const sgdn_paged* p);

/* sgdn_paged_attend for steps in which requests have many new tokens (prompts,
 * pieces of prompts, drafts), or some of them many and others one: a request's
 * context is read once for many rows, and the work is divided on the device by
 * the lengths it finds there.  (Steps of single rows alone are that call's: many
 * long ones take as long here, short ones up to twice as long, 2048 rows of 100
 * tokens 389 and 187 us, and a few wait for three launches, 17 us at least.)
 *   cu           [B + 1] rows of request b are cu[b] .. cu[b + 1] - 1 (cu of
 *                sgdn_paged_plan; must not fall)
 *   lens         [B] tokens of each request, its new ones included (lens_out of
 *                sgdn_paged_plan).  Row r of request b sees its first
 *                lens[b] - cu[b + 1] + r + 1 tokens (none where that is not
 *                positive, at most max_len).
 * All else as in sgdn_paged_attend: q, table, scale, o, lse, rows that see
 * nothing (rows of no request among them: o = 0, lse = -inf), pages that are
 * none, types, supported shapes.  Where cu falls, which request a row belongs
 * to is undefined, and rows may be left unwritten.
 * Precision: as sgdn_paged_attend, weights of 16-bit inputs in two parts
 * whatever o's type.  An element of v that is not finite makes the same element
 * of every row that sees it not finite; an infinity may come out as NaN.
 * A row's bits may depend on the other rows of its request and on the lengths of
 * the call's requests, by which the sums are divided; its error bound does not.
 * Equal calls give equal bits.
 * A row sees at most 2^31 - 128 tokens: SGDN_EUNSUPPORTED where max_len, or width
 * page without it, is larger. */
int sgdn_paged_attend_chunk(const sgdn_paged* p, const void* q, int64_t ldq, const void* k_cache,
                            const void* v_cache, const int32_t* table, const int32_t* cu,
                            const int32_t* lens, float scale, void* o, float* lse, void* ws,
                            size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SGDN_SERVE_H */
