/*
 * sgdn_attn.h - C ABI of libsgdn.so, second part: softmax attention of new
 * tokens over a paged key/value cache, for the attention layers that are
 * served beside the gated linear layers of sgdn.h, on AMD Instinct MI355X.
 *
 * One serving step of such a layer is
 *   sgdn_paged_release        (now and then) finished requests' pages go back
 *   sgdn_paged_plan           pages, slots and row descriptors of new tokens
 *   sgdn_paged_write          their keys and values into the cache
 *   sgdn_paged_attend         attention over the whole context, or
 *   sgdn_paged_select and     attention over the blocks that a cheap score
 *   sgdn_paged_attend_sparse  picks for each row
 * (plan and release once per step for all layers).  Inference only: no entry
 * point has a gradient.
 *
 * Conventions (beyond those of sgdn.h on ownership, streams, status codes
 * and reentrancy: all arrays are DEVICE memory of the caller's, dense and
 * row-major unless a stride is given, nothing is allocated, kept or
 * synchronised, and every call can be captured in a HIP graph)
 * ----------------------------------------------------------------------
 * - B requests, R rows (a row is one new token of one request), Hq query
 *   heads over Hkv key/value heads (head h reads key/value head
 *   h / (Hq / Hkv)), D elements per head, P tokens per page, W pages per
 *   block-table row.
 * - The cache holds n_pages pages: k_cache, v_cache [n_pages, Hkv, P, D].
 *   Token t of request b lives in page table[b, t / P] at place t % P; its
 *   slot is page * P + t % P.  "Block j" of a request is its tokens
 *   j P .. j P + P - 1, i.e. the page table[b, j].
 * - Row r belongs to request row_req[r] (NULL: request r) and sees the first
 *   row_len[r] tokens of it, itself included (the causal mask).  A row with
 *   row_len <= 0 or a row_req outside [0, B) sees nothing: its output is 0,
 *   its log-sum -inf, its block list all -1.  So the padding rows that
 *   sgdn_paged_plan writes behind the last token are harmless, and a step of
 *   fixed size can be captured once and replayed.  Lengths beyond max_len
 *   are cut to max_len.
 * - Device data is never trusted with an address: a page outside
 *   [0, n_pages), a block outside the row's context and a slot outside the
 *   cache take no part (nothing is read or written for them).
 * - Outputs overlap no inputs, except where said.
 * - Masked places are never read into a result: what unused slots and pages
 *   hold, NaN and infinities included, does not matter.
 * - Types: q, k, v and the caches share one of fp32, bf16, fp16; o is any of
 *   them.  Products run on the matrix cores with fp32 accumulation; the
 *   softmax maximum, sum and the output accumulate in fp32.  With 16-bit
 *   inputs the softmax weights enter their product as two numbers of that type
 *   (weight and remainder), whichever kernel takes a row: beside fp32's
 *   roundings and its own, o errs by at most 2^-17 (bf16) or 2^-23 (fp16, and
 *   2^-35 of the largest weight for each key) of the weighted mean of |v|.  So
 *   an fp32 o of bf16 inputs is good to 2^-17.  With fp32 inputs nothing is
 *   rounded below fp32.  A row's bits may depend on its neighbours' lists and
 *   on values in them that are not finite (sgdn_paged_attend_sparse of many
 *   rows: rows that share their lists are taken together, and sum in another
 *   order), its error bound not.
 * - A call's work is laid out from its shape, before the device knows any
 *   length.  max_len as the step needs it, tables without empty rows and lists
 *   no longer than the rows fill are therefore faster; so are a call of its
 *   own for a row that sees far more than the others, and for the prompts of a
 *   step that has single rows too.  Rows of one request read its context once
 *   each in sgdn_paged_attend.
 * - Alignment: q, k, v, the caches, codes and o start at 16 bytes; row
 *   strides are multiples of 16 bytes.  Otherwise SGDN_EINVAL.
 */
#ifndef SGDN_ATTN_H
#define SGDN_ATTN_H

#include "sgdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of a call.  Supported: D in {64, 128, 256}, P in {16, 32, 64, 128},
 * Hq a multiple of Hkv, W P < 2^31, n_pages P < 2^31, R Hq < 2^28, and
 * R < 2^28 - 15 for the write, R Hkv ceil(Hq / (16 Hkv)) < 2^24 - 8 for the
 * attention, R Hkv < 2^22 - 8 for the choice of blocks (SGDN_EUNSUPPORTED
 * otherwise; non-positive values are SGDN_EINVAL, rows = 0 does nothing). */
typedef struct {
  int32_t rows;      /* R: rows of q (or k, v)                               */
  int32_t batch;     /* B: rows of the block table                           */
  int32_t n_q, n_kv; /* Hq, Hkv                                              */
  int32_t d;         /* D                                                    */
  int32_t page;      /* P                                                    */
  int32_t n_pages;   /* pages of the cache                                   */
  int32_t width;     /* W: pages per block-table row                         */
  int32_t max_len;   /* upper bound of row_len, at most W P; 0 means W P     */
  int32_t dtype;     /* sgdn_dtype of q, k, v and the caches                 */
  int32_t o_dtype;   /* sgdn_dtype of o                                      */
} sgdn_paged;

/* Gives the pages of finished requests back to the ring of free pages.
 * The ring is free_list [n_free] with two running counters free_pos [2] =
 * {taken, returned}: entries taken .. returned - 1, each modulo n_free, are
 * the free pages (0 <= returned - taken <= n_free; n_free at least the number
 * of pages ever in the ring).
 *   lens         [B]     cached tokens of each request
 *   done         [B]     uint8, non-zero: the request has ended
 *   table        [B, W]  block table (read only)
 *   free_list    [n_free] in/out: the ended requests' pages are appended in
 *                request order
 *   free_pos     [2] int64 in; free_pos_out [2] out, may be free_pos
 *   lens_out     [B] out, 0 for an ended request, lens otherwise; may be lens
 * A negative length gives nothing back; one beyond W P gives W pages.
 * batch < 2^31 - 1024 (SGDN_EUNSUPPORTED otherwise). */
int sgdn_paged_release(int32_t batch, int32_t page, int32_t width, int32_t n_free,
                       const int32_t* lens, const uint8_t* done, const int32_t* table,
                       int32_t* free_list, const int64_t* free_pos, int32_t* lens_out,
                       int64_t* free_pos_out, void* stream);

/* Room and places for the new tokens of a step: takes the pages they need
 * from the ring (above), in request order, enters them in the block table
 * and describes the rows.
 *   lens, add    [B]     cached and new tokens of each request
 *   table        [B, W]  in/out: entries ceil(lens / P) .. of an admitted
 *                request are set, all others stay
 *   free_list    [n_free] read only
 *   free_pos     [2] int64 in; free_pos_out [2] out, may be free_pos
 *   lens_out     [B] out: lens + add where admitted, else lens; may be lens
 *   cu           [B + 1] out: rows of request b are cu[b] .. cu[b + 1] - 1
 *   page_cu      [B + 1] out: the same for the pages taken
 *   slot         [rows] out: slot of each row's token; -1 behind cu[B]
 *   row_req      [rows] out: its request; -1 behind cu[B]
 *   row_len      [rows] out: what it sees (its position + 1); 0 behind cu[B]
 *   status       [B] out: 0 admitted; otherwise the request gets no rows and
 *                keeps its length: 1 the ring has too few pages, 2 more than
 *                W pages, 4 more than `rows` rows, 8 a negative number
 * Requests are admitted by sums over the requests before them, the one in
 * question included, of those that are not refused for 2 or 8: a request
 * that needs pages is refused (1) if the sum of needed pages exceeds the
 * ring's, one that has rows is refused (4) if the sum of rows exceeds
 * `rows`.  The page numbers that the ring holds are taken as they are.
 * batch and rows < 2^31 - 1024 (SGDN_EUNSUPPORTED otherwise). */
int sgdn_paged_plan(int32_t batch, int32_t page, int32_t width, int32_t rows, int32_t n_free,
                    const int32_t* lens, const int32_t* add, int32_t* table,
                    const int32_t* free_list, const int64_t* free_pos, int32_t* lens_out,
                    int64_t* free_pos_out, int32_t* cu, int32_t* page_cu, int32_t* slot,
                    int32_t* row_req, int32_t* row_len, int32_t* status, void* stream);

/* Writes the new tokens' keys and values to their slots and summarises the
 * pages that they complete.
 *   k, v         [R, Hkv, D] with row strides ldk, ldv in elements (views of
 *                a joint projection's output)
 *   slot         [R] (a negative slot, or one beyond the cache: row skipped)
 *   k_cache, v_cache   in/out
 *   codes        [n_pages, Hkv, D] int8 and scale [n_pages, Hkv] fp32, both or
 *                neither NULL.  When a row fills the last place of its page,
 *                the page's summary is set: with m the mean of its P keys
 *                (summed in binary64: exact for 16-bit keys whose exponents
 *                span less than 2^39),
 *                scale = 2^e, the least power of two with max |m| < 2^(e+7)
 *                that fp32 holds as a normal number (1 for m = 0; an m that
 *                is not finite counts as 0), and
 *                codes = m / scale rounded to the nearest whole number (ties
 *                to even), held in -127 .. 127.
 * Slots of a call must differ, and the rows of one page must follow each
 * other in the order of their slots, as sgdn_paged_plan lays them out.
 * Reads rows, batch is not used; table, width and max_len are not. */
int sgdn_paged_write(const sgdn_paged* p, const void* k, const void* v, int64_t ldk, int64_t ldv,
                     const int32_t* slot, void* k_cache, void* v_cache, int8_t* codes,
                     float* scale, void* stream);

/* Device workspace of sgdn_paged_attend (n_blocks = 0), of
 * sgdn_paged_attend_sparse (n_blocks > 0, select = 0) and of
 * sgdn_paged_select (select = 1).  0 for an invalid shape; 256 for a valid
 * one that uses none, where ws may be NULL (ws_bytes is then not looked at). */
size_t sgdn_paged_workspace_bytes(const sgdn_paged* p, int32_t n_blocks, int32_t select);

/* o[r, h] = sum_t softmax_t(scale q[r, h] . k[t, h']) v[t, h'] over the
 * row_len[r] tokens t of the row's request, h' the key/value head of h.
 *   q            [R, Hq, D] with row stride ldq in elements
 *   table        [B, W]
 *   row_req      [R] or NULL (request r; R <= B);  row_len [R]
 *   scale        of the scores, finite (also times log2(e))
 *   o            [R, Hq, D] o_dtype
 *   lse          [R, Hq] fp32 natural logarithm of the sum of exp(scale q.k),
 *                or NULL
 *   ws           at least sgdn_paged_workspace_bytes(p, 0, 0) bytes */
int sgdn_paged_attend(const sgdn_paged* p, const void* q, int64_t ldq, const void* k_cache,
                      const void* v_cache, const int32_t* table, const int32_t* row_req,
                      const int32_t* row_len, float scale, void* o, float* lse, void* ws,
                      size_t ws_bytes, void* stream);

/* The same over the tokens of the listed blocks only: those of the row's
 * first row_len[r] tokens that lie in a block of blocks[r, h'].
 *   blocks       [R, Hkv, n_blocks] block numbers of the row's request, in
 *                any order, -1 for none.  A block listed twice counts twice.
 * 1 <= n_blocks <= 4096. */
int sgdn_paged_attend_sparse(const sgdn_paged* p, const void* q, int64_t ldq, const void* k_cache,
                             const void* v_cache, const int32_t* table, const int32_t* row_req,
                             const int32_t* row_len, const int32_t* blocks, int32_t n_blocks,
                             float scale, void* o, float* lse, void* ws, size_t ws_bytes,
                             void* stream);

/* Picks n_blocks blocks for each row and key/value head by a cheap score.
 * Of the nb = ceil(row_len / P) blocks that the row sees, the first n_sink
 * and the last n_local are always picked; the others are ranked by
 *     max over the group's query heads of  (q8 . codes_j) sq scale_j
 * with q8, sq the codes and the power of two of the query vector, formed as a
 * page summary's are (not finite elements count as 0).  The scores are exact
 * and the choice does not depend on any order of evaluation; equal scores go
 * to the lower block, a score that is not a number ranks last.  Exact is
 * meant for scale_j up to 2^121, the largest that sgdn_paged_write makes, and
 * for sq and sq scale_j of at least 2^-133 times the largest sq of the group's
 * heads (always so where the heads' largest elements lie within 2^7 of each
 * other); scores of a head or a summary below that are rounded in fp32.
 *   codes, scale of sgdn_paged_write
 *   blocks       [R, Hkv, n_blocks] out: min(n_blocks, nb) blocks in rising
 *                order, then -1
 * n_local >= 1 (a row's last block may be incomplete and without a summary),
 * n_sink >= 0, n_sink + n_local <= n_blocks <= 4096, ceil(max_len / P) <=
 * 16384.  ws: at least sgdn_paged_workspace_bytes(p, n_blocks, 1) bytes. */
int sgdn_paged_select(const sgdn_paged* p, const void* q, int64_t ldq, const int8_t* codes,
                      const float* scale, const int32_t* table, const int32_t* row_req,
                      const int32_t* row_len, int32_t n_blocks, int32_t n_sink, int32_t n_local,
                      int32_t* blocks, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SGDN_ATTN_H */
