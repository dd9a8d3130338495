/*
 * fa_paged.h - C ABI of the serving operators around a paged key/value cache
 * held in 8 bits: one step's block tables and slots, the quantising append,
 * attention over the cache, and the choice of pages for sparse attention.
 * Status codes, element types and the device status word are those of fa.h.
 *
 * The cache.  Pages of P tokens (P = 16, 32, 64 or 128):
 *   k, v             [num_pages, Hk, P, d] e4m3, contiguous, 16-byte aligned
 *   k_scale, v_scale [num_pages, Hk] fp32: a value is code * scale.  The
 *                    append writes powers of two in [2^-60, 2^60]; the
 *                    attention takes any scale in that range (one outside of
 *                    it counts as the nearer end).
 *   k_bounds         [num_pages, Hk, 2, d] int8, 16-byte aligned, only for
 *                    sparse attention (else NULL): per channel the floor of
 *                    (least code)/4 and the ceiling of (largest code)/4 over
 *                    the page's tokens.
 * Hk: key/value heads; d: a multiple of 16 from 16 to 256.  Token j of
 * request b is at place j % P of page block_table[b][j / P]; a slot is
 * page * P + place.  num_pages * Hk * P must be below 2^31, max_pages * P (and
 * the tokens of one append) at most 2^30.
 *
 * Device data that no entry point can check on the host (lengths, tables,
 * slots) is checked by the kernels: nothing outside the buffers is read or
 * written, and the call's device status becomes FA_ERR_INVALID_ARG
 * (fa_check_device_status).
 * Every entry point enqueues on `stream`, on the current device, allocates
 * nothing and keeps no pointer; all may be captured in CUDA graphs after a
 * call with the same sizes outside of a capture (which sets kernel attributes).
 */
#ifndef FA_GB300_FA_PAGED_H
#define FA_GB300_FA_PAGED_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Device-side status of fa_kv_tables_step: not enough free pages. */
#define FA_ERR_NO_PAGES 6

typedef struct fa_kv_cache {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    signed char* k_bounds; /* or NULL */
    int num_pages;
    int page_size;
    int Hk;
    int d;
} fa_kv_cache;

/*
 * fa_kv_tables_step - bookkeeping of one serving step for B requests.
 * new_tokens [B]: n >= 0 adds n tokens to the request, n < 0 ends it.
 * lens [B]: tokens held before the step.  block_table [B, max_pages]: the
 * first ceil(lens / P) entries of a row are the request's pages.
 * free_pages [free_capacity]: a stack of which the first *free_count entries
 * are free pages.  First the pages of the requests that end are pushed, in
 * order of request and page; then every page the step needs is popped, in
 * the same order, and written into its row of block_table.
 * Written: cu_new [B + 1] (prefix sums of the tokens added, as
 * fa_paged_args.cu_q takes them), slots [max_tokens] (the slot of every new
 * token, -1 behind the last), lens_out [B] (0 where a request ended),
 * free_count_out [1], and status [1] (device memory).  lens_out and
 * free_count_out must not be lens and free_count: the step can be repeated.
 * status: FA_OK; FA_ERR_NO_PAGES (too few free pages); FA_ERR_INVALID_ARG (a
 * negative length, more than max_tokens tokens, a row longer than max_pages
 * or a stack longer than free_capacity).  Where it is not FA_OK nothing is
 * allocated or released: cu_new is 0, slots are -1, lens_out is lens and
 * free_count_out is free_count.
 * The step knows no cache, so of a page number it checks that 32 bits hold its
 * slots (0 <= page < 2^31 / P): new tokens on another one get slot -1, with the
 * device status FA_ERR_INVALID_ARG and everything else as for a sound page.  A number
 * beyond the cache's pages is caught by the append and the attention.
 * 1 <= B <= 16384; max_tokens >= 0.  One kernel launch.
 */
int fa_kv_tables_step(const int* new_tokens, const int* lens, int* block_table, int* free_pages,
                      const int* free_count, int B, int max_pages, int free_capacity,
                      int page_size, int max_tokens, int* slots, int* cu_new, int* lens_out,
                      int* free_count_out, int* status, void* stream);

/*
 * fa_kv_cache_append - quantise T new keys and values into their slots.
 * k, v: [T, Hk, d] 16-bit (dtype), d contiguous; k_stride, v_stride = {token,
 * head} strides in elements, positive multiples of 8; 16-byte aligned.
 * slots [T] int32 as fa_kv_tables_step writes them; negative: not stored.
 * The tokens of one page must follow one another in the call with slots
 * ascending by one: a page holds no gaps.  Rows that are not stored may stand
 * between them, fewer than 128 in a row.  A token whose slot is of the same
 * page as the token's before it, but not the next one, is reported (device status
 * FA_ERR_INVALID_ARG) and not stored, nor are those that go on from it.  A page
 * written from two places of one call (other pages' tokens, or 128 and more rows
 * that are not stored, between them) is a race.
 * The scale of (page, head) is the smallest power of two s in [2^-60, 2^60]
 * with |x| <= 448 s for every finite x stored there.  A write to place 0
 * starts a page anew.  Otherwise the scale never shrinks; where it grows, the
 * page's older codes (places before the first one written) are rounded again
 * to the new scale.  Codes are rounded to nearest even; a value beyond 448 s
 * (an infinity among them) is stored as +-448 s, NaN as NaN.  k_bounds, if
 * given, follows the codes (NaN counts as 0): the bounds that stand for the
 * page's older codes are widened by the new ones, or taken anew from all codes
 * up to the last one written where the page is new or its key scale grows.
 * T >= 0 (0: nothing is launched); Hk <= 32767.
 */
int fa_kv_cache_append(const fa_kv_cache* cache, const void* k, const void* v, const int* slots,
                       int T, const long long* k_stride, const long long* v_stride, int dtype,
                       void* stream);

/*
 * fa_paged_fwd - attention of each request's new queries over its cached
 * keys: O = softmax(scale q k^T) v and the natural log-sum-exp.
 *   q [T, Hq, d], o [T, Hq, d]: 16-bit, d contiguous, {token, head} strides
 *     in elements, positive multiples of 8, 16-byte aligned; Hq a multiple
 *     of Hk (query head h reads key head h / (Hq / Hk)).
 *   lse [T, Hq] fp32 contiguous.
 *   cu_q [B + 1] int32: request b's queries are rows cu_q[b] .. cu_q[b+1]-1
 *     (at most max_q of them); NULL: one query per request (T = B, max_q = 1).
 *   lens [B] int32: keys of each request, the new tokens' own included (at
 *     most max_pages * P).
 *   causal: 0 = every query sees all keys; else query i of nq sees keys
 *     j <= i + len - nq (the last one sees all).  A query that sees no key
 *     gets O = 0 and LSE = -inf.
 *   selected [B, Hk, num_selected] int32 with selected_count [B, Hk], or
 *     NULL: only these pages (indices into the request's row of block_table,
 *     ascending) are read for the key head; one query per request.
 *   num_splits: key ranges per row, 1 .. FA_PAGED_MAX_SPLITS; 0 = chosen from
 *     the sizes (fa_paged_num_splits), for requests about as long as the table is
 *     wide: where they are known to be much shorter, a smaller count is faster.
 *     workspace: device memory of at least fa_paged_workspace_size bytes,
 *     256-byte aligned, where that is not 0; not to be shared by calls that may
 *     run at the same time.
 *   scale: finite and > 0.
 * T = 0 (B >= 0): nothing is launched; q, o and lse (for B = 0 the table and lens
 * too) may be NULL and max_q 0.
 * Rows of o and lse that are no request's (before cu_q[0], which need not be 0, and
 * from cu_q[B] on) are left as they were.
 * The softmax runs in 32 bits; its weights enter the second product in fp16,
 * scaled so that a row's largest contribution keeps all of their 11 bits and
 * one 2^-22 as large still does, and 16-bit queries are read exactly (down
 * to 2^-38 of a row's largest value).
 * That holds as long as the value scales that a row reads lie within 2^96 of each
 * other (a page of zeros has the scale 2^-60); beyond that keys of the smallest scales may be
 * missing from the sum, and so from the LSE.
 * Places of a page behind a request's last token may hold anything.  As in
 * fa_fwd, a NaN or infinity in a value that a query does not see because of the causal
 * mask may still reach it (the product of its weight 0).
 * A request with bad device data (see above) has undefined outputs; the others have theirs.
 * Where a wait ran out (FA_ERR_TIMEOUT) all outputs of the call are undefined.
 */
#define FA_PAGED_MAX_SPLITS 64

typedef struct fa_paged_args {
    const void* q;
    void* o;
    float* lse;
    const int* cu_q;
    const int* block_table;
    const int* lens;
    const int* selected;
    const int* selected_count;
    fa_kv_cache cache;
    long long q_stride[2];
    long long o_stride[2];
    int T, B, Hq, max_q, max_pages, num_selected;
    float scale;
    int causal;
    int dtype;
    int num_splits;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
} fa_paged_args;

int fa_paged_fwd(const fa_paged_args* args);

/* The count of key ranges per row that fa_paged_fwd uses for num_splits = 0; 0 where
 * it shares the keys of all requests out evenly instead. */
int fa_paged_num_splits(const fa_paged_args* args);

/* Workspace bytes fa_paged_fwd needs with these arguments (0: none; a given count of 1,
 * 2, 4, 8 or 16 ranges of few query rows is joined on chip). */
size_t fa_paged_workspace_size(const fa_paged_args* args);

/*
 * fa_kv_page_select - the pages of each key head that one query per request
 * should read.  q [B, Hq, d] as in fa_paged_fwd.  For every query head the
 * values are rounded to whole numbers qi = rint(q / u), |qi| <= 127, with u
 * the smallest power of two in [2^-60, 2^60] that allows it (NaN counts as
 * 0); a page's score is
 *   max over the heads of a group of
 *     u * 4 k_scale * sum_c max(qi_c lo_c, qi_c hi_c)
 * with (lo, hi) = k_bounds: up to rounding of q an upper bound of q . k over
 * the page's keys, computed exactly (from 2^128 on: infinite).  Kept are the page of the
 * last token and the num_selected - 1 others with the largest scores (equal ones: the lower
 * index); all of them where a request has no more.
 * selected [B, Hk, num_selected] int32: ascending indices into the request's
 * row of block_table, -1 behind the last; selected_count [B, Hk].
 * Of the cache only k_scale, k_bounds and the sizes are used (k, v and
 * v_scale may be NULL).  B >= 1; 1 <= num_selected; max_pages <= 32768.
 */
int fa_kv_page_select(const fa_kv_cache* cache, const void* q, const long long* q_stride,
                      const int* block_table, const int* lens, int B, int Hq, int max_pages,
                      int num_selected, int dtype, int* selected, int* selected_count,
                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_FA_PAGED_H */
