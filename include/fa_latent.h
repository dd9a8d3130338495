/*
 * fa_latent.h - C ABI of latent attention: keys and values of all heads come from one shared latent vector per
 * token (C channels), and R more key channels, which carry the position, are shared too.
 * Absorbed form: the projections of latents to keys and values are multiplied into the queries and the output, so a
 * head's query has C + R channels, its key is the token's row of the cache and its value the first C channels of that.
 * Expanded form: keys (Dn channels) and values (Dv) are laid out per head again.  Decoding reads least in the first,
 * prompts compute least in the second.
 * Status codes, element types and the device status word are those of fa.h; what fa_paged.h says of
 * streams, captures and bad device data holds here too.
 */
#ifndef FA_GB300_FA_LATENT_H
#define FA_GB300_FA_LATENT_H

#include "fa_rotary.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Pages of P tokens (P = 16, 32, 64 or 128): rows [num_pages, P, C + R] 16-bit, contiguous, 16-byte aligned; C =
 * value_dim and R = rope_dim: multiples of 8 (C >= 8, R >= 0), C at most 512, C + R at most 576.  Slots, block tables and
 * lengths are those of fa_paged.h (fa_kv_tables_step keeps them).  num_pages * P must be below 2^31.
 */
typedef struct fa_latent_cache {
    void* rows;
    int num_pages;
    int page_size;
    int value_dim;
    int rope_dim;
} fa_latent_cache;

/*
 * fa_latent_cache_append - rows of T tokens written into their slots (negative: not stored; beyond the cache:
 * reported and not stored; a slot that a call names twice may hold parts of both rows).
 * latent [T, C], rope [T, R] 16-bit, channels contiguous, token strides in elements (positive multiples of 8), 16-byte aligned.
 * rotary NULL: the R channels are stored as they are.  Else dim must be R, and they are turned (inverse is not taken);
 * q, if given, is [T, heads, R], turned in the same launch.  rope may be NULL where R = 0.
 */
int fa_latent_cache_append(const fa_latent_cache* cache, const void* latent, long long latent_stride, const void* rope,
                           long long rope_stride, const int* slots, int T, const fa_rotary* rotary,
                           const fa_rotary_part* q, int dtype, void* stream);

/*
 * fa_latent_paged_fwd - absorbed form: O = softmax(scale q c^T) c[:, :C] and the natural log-sum-exp of each
 * request's new queries over its cached rows c.  q [T, H, C + R], o [T, H, C], lse [T, H]; strides, cu_q, lens,
 * block_table, causal, scale, T = 0 and rows that are no request's: as in fa_paged_fwd.
 * dtype is the cache's type too.  Made for few new tokens per request (a unit of work is 128 heads x tokens); whole prompts
 * take any length, but cost less in the expanded form.
 * The softmax runs in 32 bits; its weights enter the second product in the 16-bit type, scaled so that fp16 keeps 11 bits
 * down to 2^-20 of a row's largest.
 * Places of a page behind a request's last token may hold anything; a NaN or infinity in a row that only the
 * causal mask hides may reach the query.
 * workspace: device memory of at least fa_latent_paged_workspace_size bytes, 256-byte aligned, not to be shared by
 * calls that may run at the same time.  B <= 16384.
 */
typedef struct fa_latent_paged_args {
    const void* q;
    void* o;
    float* lse;
    const int* cu_q;
    const int* block_table;
    const int* lens;
    fa_latent_cache cache;
    long long q_stride[2];
    long long o_stride[2];
    int T, B, H, max_q, max_pages;
    float scale;
    int causal;
    int dtype;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
} fa_latent_paged_args;

int fa_latent_paged_fwd(const fa_latent_paged_args* args);
size_t fa_latent_paged_workspace_size(const fa_latent_paged_args* args);

/*
 * fa_latent_fwd - expanded form, ragged requests behind one another: O = softmax(scale (q[:Dn] k^T + q[Dn:] k_rope^T)) v.
 *   q [T, H, Dn + R], k [Tk, H, Dn], v [Tk, H, Dv], o [T, H, Dv]: 16-bit, channels contiguous, {token, head} strides in
 *     elements, positive multiples of 8, 16-byte aligned; k_rope [Tk, R] with a token stride; lse [T, H] fp32 contiguous.
 *     Dn and Dv: multiples of 8 from 8 to 128, R: a multiple of 8 from 8 to 64.
 *   cu_q, cu_k [B + 1] int32: request b's queries are rows cu_q[b] .. cu_q[b + 1] - 1 (at most max_q), its keys rows
 *     cu_k[b] .. cu_k[b + 1] - 1 of k, k_rope and v, its new tokens' own last.  max_k: about the longest request's keys (a
 *     hint for the order of work; any value >= 1 gives the same results).
 *   causal: query i of nq sees keys j <= i + nk - nq.  A query that sees no key gets O = 0 and LSE = -inf.
 * Softmax and its weights as in fa_latent_paged_fwd.
 * Keys of one request never reach another, whatever they hold; a NaN or infinity in a value that only the causal mask
 * hides may reach its own request's queries.  Rows of o and lse that are no request's are left as they were.
 * A request with marks that cannot be is reported and has no output.
 */
typedef struct fa_latent_args {
    const void* q;
    const void* k;
    const void* k_rope;
    const void* v;
    void* o;
    float* lse;
    const int* cu_q;
    const int* cu_k;
    long long q_stride[2];
    long long k_stride[2];
    long long v_stride[2];
    long long o_stride[2];
    long long k_rope_stride;
    int T, Tk, B, H, Dn, R, Dv, max_q, max_k;
    float scale;
    int causal;
    int dtype;
    void* stream;
} fa_latent_args;

int fa_latent_fwd(const fa_latent_args* args);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_FA_LATENT_H */
