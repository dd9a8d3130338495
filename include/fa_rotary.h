/*
 * fa_rotary.h - C ABI of rotary positions: queries and keys turned, and keys turned on their way into
 * the paged 8-bit cache.  Status codes, element types and the device status word are those of fa.h,
 * the cache is that of fa_paged.h; what that header says of streams, captures and bad
 * device data holds here too.
 *
 * The first `dim` = 2 h channels of a head are turned in h pairs by the angle that the token's
 * position p and the pair's index give:
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * Pairs are the channels (i, i + h), or (2 i, 2 i + 1) where `interleaved`; the others are left.  Every
 * product and sum is rounded to fp32, the result once to its type.
 */
#ifndef FA_GB300_FA_ROTARY_H
#define FA_GB300_FA_ROTARY_H

#include "fa_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * table [num_positions, dim] fp32, contiguous, 16-byte aligned: row p holds cos of the h angles, then sin
 * (both times a factor, where the frequencies are scaled for long contexts and that comes
 * with one).  positions [T] int32: a token's row; negative: the token is not turned (a row of padding); from
 * num_positions on: not turned, and the device status becomes FA_ERR_INVALID_ARG.
 * dim: a multiple of 16 from 16 to 512, at most the head's width.  inverse: turned by the opposite angle (the gradient of
 * the turn with respect to its input).
 */
typedef struct fa_rotary {
    const float* table;
    const int* positions;
    int num_positions;
    int dim;
    int interleaved;
    int inverse;
} fa_rotary;

/* x, y: [T, heads, d] 16-bit, d contiguous, {token, head} strides in elements, positive multiples of 8,
 * 16-byte aligned.  y is x with the same strides (in place; FA_ERR_INVALID_ARG with others), or does not overlap it. */
typedef struct fa_rotary_part {
    const void* x;
    void* y;
    long long x_stride[2];
    long long y_stride[2];
    int heads;
} fa_rotary_part;

/*
 * fa_rotary_embed - one or two parts (queries and keys; k NULL: q alone) turned, in one launch.
 * d: head width of both, a multiple of 8, at most 512.  T >= 0 (0: nothing is launched).
 */
int fa_rotary_embed(const fa_rotary* rotary, const fa_rotary_part* q, const fa_rotary_part* k, int T, int d,
                    int dtype, void* stream);

/*
 * fa_kv_cache_append_rotary - fa_kv_cache_append of keys that are turned first (in fp32: a
 * value is rounded once, to e4m3), and, unless q is NULL, queries [T, heads, cache->d] turned as fa_rotary_embed
 * does: in the same launch, or where there are many in one of their own behind it (a call that returns an error has turned
 * none of them).  inverse is not taken (FA_ERR_INVALID_ARG).
 */
int fa_kv_cache_append_rotary(const fa_kv_cache* cache, const void* k, const void* v, const int* slots, int T,
                              const long long* k_stride, const long long* v_stride, const fa_rotary* rotary,
                              const fa_rotary_part* q, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_FA_ROTARY_H */
