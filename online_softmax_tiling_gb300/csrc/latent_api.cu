// latent_api.cu - host side of include/fa_latent.h and of fa_rotary_embed: argument checks, tensor maps, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "../../include/fa_latent.h"
#include "host_common.h"
#include "latent_append.cuh"
#include "latent_fwd_kernel.cuh"
#include "latent_paged_kernel.cuh"
#include "rotary_host.h"

namespace {

// 16-bit [rows, cols] (or [heads, rows, cols]) with element strides as a 4-D map; columns >= cols and rows >= rows read as zeros.
bool encode_rows(CUtensorMap* map, const void* ptr, bool bf16, int64_t cols, int64_t rows, int64_t heads, int64_t row_stride,
                 int64_t head_stride, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(heads), 1};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(row_stride) * 2, static_cast<cuuint64_t>(head_stride) * 2,
                                   static_cast<cuuint64_t>(head_stride) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(ptr), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_cache(CUtensorMap* map, const fa_latent_cache& c, bool bf16, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t W = static_cast<cuuint64_t>(c.value_dim + c.rope_dim);
    const cuuint64_t dims[2] = {W, static_cast<cuuint64_t>(c.num_pages) * c.page_size};
    const cuuint64_t strides[1] = {W * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, c.rows, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same in boxes of four 64-channel pieces, piece after piece (W a multiple of 64).
bool encode_cache_pieces(CUtensorMap* map, const fa_latent_cache& c, bool bf16, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t W = static_cast<cuuint64_t>(c.value_dim + c.rope_dim);
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(c.num_pages) * c.page_size, W / 64};
    const cuuint64_t strides[2] = {W * 2, 128};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 4};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, c.rows, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [T, H, W] in boxes of 64 channels x `box` heads of one token.
bool encode_queries(CUtensorMap* map, const fa_latent_paged_args& a, bool bf16, int box_heads) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.cache.value_dim + a.cache.rope_dim), static_cast<cuuint64_t>(a.H), static_cast<cuuint64_t>(a.T)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.q_stride[1]) * 2, static_cast<cuuint64_t>(a.q_stride[0]) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_latent_cache(const fa_latent_cache& c) {
    if (!c.rows || c.num_pages < 1 || shift_of(c.page_size) < 0) return FA_ERR_INVALID_ARG;
    if (c.value_dim < 8 || c.value_dim > 512 || c.value_dim % 8 != 0 || c.rope_dim < 0 || c.rope_dim % 8 != 0 ||
        c.value_dim + c.rope_dim > 576)
        return FA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c.num_pages) * c.page_size > INT32_MAX) return FA_ERR_INVALID_ARG;
    return misaligned(c.rows, 16) ? FA_ERR_MISALIGNED : FA_OK;
}
bool bad_stride(long long s) { return s <= 0 || s % 8 != 0 || s >= (1ll << 39); }

// ---- absorbed form
struct LatentPlan {
    int pairs, min_share;
};
// Shares of at least kMinShare tiles, so that a short context is not cut into more parts than the join reads quickly (one
// request of 4096 keys: 13.4 us with 2, 13.7 with 1, 14.8 with 3).
constexpr int kMinShare = 2;
int64_t most_tiles(const fa_latent_paged_args& a) {
    const int64_t blocks = (static_cast<int64_t>(a.max_q) * a.H + pg::kLatRows - 1) / pg::kLatRows;
    const int64_t tiles = std::max<int64_t>(1, (static_cast<int64_t>(a.max_pages) * a.cache.page_size + pg::kLatKeys - 1) / pg::kLatKeys);
    return a.B * blocks * tiles;
}
LatentPlan latent_plan(const fa_latent_paged_args& a) {
    LatentPlan pl;
    pl.min_share = kMinShare;
    pl.pairs = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sm_count() / 2, (most_tiles(a) + pl.min_share - 1) / pl.min_share)));
    return pl;
}
size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
size_t part_bytes(const fa_latent_paged_args& a, const LatentPlan& pl) {
    return static_cast<size_t>(pg::lat_part(2ll * pl.pairs, 0, 0, 0, a.cache.value_dim)) * 16;
}
size_t latent_workspace(const fa_latent_paged_args& a, const LatentPlan& pl) {
    if (pl.pairs < 2) return 0;
    return part_bytes(a, pl) + round256(2ull * pl.pairs * pg::kLatRows * 8) + static_cast<size_t>(pl.pairs) * 32;
}

int check_latent_paged(const fa_latent_paged_args& a) {
    const bool none = a.T == 0;
    if (!none && (!a.q || !a.o || !a.lse)) return FA_ERR_INVALID_ARG;
    if (!(none && a.B == 0) && (!a.block_table || !a.lens)) return FA_ERR_INVALID_ARG;
    if (a.B < (none ? 0 : 1) || a.T < 0 || a.H < 1 || a.max_q < (none ? 0 : 1) || a.max_pages < 1) return FA_ERR_INVALID_ARG;
    if (a.dtype != FA_FP16 && a.dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(a.scale) || !(a.scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (!a.cu_q && (a.T != a.B || (!none && a.max_q != 1))) return FA_ERR_INVALID_ARG;
    const int st = check_latent_cache(a.cache);
    if (st != FA_OK) return st;
    if (a.max_pages > kMostKeys / a.cache.page_size) return FA_ERR_INVALID_ARG;
    if (a.B > pg::kLatMaxB) return FA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(a.max_q) * a.H > INT32_MAX / 2 || static_cast<int64_t>(a.T) * a.H > INT32_MAX) return FA_ERR_INVALID_ARG;
    if (most_tiles(a) > INT32_MAX) return FA_ERR_INVALID_ARG;  // (tiles of all units are counted in 32 bits)
    if (bad_strides(a.q_stride) || bad_strides(a.o_stride) || misaligned(a.q, 16) || misaligned(a.o, 16) || misaligned(a.lse, 4) ||
        misaligned(a.block_table, 4) || misaligned(a.lens, 4) || misaligned(a.cu_q, 4))
        return FA_ERR_MISALIGNED;
    return FA_OK;
}

int check_latent(const fa_latent_args& a) {
    const bool none = a.T == 0;
    if (!none && (!a.q || !a.k || !a.k_rope || !a.v || !a.o || !a.lse)) return FA_ERR_INVALID_ARG;
    if (!(none && a.B == 0) && (!a.cu_q || !a.cu_k)) return FA_ERR_INVALID_ARG;
    if (a.B < (none ? 0 : 1) || a.T < 0 || a.Tk < 0 || a.H < 1 || a.max_q < (none ? 0 : 1) || a.max_k < (none ? 0 : 1)) return FA_ERR_INVALID_ARG;
    if (a.dtype != FA_FP16 && a.dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(a.scale) || !(a.scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (a.Dn < 8 || a.Dn > 128 || a.Dn % 8 != 0 || a.Dv < 8 || a.Dv > 128 || a.Dv % 8 != 0 || a.R < 8 || a.R > 64 || a.R % 8 != 0)
        return FA_ERR_UNSUPPORTED;
    if (a.max_q > kMostKeys || a.T > kMostKeys || a.Tk > kMostKeys || static_cast<int64_t>(a.T) * a.H > INT32_MAX) return FA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(a.B) * a.H * ((a.max_q + 255) / 256) > INT32_MAX / 2) return FA_ERR_INVALID_ARG;
    if (bad_strides(a.q_stride) || bad_strides(a.k_stride) || bad_strides(a.v_stride) || bad_strides(a.o_stride) || bad_stride(a.k_rope_stride))
        return FA_ERR_MISALIGNED;
    for (const void* t : {a.q, a.k, a.k_rope, a.v, static_cast<const void*>(a.o)})
        if (misaligned(t, 16)) return FA_ERR_MISALIGNED;
    if (misaligned(a.lse, 4) || misaligned(a.cu_q, 4) || misaligned(a.cu_k, 4)) return FA_ERR_MISALIGNED;
    return FA_OK;
}

}  // namespace

// Read and clear the status word of this file's kernels (the caller has synchronised).
__attribute__((visibility("hidden"))) bool fa_latent_take_status(unsigned int* out) {
    const unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(out, pg::g_paged_status, sizeof(*out)) != cudaSuccess) return false;
    return *out == 0 || cudaMemcpyToSymbol(pg::g_paged_status, &zero, sizeof(zero)) == cudaSuccess;
}

extern "C" {

int fa_rotary_embed(const fa_rotary* rotary, const fa_rotary_part* q, const fa_rotary_part* k, int T, int d, int dtype, void* stream) {
    if (!q || T < 0) return FA_ERR_INVALID_ARG;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    if (d < 16 || d > 512 || d % 8 != 0) return FA_ERR_UNSUPPORTED;
    int st = check_rotary(rotary, d, T);
    if (st == FA_OK) st = check_part(q, T);
    if (st == FA_OK && k) st = check_part(k, T);
    if (st != FA_OK) return st;
    if (T == 0) return FA_OK;
    return launch_rotary(rotary_work(*rotary, q, k, T, d), dtype == FA_BF16, stream);
}

int fa_latent_cache_append(const fa_latent_cache* cache, const void* latent, long long latent_stride, const void* rope,
                           long long rope_stride, const int* slots, int T, const fa_rotary* rotary, const fa_rotary_part* q, int dtype,
                           void* stream) {
    if (!cache || T < 0 || (q && !rotary)) return FA_ERR_INVALID_ARG;
    if (T > 0 && (!latent || !slots || (!rope && cache->rope_dim > 0))) return FA_ERR_INVALID_ARG;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    int st = check_latent_cache(*cache);
    const int C = cache->value_dim, R = cache->rope_dim;
    if (st == FA_OK && rotary) {
        if (rotary->inverse || rotary->dim != R) return FA_ERR_INVALID_ARG;
        st = check_rotary(rotary, R, T);
        if (st == FA_OK && q) st = check_part(q, T);
    }
    if (st != FA_OK) return st;
    if (T > kMostKeys) return FA_ERR_INVALID_ARG;
    if (bad_stride(latent_stride) || (R > 0 && bad_stride(rope_stride)) || misaligned(latent, 16) || misaligned(rope, 16) || misaligned(slots, 4))
        return FA_ERR_MISALIGNED;
    if (T == 0) return FA_OK;
    pg::LatentAppendParams p = {};
    p.latent = static_cast<const uint16_t*>(latent), p.rope = static_cast<const uint16_t*>(rope);
    p.latent_st = latent_stride, p.rope_st = rope_stride;
    p.cache = static_cast<uint16_t*>(cache->rows);
    p.slots = slots;
    p.T = T, p.C = C, p.R = R, p.num_slots = cache->num_pages * cache->page_size;
    if (rotary) p.r = rotary_table(*rotary);
    int64_t q_ctas = 0;
    bool single = true;
    if (q) {
        p.q = rotary_work(*rotary, q, nullptr, T, R);
        single = set_groups(p.q) == 1;
        const int64_t items = static_cast<int64_t>(T) * p.q.groups * (p.q.cols + p.q.tail);
        if (items > INT32_MAX) return FA_ERR_INVALID_ARG;
        q_ctas = (items + pg::kRotaryThreads - 1) / pg::kRotaryThreads;
    }
    const int64_t items = static_cast<int64_t>(T) * (C / 8 + (rotary ? R / 16 : R / 8));
    const int64_t ctas = (items + pg::kRotaryThreads - 1) / pg::kRotaryThreads;
    if (items > INT32_MAX || ctas + q_ctas > INT32_MAX) return FA_ERR_INVALID_ARG;
    p.latent_ctas = static_cast<int>(ctas);
    const bool bf16 = dtype == FA_BF16;
    const void* fn = single ? (bf16 ? reinterpret_cast<const void*>(&pg::latent_append_kernel<1, true>) : reinterpret_cast<const void*>(&pg::latent_append_kernel<1, false>))
                            : (bf16 ? reinterpret_cast<const void*>(&pg::latent_append_kernel<pg::kRotaryHeads, true>)
                                    : reinterpret_cast<const void*>(&pg::latent_append_kernel<pg::kRotaryHeads, false>));
    void* args[] = {&p};
    return launch(fn, ctas + q_ctas, 1, pg::kRotaryThreads, 0, 1, stream, args) ? FA_OK : FA_ERR_CUDA;
}

size_t fa_latent_paged_workspace_size(const fa_latent_paged_args* a) {
    if (!a || check_latent_paged(*a) != FA_OK || a->T == 0) return 0;
    return latent_workspace(*a, latent_plan(*a));
}

int fa_latent_paged_fwd(const fa_latent_paged_args* args) {
    if (!args) return FA_ERR_INVALID_ARG;
    const fa_latent_paged_args& a = *args;
    const int st = check_latent_paged(a);
    if (st != FA_OK) return st;
    if (a.T == 0) return FA_OK;
    const LatentPlan pl = latent_plan(a);
    const size_t need = latent_workspace(a, pl);
    if (need > 0) {
        if (!a.workspace) return FA_ERR_INVALID_ARG;
        if (misaligned(a.workspace, 256)) return FA_ERR_MISALIGNED;
        if (a.workspace_bytes < need) return FA_ERR_INVALID_ARG;
    }
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return FA_ERR_CUDA;
    const bool bf16 = a.dtype == FA_BF16;
    pg::LatentParams p = {};
    p.q = static_cast<const uint16_t*>(a.q), p.o = static_cast<uint16_t*>(a.o), p.lse = a.lse;
    p.cu_q = a.cu_q, p.table = a.block_table, p.lens = a.lens;
    p.cache = static_cast<const uint16_t*>(a.cache.rows);
    p.q_st = a.q_stride[0], p.q_sh = a.q_stride[1], p.o_st = a.o_stride[0], p.o_sh = a.o_stride[1];
    p.T = a.T, p.B = a.B, p.H = a.H, p.C = a.cache.value_dim, p.W = a.cache.value_dim + a.cache.rope_dim;
    p.max_q = a.max_q, p.max_pages = a.max_pages, p.num_pages = a.cache.num_pages, p.page_shift = shift_of(a.cache.page_size);
    p.min_share = pl.min_share;
    p.box_rows = std::min(a.cache.page_size, 64);
    p.causal = a.causal != 0;
    p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    if (need > 0) {
        char* ws = static_cast<char*>(a.workspace);
        p.o_part = reinterpret_cast<float4*>(ws);
        ws += part_bytes(a, pl);
        p.stats = reinterpret_cast<float2*>(ws);
        p.shares = reinterpret_cast<int4*>(ws + round256(2ull * pl.pairs * pg::kLatRows * 8));
    } else {
        p.min_share = INT32_MAX;  // one pair: all of it
    }
    CUtensorMap tm, tm_k = {}, tm_q = {};
    if (!encode_cache(&tm, a.cache, bf16, p.box_rows)) return FA_ERR_CUDA;
    // four pieces of keys in one load, where a page has a CTA's 64 keys and pieces end with the row
    p.box_pieces = p.box_rows == 64 && p.W % 64 == 0 ? 4 : 1;
    if (p.box_pieces > 1 && !encode_cache_pieces(&tm_k, a.cache, bf16, p.box_rows)) return FA_ERR_CUDA;
    // boxes of queries: as many heads as divide both H and a CTA's 64 rows, a whole swizzle pattern (eight rows) at least
    int box = 64;
    while (a.H % box != 0) box /= 2;
    p.q_box = box >= 8 ? box : 0;
    if (p.q_box && !encode_queries(&tm_q, a, bf16, p.q_box)) return FA_ERR_CUDA;
    const void* fn = bf16 ? reinterpret_cast<const void*>(&pg::latent_paged_kernel<true>) : reinterpret_cast<const void*>(&pg::latent_paged_kernel<false>);
    void* kargs[] = {&tm, &tm_k, &tm_q, &p};
    if (!ensure_smem(fn, pg::kLatSmem, device) || !launch(fn, 2ll * pl.pairs, 1, pg::kLatThreads, pg::kLatSmem, 2, a.stream, kargs))
        return FA_ERR_CUDA;
    if (need > 0) {
        // units cut into eight parts and more: a CTA per job of the join
        const int64_t units = a.B * ((static_cast<int64_t>(a.max_q) * a.H + pg::kLatRows - 1) / pg::kLatRows);
        const bool split = 8 * units <= pl.pairs;
        const int jobs = 8 * pg::lat_chunks(p.C);
        const void* join = split ? (bf16 ? reinterpret_cast<const void*>(&pg::latent_join_kernel<true, true>)
                                         : reinterpret_cast<const void*>(&pg::latent_join_kernel<false, true>))
                                 : (bf16 ? reinterpret_cast<const void*>(&pg::latent_join_kernel<true, false>)
                                         : reinterpret_cast<const void*>(&pg::latent_join_kernel<false, false>));
        void* jargs[] = {&p};
        if (!launch(join, pl.pairs - 1, split ? jobs : jobs / pg::kLatJoinWarps, 32 * pg::kLatJoinWarps, 0, 1, a.stream, jargs))
            return FA_ERR_CUDA;
    }
    return FA_OK;
}

int fa_latent_fwd(const fa_latent_args* args) {
    if (!args) return FA_ERR_INVALID_ARG;
    const fa_latent_args& a = *args;
    const int st = check_latent(a);
    if (st != FA_OK) return st;
    if (a.T == 0) return FA_OK;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return FA_ERR_CUDA;
    const bool bf16 = a.dtype == FA_BF16;
    pg::LatentFwdParams p = {};
    p.o = static_cast<uint16_t*>(a.o), p.lse = a.lse, p.cu_q = a.cu_q, p.cu_k = a.cu_k;
    p.o_st = a.o_stride[0], p.o_sh = a.o_stride[1];
    p.T = a.T, p.Tk = a.Tk, p.B = a.B, p.H = a.H, p.Dn = a.Dn, p.Dv = a.Dv, p.max_q = a.max_q;
    p.pieces = (a.Dn + 63) / 64 + 1, p.half_v = (a.Dv + 31) / 32 * 16;
    p.q_blocks = (a.max_q + pg::kLfRows - 1) / pg::kLfRows;
    // Blocks of all requests, at most: where that is well below one for every request and block of the longest, the kernel
    // counts them (a prompt among many short ones).
    const int64_t blocks = static_cast<int64_t>(a.B) * p.q_blocks, most = a.T / pg::kLfRows + static_cast<int64_t>(a.B);
    p.compact = a.B <= pg::kLfMaxB && 2 * most <= blocks;
    const int64_t units = a.H * (p.compact ? most : blocks);
    p.causal = a.causal != 0;
    p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    // (request, head) pairs in groups of equal size whose keys and values come to about 96 MB (of 129 MB of L2).  Fewer and
    // larger groups leave the pairs of CTAs more even work at the end: 32 heads, pieces of 4000 and 2516 queries 328 us with
    // groups of 96 MB, 344 with 48, 349 without (197 MB).
    const int64_t all = static_cast<int64_t>(a.B) * a.H;
    const double bytes = 2.0 * all * std::max(a.max_k, 1) * (a.Dn + a.Dv);  // (max_k is any hint: beyond 64 bits)
    const int64_t groups = static_cast<int64_t>(std::max(1.0, std::min<double>(all, std::floor(bytes / (96 << 20) + 0.5))));
    p.group = static_cast<int>(std::min<int64_t>((all + groups - 1) / groups, INT32_MAX / p.q_blocks));
    CUtensorMap tq, tk, ts, tv;
    const int keys = std::max(a.Tk, 1);  // (no key at all: nothing is read)
    if (!encode_rows(&tq, a.q, bf16, a.Dn + a.R, a.T, a.H, a.q_stride[0], a.q_stride[1], 128) ||
        !encode_rows(&tk, a.k, bf16, a.Dn, keys, a.H, a.k_stride[0], a.k_stride[1], 32) ||
        !encode_rows(&ts, a.k_rope, bf16, a.R, keys, 1, a.k_rope_stride, a.k_rope_stride, 32) ||
        !encode_rows(&tv, a.v, bf16, a.Dv, keys, a.H, a.v_stride[0], a.v_stride[1], 128))
        return FA_ERR_CUDA;
    const void* fn = bf16 ? reinterpret_cast<const void*>(&pg::latent_fwd_kernel<true>) : reinterpret_cast<const void*>(&pg::latent_fwd_kernel<false>);
    void* kargs[] = {&tq, &tk, &ts, &tv, &p};
    if (!ensure_smem(fn, pg::kLfSmem, device) ||
        !launch(fn, 2 * units, 1, pg::kLfThreads, pg::kLfSmem, 2, a.stream, kargs))
        return FA_ERR_CUDA;
    return FA_OK;
}

}  // extern "C"
