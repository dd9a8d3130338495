// paged_api.cu - host side of include/fa_paged.h and of fa_kv_cache_append_rotary: argument checks, tensor
// maps, the choice of kernel and of key ranges, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "../../include/fa_paged.h"
#include "../../include/fa_rotary.h"
#include "host_common.h"
#include "kv_append.cuh"
#include "kv_page_select.cuh"
#include "kv_tables.cuh"
#include "paged_fwd_kernel.cuh"
#include "paged_prompt_kernel.cuh"
#include "paged_prompt_wide_kernel.cuh"
#include "rotary_host.h"

namespace {

namespace pg = fa::paged;

// Codes [rows, d] of a cache (rows = num_pages Hk P) as a 2-D map of bytes;
// columns >= d read as zeros.
bool encode_codes(CUtensorMap* map, const void* ptr, int64_t rows, int d, int box_cols, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The sizes of a cache: FA_OK, or what is wrong with them.
int check_sizes(const fa_kv_cache& c) {
    if (c.num_pages < 1 || c.Hk < 1 || shift_of(c.page_size) < 0) return FA_ERR_INVALID_ARG;
    if (c.d < 16 || c.d > 256 || c.d % 16 != 0) return FA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c.num_pages) * c.page_size > INT32_MAX / c.Hk) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

int check_cache(const fa_kv_cache& c) {
    if (!c.k || !c.v || !c.k_scale || !c.v_scale) return FA_ERR_INVALID_ARG;
    const int st = check_sizes(c);
    if (st != FA_OK) return st;
    if (misaligned(c.k, 16) || misaligned(c.v, 16) || misaligned(c.k_scale, 4) || misaligned(c.v_scale, 4) ||
        misaligned(c.k_bounds, 16))
        return FA_ERR_MISALIGNED;
    return FA_OK;
}

// Kernel width that serves d.
int width_of(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// Packed rows a CTA holds: 8 or 16 where those of a request fit, else 32 (each
// key is then read half as often as with 16), but 16 for d > 128, where a
// second accumulator does not fit the registers.
int block_rows_of(int width, int64_t rows) { return rows <= 8 ? 8 : width == 256 || rows <= 16 ? 16 : 32; }

struct Plan {
    bool prompt;    // a tcgen05 kernel (256 packed rows per unit, 128 for d > 128)
    int width, block_rows, row_blocks;
    int64_t units;  // row blocks x heads x requests
    int even;       // CTAs of equal shares of all keys (0: key ranges per row block)
};

// Packed rows above which the tcgen05 kernel serves a request: 8 requests of 4000
// keys and 8 heads take 35 us for 32 rows on the few-row kernel and 38 on the other, 52
// and 40 for 48 rows (which the few-row kernel reads every key twice for).  With d = 256 and
// 16 requests of up to 6000 keys, 8 heads: 140 and 121 us for 32 rows, 184 and 121 for 48
// (2 requests, 2 heads: 20 and 30, 21 and 30).
constexpr int kPromptRows = 32;

// CTAs that share all keys evenly, one wave of them, or 0 where ranges per row
// block do better: with few units (a unit's parts are joined one after the other),
// with so many that they even themselves out, or with few keys (the join is a second launch).
int even_ctas(const fa_paged_args& a, const Plan& pl) {
    const int64_t keys = static_cast<int64_t>(a.selected ? a.num_selected : a.max_pages) * a.cache.page_size;
    const int64_t wave = static_cast<int64_t>(sm_count()) * (pl.width == 256 || pl.block_rows == 32 ? 2 : 3);
    const int64_t chunk = pl.width == 256 ? 16 : 32;
    if (pl.prompt || pl.row_blocks != 1 || a.B > pg::kEvenMaxB) return 0;
    if (16 * pl.units < wave || 4 * pl.units > 5 * wave) return 0;
    // 64 chunks per CTA at least, by the tables' width (64 requests of 5000 to 16384 keys and 8 heads: 227 us
    // against 236 with 4 ranges; 32 of 4096 selected keys: 60 against 63; below, the second launch
    // costs more than it saves: 24 of up to 8000 keys and 4 heads, 41 us against 37)
    if (pl.units * (keys / chunk) < wave * 64 || pl.units * (keys / chunk) > INT32_MAX / 2) return 0;
    return static_cast<int>(wave);
}

Plan plan_of(const fa_paged_args& a) {
    Plan pl{};
    const int64_t rows = static_cast<int64_t>(a.max_q) * (a.Hq / a.cache.Hk);
    pl.width = width_of(a.cache.d);
    pl.prompt = rows > kPromptRows && !a.selected;
    pl.block_rows = !pl.prompt ? block_rows_of(pl.width, rows) : pl.width == 256 ? pg::kPwRows : pg::kPrRows;
    pl.row_blocks = static_cast<int>((rows + pl.block_rows - 1) / pl.block_rows);
    pl.units = static_cast<int64_t>(pl.row_blocks) * a.cache.Hk * a.B;
    pl.even = a.num_splits == 0 ? even_ctas(a, pl) : 0;
    return pl;
}

// The requests of a mixed call that bring no more than `rows` packed rows.
Plan single_token_plan(const fa_paged_args& a, int width, int rows) {
    Plan pl{};
    pl.width = width, pl.block_rows = rows, pl.row_blocks = 1;
    pl.units = static_cast<int64_t>(a.cache.Hk) * a.B;
    return pl;
}

// Whether the ranges of a row block are joined inside a cluster.
bool in_cluster(const Plan& pl, int splits) {
    return !pl.prompt && !pl.even && (splits == 2 || splits == 4 || splits == 8 || splits == 16);
}

// Clusters of s CTAs (1, 2, 4, 8 or 16) that the GPU holds at once with one CTA on an SM: a
// cluster lies within one group of SMs.  One more waits for a whole wave (one
// request of 2000 keys: 7.6 us for 15 clusters of 8 and 13.4 for 16; 9.1 for 36 of 4 and
// 16.0 for 37).
int places(int s) {
    return s == 1 ? sm_count() : s == 2 ? sm_count() / 2 : s == 4 ? sm_count() * 9 / 38 : s == 8 ? sm_count() / 10 : sm_count() / 20;
}

// Key ranges for num_splits = 0.
int choose_splits(const fa_paged_args& a, const Plan& pl) {
    const int64_t keys = static_cast<int64_t>(a.selected ? a.num_selected : a.max_pages) * a.cache.page_size;
    const int64_t sms = sm_count();
    if (pl.prompt) {
        // one CTA per SM; ranges only where the units fill less than half of
        // the SMs, each of at least four key tiles
        if (2 * pl.units > sms) return 1;
        return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({sms / pl.units, keys / 512, FA_PAGED_MAX_SPLITS})));
    }
    // One CTA of eight warps per SM where that fills three quarters of them, or
    // leaves a warp at most eight chunks (one request of 4096 keys, 8 heads: 8.6 us, 10.1
    // with CTAs of four warps; 16 of 2048: 16.4 and 20.7; 24 of 8000 and 4 heads, 96 of 152
    // SMs: 52 and 37).
    int s = 8;
    while (s > 1 && (pl.units > places(s) || keys < s * 256)) s /= 2;
    if (pl.units <= places(s) && (4 * s * pl.units >= 3 * sms || keys <= s * 2048)) return s;
    // Else one wave of about two CTAs per SM, in a count that a cluster can join;
    // each range of at least 256 keys.
    s = 1;
    const int resident = pl.width == 256 || pl.block_rows == 32 ? 2 : 3;
    while (s < pg::kDecMaxCluster && 2 * s * pl.units <= 2 * sms && pl.units <= resident * places(2 * s) && keys >= 2 * s * 256)
        s *= 2;
    // Few heads and a long context: more ranges than a cluster holds, through a
    // workspace (one request of 8 key heads and 65536 keys: 37 us with 32, 55 with 16).
    if (s == pg::kDecMaxCluster && s * pl.units < sms)
        while (s < FA_PAGED_MAX_SPLITS && 2 * s * pl.units <= 2 * sms && keys >= 2 * s * 1024) s *= 2;
    // Otherwise, as long as a range keeps 1024 keys, enough ranges for four waves of three
    // CTAs per SM: they even out unequal lengths (64 requests of 5000 to 16384 keys: 234 us
    // with 4, 251 with 2, 274 with 1) and partly filled waves.
    while (s < 8 && s * pl.units < 12 * sms && keys >= 2 * s * 1024) s *= 2;
    return s;
}

size_t part_bytes(int64_t rows, int splits, int d) {
    return (static_cast<size_t>(rows) * splits * d * 4 + 255) & ~static_cast<size_t>(255);
}

size_t workspace_bytes(const fa_paged_args& a, const Plan& pl, int splits) {
    if (pl.even) {
        const int64_t rows = 2ll * pl.even * pl.block_rows;
        return part_bytes(rows, 1, a.cache.d) + part_bytes(rows, 1, 1) + (static_cast<size_t>(pl.even) + 1) * 16;
    }
    if (splits < 2 || in_cluster(pl, splits)) return 0;
    const int64_t rows = static_cast<int64_t>(a.T) * a.Hq;
    return part_bytes(rows, splits, a.cache.d) + static_cast<size_t>(rows) * splits * 4;
}

struct KernelEntry {
    const void* fn;
    int smem;
};
template <int D, int R>
KernelEntry few_rows(bool even, int warps) {
    static_assert(pg::dec_smem<D, R, true, 4>() <= 232448 && pg::dec_smem<D, R, false, 8>() <= 232448, "shared memory of a CTA");
    if (even) return {reinterpret_cast<const void*>(&pg::paged_fwd_kernel<D, R, true, 4>), pg::dec_smem<D, R, true, 4>()};
    if (warps == 8) return {reinterpret_cast<const void*>(&pg::paged_fwd_kernel<D, R, false, 8>), pg::dec_smem<D, R, false, 8>()};
    return {reinterpret_cast<const void*>(&pg::paged_fwd_kernel<D, R, false, 4>), pg::dec_smem<D, R, false, 4>()};
}
KernelEntry select_kernel(int width, int rows, bool even, int warps) {
    if (width == 64)
        return rows == 8 ? few_rows<64, 8>(even, warps) : rows == 16 ? few_rows<64, 16>(even, warps) : few_rows<64, 32>(even, warps);
    if (width == 128)
        return rows == 8 ? few_rows<128, 8>(even, warps) : rows == 16 ? few_rows<128, 16>(even, warps) : few_rows<128, 32>(even, warps);
    return rows == 8 ? few_rows<256, 8>(even, warps) : few_rows<256, 16>(even, warps);
}
const void* select_even_join(int rows) {
    return rows == 8    ? reinterpret_cast<const void*>(&pg::paged_even_join_kernel<8>)
           : rows == 16 ? reinterpret_cast<const void*>(&pg::paged_even_join_kernel<16>)
                        : reinterpret_cast<const void*>(&pg::paged_even_join_kernel<32>);
}

template <int NL, bool BF16, bool ROT>
const void* append_kernel_of(bool bounds) {
    return bounds ? reinterpret_cast<const void*>(&pg::kv_append_kernel<NL, BF16, true, ROT>)
                  : reinterpret_cast<const void*>(&pg::kv_append_kernel<NL, BF16, false, ROT>);
}
template <bool ROT>
const void* append_kernel(int page_size, int d, bool bf16, bool bounds) {
    // rows of a whole page that a thread of the CTA would hold
    const int rows = pg::kAppendThreads / (d / 8);
    if ((page_size + rows - 1) / rows <= 4) return bf16 ? append_kernel_of<4, true, ROT>(bounds) : append_kernel_of<4, false, ROT>(bounds);
    return bf16 ? append_kernel_of<16, true, ROT>(bounds) : append_kernel_of<16, false, ROT>(bounds);
}

int check_args(const fa_paged_args& a) {
    // no query: nothing is read or written, and empty tensors have no address
    const bool none = a.T == 0;
    if (!none && (!a.q || !a.o || !a.lse)) return FA_ERR_INVALID_ARG;
    if (!(none && a.B == 0) && (!a.block_table || !a.lens)) return FA_ERR_INVALID_ARG;
    if (!none && (a.selected == nullptr) != (a.selected_count == nullptr)) return FA_ERR_INVALID_ARG;
    if (a.B < (none ? 0 : 1) || a.T < 0 || a.Hq < 1 || a.max_q < (none ? 0 : 1) || a.max_pages < 1) return FA_ERR_INVALID_ARG;
    if (a.dtype != FA_FP16 && a.dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(a.scale) || !(a.scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (a.num_splits < 0 || a.num_splits > FA_PAGED_MAX_SPLITS) return FA_ERR_INVALID_ARG;
    if (!a.cu_q && (a.T != a.B || (!none && a.max_q != 1))) return FA_ERR_INVALID_ARG;
    if (a.selected && (a.num_selected < 1 || (!none && a.max_q != 1))) return FA_ERR_INVALID_ARG;
    const int st = check_cache(a.cache);
    if (st != FA_OK) return st;
    if (a.Hq % a.cache.Hk != 0) return FA_ERR_INVALID_ARG;
    if (a.max_pages > kMostKeys / a.cache.page_size) return FA_ERR_INVALID_ARG;
    if (a.selected && a.num_selected > kMostKeys / a.cache.page_size) return FA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(a.max_q) * (a.Hq / a.cache.Hk) > INT32_MAX / 2) return FA_ERR_INVALID_ARG;
    if (bad_strides(a.q_stride) || bad_strides(a.o_stride)) return FA_ERR_MISALIGNED;
    if (misaligned(a.q, 16) || misaligned(a.o, 16) || misaligned(a.lse, 4) || misaligned(a.block_table, 4) ||
        misaligned(a.lens, 4) || misaligned(a.cu_q, 4) || misaligned(a.selected, 4) || misaligned(a.selected_count, 4))
        return FA_ERR_MISALIGNED;
    return FA_OK;
}

// Keys and values into their slots; with `rotary` the keys are turned first, and the queries beside them.
int append(const fa_kv_cache* cache, const void* k, const void* v, const int* slots, int T, const long long* k_stride,
           const long long* v_stride, const fa_rotary* rotary, const fa_rotary_part* q, int dtype, void* stream) {
    if (!cache || !k || !v || !slots || !k_stride || !v_stride || T < 0) return FA_ERR_INVALID_ARG;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    const int st = check_cache(*cache);
    if (st != FA_OK) return st;
    if (cache->Hk > 32767) return FA_ERR_UNSUPPORTED;
    if (T > kMostKeys) return FA_ERR_INVALID_ARG;
    if (bad_strides(k_stride) || bad_strides(v_stride) || misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 4))
        return FA_ERR_MISALIGNED;
    if (rotary) {
        int bad = check_rotary(rotary, cache->d, T);
        if (bad == FA_OK && q) bad = check_part(q, T);
        if (bad != FA_OK) return bad;
    }
    if (T == 0) return FA_OK;
    pg::AppendParams p = {};
    p.x[0] = static_cast<const uint16_t*>(k), p.x[1] = static_cast<const uint16_t*>(v);
    p.st[0] = k_stride[0], p.sh[0] = k_stride[1], p.st[1] = v_stride[0], p.sh[1] = v_stride[1];
    p.codes[0] = static_cast<uint8_t*>(cache->k), p.codes[1] = static_cast<uint8_t*>(cache->v);
    p.scale[0] = cache->k_scale, p.scale[1] = cache->v_scale;
    p.bounds = reinterpret_cast<int8_t*>(cache->k_bounds);
    p.slots = slots;
    p.T = T, p.Hk = cache->Hk, p.d = cache->d, p.num_pages = cache->num_pages, p.page_shift = shift_of(cache->page_size);
    // Slots a CTA looks through (64 down to 8, one per warp) and (head, K or V)
    // pairs it takes (4 or 1): the most that leaves four CTAs per SM.
    const int64_t sms = sm_count();
    auto ctas = [&] { return (static_cast<int64_t>(T) + p.chunk - 1) / p.chunk * ((2 * p.Hk + p.pairs - 1) / p.pairs); };
    p.chunk = pg::kAppendMaxChunk, p.pairs = 4;
    if (ctas() < 4 * sms) p.pairs = 1;
    while (p.chunk > 8 && ctas() < 4 * sms) p.chunk /= 2;
    const bool bf16 = dtype == FA_BF16;
    const int64_t columns = (static_cast<int64_t>(T) + p.chunk - 1) / p.chunk;
    p.pair_rows = (2 * p.Hk + p.pairs - 1) / p.pairs;
    int64_t rows = p.pair_rows;
    pg::RotaryWork queries = {};
    const void* fn = rotary ? append_kernel<true>(cache->page_size, p.d, bf16, p.bounds != nullptr)
                            : append_kernel<false>(cache->page_size, p.d, bf16, p.bounds != nullptr);
    if (rotary) {
        p.turn = rotary_table(*rotary);
        if (q) {
            p.q = rotary_work(*rotary, q, nullptr, T, p.d);
            p.q.groups = q->heads;
            const int64_t items = static_cast<int64_t>(T) * q->heads * (p.q.cols + p.q.tail);
            if (items > INT32_MAX) return FA_ERR_INVALID_ARG;
            if (items > 1024ll * sm_count()) {
                // Many: a launch of their own, at the occupancy that turning alone has (24.6 thousand tokens of 32 heads, d 128:
                // 61 us of it, behind this kernel's registers 180).  It comes last, so that a call that fails has turned no query in place.
                queries = p.q;
                p.q.T = 0;
            } else {  // an item per thread; the grid's rows end at 65535, what is beyond goes round
                rows = std::min<int64_t>(65535, rows + (items + columns * pg::kAppendThreads - 1) / (columns * pg::kAppendThreads));
            }
        }
    }
    void* args[] = {&p};
    if (!launch(fn, columns, static_cast<int>(rows), pg::kAppendThreads, 0, 1, stream, args)) return FA_ERR_CUDA;
    return queries.T > 0 ? launch_rotary(queries, bf16, stream) : FA_OK;
}

}  // namespace

// Read and clear the paged kernels' status word (the caller has synchronised).
__attribute__((visibility("hidden"))) bool fa_paged_take_status(unsigned int* out) {
    const unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(out, pg::g_paged_status, sizeof(*out)) != cudaSuccess) return false;
    return *out == 0 || cudaMemcpyToSymbol(pg::g_paged_status, &zero, sizeof(zero)) == cudaSuccess;
}

extern "C" {

int fa_kv_tables_step(const int* new_tokens, const int* lens, int* block_table, int* free_pages,
                      const int* free_count, int B, int max_pages, int free_capacity, int page_size,
                      int max_tokens, int* slots, int* cu_new, int* lens_out, int* free_count_out,
                      int* status, void* stream) {
    if (!new_tokens || !lens || !block_table || !free_pages || !free_count || !cu_new || !lens_out ||
        !free_count_out || !status || (!slots && max_tokens > 0))
        return FA_ERR_INVALID_ARG;
    const int shift = shift_of(page_size);
    if (B < 1 || max_pages < 1 || free_capacity < 1 || max_tokens < 0 || shift < 0) return FA_ERR_INVALID_ARG;
    if (lens_out == lens || free_count_out == free_count) return FA_ERR_INVALID_ARG;
    if (max_pages > kMostKeys / page_size) return FA_ERR_INVALID_ARG;
    if (B > pg::kTablesMaxB) return FA_ERR_UNSUPPORTED;
    for (const void* q : {static_cast<const void*>(new_tokens), static_cast<const void*>(lens),
                          static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_count), static_cast<const void*>(slots),
                          static_cast<const void*>(cu_new), static_cast<const void*>(lens_out),
                          static_cast<const void*>(free_count_out), static_cast<const void*>(status)})
        if (misaligned(q, 4)) return FA_ERR_MISALIGNED;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return FA_ERR_CUDA;
    const void* fn = reinterpret_cast<const void*>(&pg::kv_tables_kernel);
    const int smem = (3 * (B + 1) + (B <= pg::kTablesKeptLens ? B : 0)) * 4;
    if (!ensure_smem(fn, 3 * (pg::kTablesMaxB + 1) * 4, device)) return FA_ERR_CUDA;
    pg::TablesParams p{new_tokens, lens, block_table, free_pages, free_count, B, max_pages, free_capacity,
                       shift, max_tokens, slots, cu_new, lens_out, free_count_out, status};
    // a token (or a request) per thread, at most one CTA per SM: every CTA repeats the prefix sums
    const int64_t work = std::max<int64_t>(max_tokens, B);
    const int64_t ctas = std::min<int64_t>((work + pg::kTablesThreads - 1) / pg::kTablesThreads, sm_count());
    void* args[] = {&p};
    if (!launch(fn, std::max<int64_t>(1, ctas), 1, pg::kTablesThreads, smem, 1, stream, args)) return FA_ERR_CUDA;
    return FA_OK;
}

int fa_kv_cache_append(const fa_kv_cache* cache, const void* k, const void* v, const int* slots, int T,
                       const long long* k_stride, const long long* v_stride, int dtype, void* stream) {
    return append(cache, k, v, slots, T, k_stride, v_stride, nullptr, nullptr, dtype, stream);
}

int fa_kv_cache_append_rotary(const fa_kv_cache* cache, const void* k, const void* v, const int* slots, int T,
                              const long long* k_stride, const long long* v_stride, const fa_rotary* rotary,
                              const fa_rotary_part* q, int dtype, void* stream) {
    if (!rotary || rotary->inverse) return FA_ERR_INVALID_ARG;
    return append(cache, k, v, slots, T, k_stride, v_stride, rotary, q, dtype, stream);
}

int fa_paged_num_splits(const fa_paged_args* a) {
    if (!a || check_args(*a) != FA_OK || a->T == 0) return 1;
    const Plan pl = plan_of(*a);
    return pl.even ? 0 : choose_splits(*a, pl);
}

size_t fa_paged_workspace_size(const fa_paged_args* a) {
    if (!a || check_args(*a) != FA_OK || a->T == 0) return 0;
    const Plan pl = plan_of(*a);
    return workspace_bytes(*a, pl, a->num_splits == 0 ? choose_splits(*a, pl) : a->num_splits);
}

int fa_paged_fwd(const fa_paged_args* args) {
    if (!args) return FA_ERR_INVALID_ARG;
    const fa_paged_args& a = *args;
    const int st = check_args(a);
    if (st != FA_OK) return st;
    if (a.T == 0) return FA_OK;
    const Plan pl = plan_of(a);
    const int splits = pl.even ? 1 : a.num_splits == 0 ? choose_splits(a, pl) : a.num_splits;
    const size_t need = workspace_bytes(a, pl, splits);
    if (need > 0) {
        if (!a.workspace) return FA_ERR_INVALID_ARG;
        if (misaligned(a.workspace, 256)) return FA_ERR_MISALIGNED;
        if (a.workspace_bytes < need) return FA_ERR_INVALID_ARG;
    }
    // Tokens far below B * max_q: prompts beside requests of a few tokens.  Those with no
    // more rows than a block of the few-row kernel for one token holds are served by it, in a launch
    // of their own, and the tcgen05 kernel starts a CTA for the others' blocks only (one prompt of
    // 2000 tokens among 200 requests of 4000 keys, 32 / 8 heads, d 128: 413 us; 884 with
    // a CTA for every block there could be, 1132 with the tcgen05 kernel alone).
    const int few = block_rows_of(pl.width, a.Hq / a.cache.Hk);
    const bool mixed = pl.prompt && a.B > 1 && a.num_splits == 0 && splits == 1 && a.Hq / a.cache.Hk <= few &&
                       2ll * a.T <= static_cast<int64_t>(a.B) * a.max_q;
    int64_t units = pl.even ? pl.even : pl.units * splits;
    if (mixed) {  // (the blocks of all requests with more than `few` rows are no more than this)
        const int64_t packed = static_cast<int64_t>(a.T) * (a.Hq / a.cache.Hk);
        units = a.cache.Hk * std::min<int64_t>(units / a.cache.Hk, packed / pl.block_rows + std::min<int64_t>(a.B, packed / (few + 1)));
    }
    const int64_t rows = static_cast<int64_t>(a.T) * a.Hq;
    if (units > INT32_MAX || rows > INT32_MAX) return FA_ERR_INVALID_ARG;

    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return FA_ERR_CUDA;
    const int keys = pl.width == 256 ? 16 : 32;
    const int box_rows = std::min(a.cache.page_size, keys), box_cols = std::min(pl.width, 128);
    const int64_t cache_rows = static_cast<int64_t>(a.cache.num_pages) * a.cache.Hk * a.cache.page_size;
    CUtensorMap tk, tv;
    if ((!pl.prompt || mixed) && (!encode_codes(&tk, a.cache.k, cache_rows, a.cache.d, box_cols, box_rows) ||
                                  !encode_codes(&tv, a.cache.v, cache_rows, a.cache.d, box_cols, box_rows)))
        return FA_ERR_CUDA;

    pg::PagedParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.o = static_cast<uint16_t*>(a.o);
    p.lse = a.lse;
    p.cu_q = a.cu_q, p.table = a.block_table, p.lens = a.lens;
    p.sel = a.selected, p.sel_count = a.selected_count;
    p.k_scale = a.cache.k_scale, p.v_scale = a.cache.v_scale;
    p.q_st = a.q_stride[0], p.q_sh = a.q_stride[1], p.o_st = a.o_stride[0], p.o_sh = a.o_stride[1];
    p.T = a.T, p.B = a.B, p.Hq = a.Hq, p.Hk = a.cache.Hk, p.G = a.Hq / a.cache.Hk, p.d = a.cache.d;
    p.max_q = a.max_q, p.max_pages = a.max_pages, p.num_sel = a.num_selected;
    p.num_pages = a.cache.num_pages, p.page_shift = shift_of(a.cache.page_size);
    p.in_cluster = in_cluster(pl, splits);
    p.row_blocks = pl.row_blocks, p.splits = splits, p.box_rows = box_rows, p.causal = a.causal != 0;
    p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    const int64_t part_rows = pl.even ? 2ll * pl.even * pl.block_rows : rows * splits;
    char* ws = static_cast<char*>(a.workspace);
    const size_t o_bytes = part_bytes(part_rows, 1, a.cache.d);
    p.o_part = need > 0 ? reinterpret_cast<float*>(ws) : nullptr;
    p.lse_part = need > 0 ? reinterpret_cast<float*>(ws + o_bytes) : nullptr;
    p.shares = pl.even ? reinterpret_cast<int4*>(ws + o_bytes + part_bytes(part_rows, 1, 1)) : nullptr;
    p.rows_from = mixed ? few + 1 : 0, p.rows_to = INT32_MAX, p.packed = mixed;
    bool bf16 = a.dtype == FA_BF16;
    auto launch_few = [&](const Plan& pl, int splits, int64_t units) {
        // eight warps where one CTA per SM is all there is (not for clusters of 16: 13.7
        // us against 10.1 for one request of 4096 keys and 8 heads)
        const bool one_each = in_cluster(pl, splits) ? pl.units <= places(splits) : units <= sm_count();
        const int warps = !pl.even && one_each && splits != pg::kDecMaxCluster ? 8 : 4;
        const KernelEntry ke = select_kernel(pl.width, pl.block_rows, pl.even != 0, warps);
        void* kargs[] = {&tk, &tv, &p, &bf16};
        return ensure_smem(ke.fn, ke.smem, device) &&
               launch(ke.fn, units, 1, 32 * warps, ke.smem, p.in_cluster ? splits : 1, a.stream, kargs);
    };
    if (pl.prompt && units > 0) {
        const uint8_t *kc = static_cast<const uint8_t*>(a.cache.k), *vc = static_cast<const uint8_t*>(a.cache.v);
        const void* fn = pl.width == 64    ? reinterpret_cast<const void*>(&pg::paged_prompt_kernel<64>)
                         : pl.width == 128 ? reinterpret_cast<const void*>(&pg::paged_prompt_kernel<128>)
                                           : reinterpret_cast<const void*>(&pg::paged_prompt_wide_kernel);
        const int smem = pl.width == 64 ? pg::PrCfg<64>::kSmem : pl.width == 128 ? pg::PrCfg<128>::kSmem : pg::kPwSmem;
        const int threads = pl.width == 256 ? pg::kPwThreads : pg::kPrThreads;
        void* kargs[] = {&kc, &vc, &p, &bf16};
        if (!ensure_smem(fn, smem, device) || !launch(fn, units, 1, threads, smem, 1, a.stream, kargs)) return FA_ERR_CUDA;
    } else if (!pl.prompt && !launch_few(pl, splits, units)) {
        return FA_ERR_CUDA;
    }
    if (mixed) {
        const Plan one = single_token_plan(a, pl.width, few);
        const int ranges = std::min(choose_splits(a, one), pg::kDecMaxCluster);  // (joined without a workspace)
        p.rows_from = 0, p.rows_to = few, p.row_blocks = 1, p.splits = ranges, p.in_cluster = in_cluster(one, ranges);
        if (!launch_few(one, ranges, one.units * ranges)) return FA_ERR_CUDA;
    }
    if (pl.even) {
        void* margs[] = {&p, &bf16};
        if (!launch(select_even_join(pl.block_rows), pl.even - 1, 1, pg::kJoinThreads, 0, 1, a.stream, margs)) return FA_ERR_CUDA;
    } else if (need > 0) {
        void* margs[] = {&p, &bf16};
        if (!launch(reinterpret_cast<const void*>(&pg::paged_merge_kernel), (rows + pg::kMergeWarps - 1) / pg::kMergeWarps, 1,
                    32 * pg::kMergeWarps, 0, 1, a.stream, margs))
            return FA_ERR_CUDA;
    }
    return FA_OK;
}

int fa_kv_page_select(const fa_kv_cache* cache, const void* q, const long long* q_stride, const int* block_table,
                      const int* lens, int B, int Hq, int max_pages, int num_selected, int dtype, int* selected,
                      int* selected_count, void* stream) {
    if (!cache || !cache->k_scale || !cache->k_bounds || !q || !q_stride || !block_table || !lens || !selected ||
        !selected_count)
        return FA_ERR_INVALID_ARG;
    if (B < 1 || Hq < 1 || max_pages < 1 || num_selected < 1) return FA_ERR_INVALID_ARG;
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    const int st = check_sizes(*cache);
    if (st != FA_OK) return st;
    if (Hq % cache->Hk != 0 || max_pages > kMostKeys / cache->page_size ||
        static_cast<int64_t>(B) * cache->Hk > INT32_MAX)
        return FA_ERR_INVALID_ARG;
    if (max_pages > pg::kSelectMaxPages) return FA_ERR_UNSUPPORTED;
    if (bad_strides(q_stride) || misaligned(q, 16) || misaligned(cache->k_bounds, 16) || misaligned(cache->k_scale, 4) ||
        misaligned(block_table, 4) || misaligned(lens, 4) || misaligned(selected, 4) || misaligned(selected_count, 4))
        return FA_ERR_MISALIGNED;
    pg::SelectParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.q_st = q_stride[0], p.q_sh = q_stride[1];
    p.bounds = reinterpret_cast<const int8_t*>(cache->k_bounds);
    p.k_scale = cache->k_scale;
    p.table = block_table, p.lens = lens;
    p.Hk = cache->Hk, p.G = Hq / cache->Hk, p.d = cache->d, p.num_pages = cache->num_pages;
    p.page_shift = shift_of(cache->page_size), p.max_pages = max_pages, p.keep = num_selected;
    p.selected = selected, p.count = selected_count;
    const int64_t smem = 4ll * (2ll * p.G * (p.d / 4) + p.G + max_pages) + 16;
    if (smem > 200 * 1024) return FA_ERR_UNSUPPORTED;  // a group of very many query heads
    const void* fn = dtype == FA_BF16 ? reinterpret_cast<const void*>(&pg::kv_page_select_kernel<true>)
                                      : reinterpret_cast<const void*>(&pg::kv_page_select_kernel<false>);
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || !ensure_smem(fn, 200 * 1024, device)) return FA_ERR_CUDA;
    // 128 pages per CTA, what its groups of lanes have on their way at once, unless
    // the CTAs would not fit the GPU together (four per SM)
    p.cluster = 1;
    while (p.cluster < pg::kSelectMaxCluster && p.cluster * 128 < max_pages &&
           2ll * p.cluster * B * p.Hk <= 4ll * sm_count())
        p.cluster *= 2;
    const int64_t ctas = static_cast<int64_t>(B) * p.Hk * p.cluster;
    if (ctas > INT32_MAX) return FA_ERR_INVALID_ARG;
    void* args[] = {&p};
    if (!launch(fn, ctas, 1, pg::kSelectThreads, static_cast<int>(smem), p.cluster, stream, args)) return FA_ERR_CUDA;
    return FA_OK;
}

}  // extern "C"
