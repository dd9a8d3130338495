// latent_paged_kernel.cuh - latent attention in its absorbed form over a paged latent cache.
//
// Every head of a request reads the same keys, rows of W = C + R channels, and the values are the
// first C channels of the same rows:
//   O = softmax(scale q c^T) c[:, :C],   W <= 576, C <= 512.
// A key brings 2 W bytes and 2 (W + C) operations per head: with 128 heads and one token 241 per byte,
// below the 286 at which the tensor cores and HBM take the same time, so HBM bounds decoding as
// long as each key is read from it once, enters both products from shared memory, and the tensor cores run at their full rate.
//
// Mapping.  Packed rows r = i H + g (query i, head g) of a request; a unit is 128 of them over some tiles of 128 keys,
// and a pair of CTAs (a cluster, one CTA per SM) works on it with tcgen05.mma of both (cta_group::2, M = 128):
// each CTA holds 64 rows of queries, weights and U, and one half of every B operand.  64 x 512 fp32 of U
// take 256 columns of tensor memory (lanes 0-63 hold the first half of a product's columns, lanes 64-127 the other), which
// leaves room for two tiles of scores; 128 rows in one CTA would leave none.  (One CTA per 64 rows with M = 64 runs the
// tensor core at half this rate and reads every key twice for 128 heads.)
//   S = Q K^T, N = 128 keys: CTA r loads keys 64 r .. 64 r + 63 of the tile, all channels.
//   U += P V, N = 256 channels twice: CTA r brings channels 128 r .. of each 256, of all 128 keys.  Half of that it has
//     loaded as keys.  The other half, the peer's keys, is loaded once S is done into the places of its own
//     keys' other channels, which nothing needs any more: slots 4 b + 2 h and 4 b + 2 h + 1 of both CTAs hold the CTA's
//     channels of block b for the tile's half h.
// So two stages of a tile fit beside the queries: 72 KB of queries, 2 x 64 KB of latents, 8 KB of channels from 512 on (one
// stage: they are read by S alone), 16 KB through which warps exchange weights.
// Roles:
//   * warps 0-3: softmax and epilogue.  Warp w has rows 32 (w & 1) .. and keys 64 (w >> 1) .. of a tile;
//     the two warps of a row exchange its maximum and their weights through shared memory;
//   * warp 4: TMA of the CTA's keys, pages looked up three tiles ahead, in two halves of four pieces with barriers of
//     their own: S begins with the first half while the second is on its way, and U += P V frees them one by one;
//   * warps 5 and 9 (of the first CTA): tcgen05.mma, S and U += P V, each as its operands are ready (one warp for both left the
//     tensor cores waiting for the instructions between a barrier and the next product);
//   * warp 6: TMA of the peer's keys as values, half by half behind S, and of channels from 512 on;
//   * warps 7-8: queries, for the next unit as soon as the last S of this one is done: TMA boxes of gcd(H, 64) heads, or
//     where these are below eight cp.async.
// TMEM: U 0-255, S 256-319 and 320-383, weights 384-447 and 448-511.
//
// Weights are 2^(x - ref + 7) in the operands' 16-bit type; ref is the row's maximum when it last moved, and moves only
// where the maximum has grown by more than 2^8 (fp16 holds 2^15), with U rescaled then.  O is divided by the sum of
// the rounded weights, the LSE takes the sum of the fp32 ones.
//
// Sharing out.  All (request, 128 rows, tile) of a call, in that order, are dealt out in equal shares to as many
// pairs as run at once, whatever the lengths.  Parts of a unit go through a workspace and are joined by a second launch.
//
// What bounds it.  A tile passes through load (1.1 us), S (1.3, with the other stage's U += P V between its halves), softmax
// (0.8) and U += P V (0.5 and the signals), and two are under way: 1.9 us a tile, where HBM would take 1.7
// and the tensor cores work 1.15.  64 requests of 5000 to 16384 keys, 128 heads, in a graph: 166 us, 4.9 TB/s and 1.15 PFLOP/s (16 heads: 158), from a
// cold L2 177 us, 4.5 TB/s;
// 8 us of it pass before the first product, 12 in the join.  One request of 4096 keys, 32 heads: 13.4 us, latency: lengths,
// queries and keys, two tiles, parts, the join's start and its reads.
// Tried (against 178, before what prefetch() says): tiles of 64 keys in four stages 186 us (loads of 4 KB: TMA brings an SM 36 bytes a cycle so, 47 in 8 KB, 55 in 32 KB,
// and a tile needs its keys twice); eight softmax warps 191; a second warp for each kind of load 185; table entries 32 at a time 182.
#pragma once

#include "pair_ptx.cuh"

namespace fa {
namespace paged {

constexpr int kLatRows = 128, kLatKeys = 128; // of a unit and a tile; half of each per CTA
constexpr int kLatThreads = 320;
constexpr int kLatPieces = 9;                 // 64-channel pieces of a row: W <= 576
constexpr int kLatPiece = 64 * 128;           // 64 rows x 64 16-bit channels, 128-byte swizzle
constexpr int kLatStages = 2, kLatSlots = 8;  // pieces of a stage
constexpr int kLatOffK = kLatPieces * kLatPiece;
constexpr int kLatOffTail = kLatOffK + kLatStages * kLatSlots * kLatPiece;  // the ninth piece
constexpr int kLatOffP = kLatOffTail + kLatPiece;
constexpr int kLatOffCtl = kLatOffP + 2 * kLatPiece;
constexpr int kLatMaxB = 16384;
constexpr float kLatShift = 7.f, kLatLag = 8.f;

struct LatentParams {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    const int* cu_q;
    const int* table;
    const int* lens;
    const uint16_t* cache;
    long long q_st, q_sh, o_st, o_sh;
    int T, B, H, C, W, max_q, max_pages, num_pages, page_shift;
    int min_share;    // tiles
    int q_box;        // heads of a box of queries (0: read by cp.async)
    int box_rows;
    int box_pieces;   // of a load of keys: 4 or 1
    int causal;
    float scale_log2;
    float4* o_part;   // the parts of a share's first and last unit: [2 pairs][CTA][warp][32 channels][quad][lane], as lat_part says
    float2* stats;    // [2 pairs][128]: log2 of the sums of the fp32 and of the rounded weights
    int4* shares;     // [pairs][2]: the first unit's begin, end and row block, and the share; its request's first row and rows
};

// Rows and keys of request b, and its units: blocks of 128 rows times tiles of keys (at least one).
struct LatRequest {
    int q0, nq, len, blocks, tiles;
};
// 32-channel pieces of U that a softmax warp holds: columns of tensor memory over 32.
__host__ __device__ constexpr int lat_chunks(int C) { return C <= 128 ? 2 : C <= 256 ? 4 : C <= 384 ? 6 : 8; }
// A part in the workspace: a warp's quads of channels lie as its lanes hold them, so that they are written and read 512 bytes at
// a time.
__host__ __device__ constexpr long long lat_part(long long part, int rank, int warp, int chunk, int C) {
    return (((part * 2 + rank) * 4 + warp) * lat_chunks(C) + chunk) * 8 * 32;
}
// Output channel of column 32 `chunk` of a warp with key half (here: channel half) `half`.
__host__ __device__ constexpr int lat_channel(int chunk, int half, int C) {
    const int block = chunk >> 2, wide = C - 256 * block > 128 ? 128 : 64;
    return 256 * block + half * wide + 32 * (chunk & 3);
}

struct LatCtl {
    // signalled in the first CTA by both: queries, keys, values, weights, U read; in both by the tensor core; by a CTA's own loads.
    // k: by stage and half of its pieces; k_empty of the second half says that U += P V of the tile is done
    uint64_t q_full, k_full[4], v_full[2], p_full[2], o_empty;
    uint64_t q_empty, k_empty[4], s_half[2], s_full[2], drain[2];
    uint64_t v_last[2];          // values of a tile with keys that were not loaded
    uint32_t tmem_base;
    int start[3];                // request, row block, tile of the share's first unit
    LatRequest first;            // that request
    float top[2][2][64];         // by tile parity, key half, row
};
static_assert(kLatOffCtl + sizeof(LatCtl) + 1024 <= 232448, "shared memory of a CTA");
constexpr int kLatSmem = kLatOffCtl + static_cast<int>(sizeof(LatCtl)) + 1024;

__device__ __forceinline__ uint64_t lat_desc(uint32_t saddr, uint32_t lbo) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint32_t lat_instr(bool bf16, int n, bool b_mn_major) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           ((static_cast<uint32_t>(n) >> 3) << 17) | ((128u >> 4) << 24);
}
// A line on its way to L2, whoever writes it meanwhile.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Device data that cannot be leaves a request without rows or keys.
__device__ __forceinline__ LatRequest lat_request(const LatentParams& p, int b, bool& bad) {
    LatRequest r;
    r.q0 = b, r.nq = 1;
    if (p.cu_q) {
        r.q0 = ld_meta(p.cu_q + b);
        r.nq = ld_meta(p.cu_q + b + 1) - r.q0;
        if (r.q0 < 0 || r.nq < 0 || r.nq > p.max_q || r.q0 > p.T - r.nq) bad = true, r.nq = 0;
    }
    r.len = ld_meta(p.lens + b);
    if (r.len < 0 || r.len > (p.max_pages << p.page_shift)) bad = true, r.len = 0;
    r.blocks = (r.nq * p.H + kLatRows - 1) / kLatRows;
    r.tiles = max(1, (r.len + kLatKeys - 1) / kLatKeys);
    return r;
}

// Walks the parts of a pair's share: for every unit some tiles of its keys.
struct LatWalk {
    const LatentParams& p;
    const int f0, f1;
    int f, b, block, first;
    LatRequest rq;
    // of the current part
    int r0, rows, lo, hi, load_end;   // first row, rows; tiles [lo, hi); keys that are loaded (whole boxes up to the last seen)
    bool whole, at_start;

    __device__ LatWalk(const LatentParams& p_, const LatCtl* ctl, int f0_, int f1_)
        : p(p_), f0(f0_), f1(f1_), f(f0_), b(ctl->start[0]), block(ctl->start[1]), first(ctl->start[2]), rq(ctl->first) {}
    __device__ int limit(int r) const { return p.causal ? min(rq.len, rq.len - rq.nq + r / p.H + 1) : rq.len; }
    // the next part; false behind the last
    __device__ bool next() {
        if (f >= f1) return false;
        while (block >= rq.blocks) {  // (units are left, so there is a request that has some)
            if (b + 1 >= p.B) return false;
            bool bad = false;
            ++b, block = 0;
            rq = lat_request(p, b, bad);
        }
        const int n = min(rq.tiles - first, f1 - f);
        r0 = block * kLatRows;
        rows = min(kLatRows, rq.nq * p.H - r0);
        const int kend = max(0, limit(r0 + rows - 1)), kt = (kend + kLatKeys - 1) / kLatKeys;
        load_end = min(rq.len, (kend + p.box_rows - 1) & -p.box_rows);
        lo = min(first, kt), hi = min(first + n, kt);
        whole = first == 0 && n == rq.tiles;
        at_start = f == f0;
        f += n;
        first = 0;
        ++block;
        return true;
    }
};

// The pages of one half of the tiles of a part, looked up three tiles ahead: lane i has box i of the half.
struct LatPages {
    const LatentParams& p;
    const LatWalk& w;
    const int* trow;
    const int half;
    int page, page1, page2;
    __device__ LatPages(const LatentParams& p_, const LatWalk& w_, int half_, int lane) : p(p_), w(w_), half(half_) {
        trow = p.table + static_cast<long long>(w.b) * p.max_pages;
        page = at(w.lo, lane), page1 = at(w.lo + 1, lane), page2 = at(w.lo + 2, lane);
    }
    __device__ int key(int j, int lane) const { return j * kLatKeys + half * 64 + lane * p.box_rows; }
    __device__ bool wanted(int j, int lane) const { return j < w.hi && lane * p.box_rows < 64 && key(j, lane) < w.load_end; }
    // bytes of a piece of tile j that both halves load
    __device__ int both(int j) const { return min(kLatKeys, (w.load_end - j * kLatKeys + p.box_rows - 1) & -p.box_rows) * 128; }
    __device__ int at(int j, int lane) const { return wanted(j, lane) ? ld_meta(trow + (key(j, lane) >> p.page_shift)) : -1; }
    // Has the boxes of tile j brought to L2 (a page's rows lie together) while the tile's place in shared memory is still
    // taken.  A tile earlier it costs more than it brings, as tiles that are waited for queue behind it (64 requests, 128 heads: 165 us;
    // one tile ahead 167, two 177, three 193, nothing 200).  By lines where a half is one box, else a box a lane (ragged batch
    // 165 and 167 us; 64 requests in pages of 16 114 and 106).
    __device__ void prefetch(int j, int lane) const {
        const uint16_t* from = p.cache + ((static_cast<long long>(page) << p.page_shift) + (key(j, lane) & ((1 << p.page_shift) - 1))) * p.W;
        const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
        if (p.box_rows < 64) {
            if (there) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(p.box_rows * p.W * 2) : "memory");
        } else if (__shfl_sync(0xffffffffu, there, 0)) {
            const char* at = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<long long>(from), 0));
            for (int i = lane * 128; i < 64 * p.W * 2; i += 32 * 128) prefetch_l2(at + i);
        }
    }
    // First row of the lane's box of tile j in the cache, one before the cache (where TMA reads zeros) if the table names no page
    // of it; moves on to tile j + 1.
    __device__ int take(int j, int lane) {
        const int ahead = at(j + 3, lane);
        const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
        if (wanted(j, lane) && !there) report(kBadData);
        const int row = there ? (page << p.page_shift) + (key(j, lane) & ((1 << p.page_shift) - 1)) : -p.box_rows;
        page = page1, page1 = page2, page2 = ahead;
        return row;
    }
};

template <bool BF16>
__global__ void __launch_bounds__(kLatThreads, 1)
    latent_paged_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q, const LatentParams p) {
    extern __shared__ __align__(16) uint8_t lat_raw[];
    const uint32_t raw = ptx::smem_addr(lat_raw);
    uint8_t* smem = lat_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = ptx::smem_addr(smem);
    LatCtl* ctl = reinterpret_cast<LatCtl*>(smem + kLatOffCtl);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_rank());
    const int kp = (p.W + 63) >> 6;
    const bool tail = kp > kLatSlots;

    const uint32_t b_qf = ptx::smem_addr(&ctl->q_full), b_qe = ptx::smem_addr(&ctl->q_empty);
    const uint32_t b_kf = ptx::smem_addr(&ctl->k_full[0]), b_ke = ptx::smem_addr(&ctl->k_empty[0]);
    const uint32_t b_sh = ptx::smem_addr(&ctl->s_half[0]), b_sf = ptx::smem_addr(&ctl->s_full[0]), b_vf = ptx::smem_addr(&ctl->v_full[0]);
    const uint32_t b_pf = ptx::smem_addr(&ctl->p_full[0]), b_pv = ptx::smem_addr(&ctl->k_empty[1]), b_vl = ptx::smem_addr(&ctl->v_last[0]), b_oe = ptx::smem_addr(&ctl->o_empty);
    const uint32_t b_drain = ptx::smem_addr(&ctl->drain[0]);
    if (tid == 0) {
        ptx::mbar_init(b_qf, 2 * (p.q_box ? 1 : 64));
        ptx::mbar_init(b_qe, 1);
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(b_kf + 16 * s, 1);  // (the first CTA's expectation covers both CTAs' loads)
            ptx::mbar_init(b_kf + 16 * s + 8, 1);
            ptx::mbar_init(b_ke + 16 * s, 1);
            ptx::mbar_init(b_ke + 16 * s + 8, 1);
            ptx::mbar_init(b_sh + 8 * s, 1);
            ptx::mbar_init(b_sf + 8 * s, 1);
            ptx::mbar_init(b_vl + 8 * s, 1);
            ptx::mbar_init(b_pf + 8 * s, 2 * 4);  // (a warp may be a tile ahead of another)
            ptx::mbar_init(b_vf + 8 * s, 1);
        }
        ptx::mbar_init(b_oe, 2 * 4);
        ptx::mbar_init(b_drain, 1);
        ptx::mbar_init(b_drain + 8, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tm);
        if (p.box_pieces > 1) ptx::prefetch_tensormap(&tm_k);
        if (p.q_box) ptx::prefetch_tensormap(&tm_q);
    }
    if (warp == 5) {
        tmem_alloc_pair(ptx::smem_addr(&ctl->tmem_base));
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // barriers and tensor memory of both CTAs are there
    ptx::tc_fence_after_sync();
    dependents_may_start();
    // lengths and the table on their way to L2, as far as a line per thread goes
    {
        const long long i = (static_cast<long long>(blockIdx.x) * kLatThreads + tid) * 32;
        if (i < p.B) prefetch_l2(p.lens + i);
        if (p.cu_q && i <= p.B) prefetch_l2(p.cu_q + i);
        if (i < static_cast<long long>(p.B) * p.max_pages) prefetch_l2(p.table + i);
    }
    wait_for_previous();

    // ---- this pair's share [f0, f1) of all tiles, in order of request, row block, tile
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    int f0, f1;
    {
        int* before = reinterpret_cast<int*>(smem);  // (the queries' memory)
        const int per = (p.B + kLatThreads - 1) / kLatThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
        bool bad = false;
        int own = 0;
        LatRequest r = {};
        for (int b = b0; b < b1; ++b) {
            r = lat_request(p, b, bad);
            own += r.blocks * r.tiles;
        }
        if (bad) report(kBadData);
        int incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) before[warp] = incl;
        __syncthreads();
        int run = incl - own, all = 0;
#pragma unroll
        for (int w = 0; w < kLatThreads / 32; ++w) {
            if (w < warp) run += before[w];
            all += before[w];
        }
        const int share = max((all + pairs - 1) / pairs, p.min_share);
        f0 = static_cast<int>(min(static_cast<long long>(pair) * share, static_cast<long long>(all)));
        f1 = static_cast<int>(min(static_cast<long long>(f0) + share, static_cast<long long>(all)));
        if (f0 < f1 && run <= f0 && f0 < run + own) {
            for (int b = b0; b < b1; ++b) {
                if (per > 1) r = lat_request(p, b, bad);
                const int n = r.blocks * r.tiles;
                if (f0 < run + n) {
                    const int rel = f0 - run;
                    ctl->start[0] = b, ctl->start[1] = rel / r.tiles, ctl->start[2] = rel % r.tiles, ctl->first = r;
                    break;
                }
                run += n;
            }
        }
        ptx::fence_proxy_async_smem();  // (what was read and written here is the queries' memory)
        __syncthreads();
        if (p.shares && rank == 0 && tid == 0) {
            const int begin = f0 - (f0 < f1 ? ctl->start[2] : 0);
            p.shares[2 * pair] = make_int4(begin, f0 < f1 ? begin + ctl->first.tiles : begin, ctl->start[1], share);
            p.shares[2 * pair + 1] = make_int4(ctl->first.q0, ctl->first.nq, 0, 0);
        }
    }
    const uint32_t tmem = ctl->tmem_base;
    LatWalk walk(p, ctl, f0, f1);

    if (warp < 4) {
        // ================================================ softmax and epilogue
        const int half = warp >> 1, row = (warp & 1) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        // the warp's 32 rows x 128 bytes of exchange memory, and those of the warp with the same rows
        const uint32_t box = sbase + kLatOffP + warp * 4096, own = box + lane * 128, other = sbase + kLatOffP + (warp ^ 2) * 4096 + lane * 128;
        const uint32_t r_pf = in_first_cta(b_pf), r_oe = in_first_cta(b_oe);
        const int pair_barrier = 1 + (warp & 1);
        int c = 0, last_phase = 0;  // tiles so far; phases of v_last
        bool ok = true;  // (after a wait that ran out nothing is waited for, but every barrier of the two warps is still met)
        while (walk.next()) {
            const int r = walk.r0 + rank * 64 + row;
            const bool mine = rank * 64 + row < walk.rows;
            const int my_limit = mine ? walk.limit(r) : walk.rq.len;
            const int first_limit = walk.limit(walk.r0);  // the least of the unit's rows
            float ref = -INFINITY, sum = 0.f, rsum = 0.f;  // sums of this thread's keys: fp32 and rounded weights
            for (int j = walk.lo; j < walk.hi; ++j, ++c) {
                ok = ok && wait_warp(b_sf + 8 * (c & 1), (c >> 1) & 1);
                ptx::tc_fence_after_sync();
                const int key0 = j * kLatKeys;
                uint32_t sv[64];
                ptx::tmem_ld_32x32b_x64(tmem + lane_off + 256 + 64 * (c & 1), sv);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 64; ++e) ptx::reg_fence(sv[e]);
                if (key0 + kLatKeys > first_limit) {
                    const int seen = my_limit - key0 - 64 * half;
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (e >= seen) sv[e] = __float_as_uint(-INFINITY);
                }
                float top = __uint_as_float(sv[0]), top2 = __uint_as_float(sv[1]);
#pragma unroll
                for (int e = 2; e + 3 < 64; e += 4) {
                    top = ptx::fmax3(top, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                    top2 = ptx::fmax3(top2, __uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3]));
                }
                top = ptx::fmax3(fmaxf(top, top2), __uint_as_float(sv[62]), __uint_as_float(sv[63]));
                ctl->top[c & 1][half][row] = top;
                ptx::named_barrier_sync(pair_barrier, 64);
                top = fmaxf(top, ctl->top[c & 1][half ^ 1][row]) * p.scale_log2;
                const bool moves = top > ref + kLatLag;  // (the same in both warps of the row)
                if (__any_sync(0xffffffffu, moves)) {
                    // U holds the products of the tiles before
                    if (c > 0) ok = ok && wait_warp(b_pv + 16 * ((c - 1) & 1), ((c - 1) >> 1) & 1);
                    ptx::tc_fence_after_sync();
                    float alpha = 1.f;
                    if (moves) {
                        if (ref != -INFINITY) alpha = ptx::ex2_approx(ref - top);
                        ref = top;
                    }
                    sum *= alpha, rsum *= alpha;
                    if (j > walk.lo) {
                        const float2 av = make_float2(alpha, alpha);
                        const int cols = p.C <= 128 ? 64 : p.C <= 256 ? 128 : p.C <= 384 ? 192 : 256;
#pragma unroll 1
                        for (int x = 0; x < cols; x += 32) {
                            uint32_t ov[32];
                            ptx::tmem_ld_32x32b_x32(tmem + lane_off + x, ov);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                ptx::reg_fence(ov[e]);
                                ptx::reg_fence(ov[e + 1]);
                                const float2 y = __fmul2_rn(make_float2(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])), av);
                                ov[e] = __float_as_uint(y.x), ov[e + 1] = __float_as_uint(y.y);
                            }
                            ptx::tmem_st_32x32b_x32(tmem + lane_off + x, ov);
                        }
                        ptx::tmem_wait_st();
                    }
                }
                const float sub = (ref == -INFINITY ? 0.f : ref) - kLatShift;
                const float2 fv = make_float2(p.scale_log2, p.scale_log2), nv = make_float2(-sub, -sub);
                float2 acc = make_float2(0.f, 0.f), racc = make_float2(0.f, 0.f);
                uint32_t pk[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
#pragma unroll
                    for (int e = 4 * i; e < 4 * i + 4; ++e) {
                        const float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), fv, nv);
                        const float2 w = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
                        acc = __fadd2_rn(acc, w);
                        pk[e] = pack16(w.x, w.y, BF16);
                        racc = __fadd2_rn(racc, unpack16(pk[e], BF16));
                    }
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(own + ((i ^ (lane & 7)) << 4)), "r"(pk[4 * i]), "r"(pk[4 * i + 1]),
                                 "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3])
                                 : "memory");
                }
                sum += acc.x + acc.y, rsum += racc.x + racc.y;
                // Both lanes of a row take the weights of all its keys: the product's first half of channels reads lanes
                // 0-63, the second lanes 64-127.  (Weights go through tensor memory because written to shared memory they would
                // need a proxy fence.)  Their columns are free: U += P(c - 2) V is done, this tile's keys lie where its were.
                const uint32_t p_addr = tmem + lane_off + 384 + 64 * (c & 1);
                ptx::tmem_st_32x32b_x32(p_addr + 32 * half, pk);
                ptx::named_barrier_sync(pair_barrier, 64);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(pk[4 * i]), "=r"(pk[4 * i + 1]), "=r"(pk[4 * i + 2]), "=r"(pk[4 * i + 3])
                                 : "r"(other + ((i ^ (lane & 7)) << 4))
                                 : "memory");
                ptx::tmem_st_32x32b_x32(p_addr + 32 * (half ^ 1), pk);
                ptx::tmem_wait_st();
                // Rows behind the last key that was loaded may hold anything: as values they are zeros, written once the peer's
                // keys are there (S of this tile is done, so nothing else reads them).
                if (key0 + kLatKeys > walk.load_end) {
                    ok = ok && wait_warp(b_vl + 8 * (c & 1), last_phase >> (c & 1) & 1);
                    last_phase ^= 1 << (c & 1);
                    const uint32_t stage = sbase + kLatOffK + (c & 1) * (kLatSlots * kLatPiece);
                    for (int s = 0; s < kLatSlots; ++s) {
                        const bool wide = p.C - 256 * (s >> 2) > 128;   // channels of the slot's block: 256 or 128
                        const int from = max(0, walk.load_end - key0 - 64 * (wide ? (s & 3) >> 1 : s & 1));
                        for (int i = from * 8 + tid; i < 64 * 8; i += 128)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(stage + s * kLatPiece + i * 16), "r"(0) : "memory");
                    }
                    ptx::fence_proxy_async_smem();
                }
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (key0 + kLatKeys > walk.load_end)
                        arrive_remote_release(r_pf + 8 * (c & 1));
                    else
                        arrive_remote(r_pf + 8 * (c & 1));
                }
            }
            // ---- O = U / sum, whole or as a part
            const bool any = walk.hi > walk.lo;
            if (any) {
                ok = ok && wait_warp(b_pv + 16 * ((c - 1) & 1), ((c - 1) >> 1) & 1);
                ptx::tc_fence_after_sync();
            }
            // the two halves' sums (the barrier behind the last exchange of maxima has been passed by both)
            ptx::named_barrier_sync(pair_barrier, 64);
            ctl->top[0][half][row] = sum, ctl->top[1][half][row] = rsum;
            ptx::named_barrier_sync(pair_barrier, 64);
            sum += ctl->top[0][half ^ 1][row], rsum += ctl->top[1][half ^ 1][row];
            ptx::named_barrier_sync(pair_barrier, 64);
            const float inv = rsum != 0.f ? 1.f / rsum : 0.f;
            const float lse2 = sum != 0.f ? ref - kLatShift + log2f(sum) : -INFINITY;
            const int tok = walk.rq.q0 + r / p.H, head = r % p.H;
            const long long part = static_cast<long long>(pair) * 2 + (walk.at_start ? 0 : 1);
            auto u_chunk = [&](int x, uint32_t(&ov)[32]) {  // columns 32 x .. of U over the sum
                if (any) {
                    ptx::tmem_ld_32x32b_x32(tmem + lane_off + 32 * x, ov);
                    ptx::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    if (any) ptx::reg_fence(ov[e]); else ov[e] = 0;
                    ov[e] = __float_as_uint(__uint_as_float(ov[e]) * inv);
                }
            };
            if (walk.whole) {
                // Stores of a row per thread would touch 32 lines each; through the warp's exchange memory eight lanes write
                // 128 bytes of a row.
                const long long at = mine ? static_cast<long long>(tok) * p.o_st + static_cast<long long>(head) * p.o_sh : -1;
                for (int x = 0; x < lat_chunks(p.C); x += 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t ov[32];
                        u_chunk(x + h, ov);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[i] = pack16(__uint_as_float(ov[8 * e + 2 * i]), __uint_as_float(ov[8 * e + 2 * i + 1]), BF16);
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(own + (((4 * h + e) ^ (lane & 7)) << 4)), "r"(w[0]),
                                         "r"(w[1]), "r"(w[2]), "r"(w[3])
                                         : "memory");
                        }
                    }
                    __syncwarp();
                    const int ch = lat_channel(x, half, p.C) + (lane & 7) * 8;
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int y = 4 * i + (lane >> 3);  // row of the box
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                                     : "r"(box + y * 128 + (((lane & 7) ^ (y & 7)) << 4))
                                     : "memory");
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const long long to = __shfl_sync(0xffffffffu, at, 4 * i + (lane >> 3));
                        if (to >= 0 && ch < p.C) *reinterpret_cast<uint4*>(p.o + to + ch) = v[i];
                    }
                    __syncwarp();
                }
            } else if (any && rank * 64 + (warp & 1) * 32 < walk.rows) {  // (an SM stores 32 bytes per cycle: 2 us for all 128 KB)
                for (int x = 0; x < lat_chunks(p.C); ++x) {
                    uint32_t ov[32];
                    u_chunk(x, ov);
                    float4* dst = p.o_part + lat_part(part, rank, warp, x, p.C) + lane;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[32 * e] = make_float4(__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]), __uint_as_float(ov[4 * e + 2]),
                                                  __uint_as_float(ov[4 * e + 3]));
                }
            }
            if (any) {
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_remote(r_oe);
            }
            if (mine && half == 0) {
                if (walk.whole)
                    p.lse[static_cast<long long>(tok) * p.H + head] = lse2 * 0.69314718055994531f;
                else
                    p.stats[part * kLatRows + rank * 64 + row] = make_float2(lse2, rsum != 0.f ? ref - kLatShift + log2f(rsum) : -INFINITY);
            }
        }
    } else if (warp == 4) {
        // ================================================ this CTA's keys
        const uint32_t r_kf = in_first_cta(b_kf);
        int c = 0;
        bool ok = true;
        while (ok && walk.next()) {
            LatPages pages(p, walk, rank, lane);
            if (c > 0 && walk.hi > walk.lo) {
                // the next unit's queries are loaded when the last S of this one is done, which is to be from L2
                for (int i = lane; i < 64 && rank * 64 + i < walk.rows; i += 32) {
                    const int r = walk.r0 + rank * 64 + i;
                    const char* from = reinterpret_cast<const char*>(p.q + static_cast<long long>(walk.rq.q0 + r / p.H) * p.q_st + static_cast<long long>(r % p.H) * p.q_sh);
                    for (int x = 0; x < p.W * 2; x += 128) prefetch_l2(from + x);
                }
                __syncwarp();
            }
            for (int j = walk.lo; ok && j < walk.hi; ++j, ++c) {
                // A share's first two tiles and queries come first of all from memory (128 heads in graphs, 3 to 33 tiles a pair: 0.1
                // to 0.5 us less than without this wait; 16 heads: level up to 4 tiles, then 0.1 to 0.4 less; 71 tiles: level).
                if (c == kLatStages && !(ok = wait_warp(kp > 4 ? b_sh : b_sf, 0))) break;
                if (c >= kLatStages) pages.prefetch(j, lane);
                const int s = c & 1, bytes = pages.both(j);
                const bool load = pages.wanted(j, lane);
                const int row = pages.take(j, lane);
                const uint32_t dst = sbase + kLatOffK + s * (kLatSlots * kLatPiece) + lane * p.box_rows * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int bar = 16 * s + 8 * h, pieces = kp > 4 * h ? max(p.box_pieces, min(4, kp - 4 * h)) : 0;
                    if (c >= kLatStages && !(ok = wait_warp(b_ke + bar, ((c >> 1) - 1) & 1))) break;
                    if (rank == 0 && lane == 0) ptx::mbar_arrive_expect_tx(b_kf + bar, bytes * (pieces + (h == 0 && tail ? 1 : 0)));
                    __syncwarp();
                    if (load && pieces > 0) {
                        if (p.box_pieces > 1)
                            tma_load_3d_pair(dst + 4 * h * kLatPiece, &tm_k, r_kf + bar, 0, row, 4 * h);
                        else
                            for (int i = 4 * h; i < 4 * h + pieces; ++i) tma_load_2d_pair(dst + i * kLatPiece, &tm, r_kf + bar, 64 * i, row);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp == 6) {
        // ============================== the peer's keys as values; channels from 512 on
        const uint32_t r_kf = in_first_cta(b_kf), r_vf = in_first_cta(b_vf);
        auto load_tail = [&](int c, int row) {
            if (row != INT32_MIN) tma_load_2d_pair(sbase + kLatOffTail + lane * p.box_rows * 128, &tm, r_kf + 16 * (c & 1), 64 * kLatSlots, row);
            __syncwarp();
        };
        // The channels from 512 on go a tile ahead: of tile c + 1 as soon as S(c), which takes them first, is half done.
        LatWalk ahead(p, ctl, f0, f1);
        int ca = 0, ja = 0;
        bool more = tail;
        int next_page = -1;
        bool next_wanted = false;
        auto key_of = [&] { return ja * kLatKeys + rank * 64 + lane * p.box_rows; };
        auto advance = [&] {  // to the next tile of the share, its page on its way
            ++ja;
            while (more && ja >= ahead.hi) {
                more = ahead.next();
                if (more) ja = ahead.lo;
            }
            next_wanted = more && lane * p.box_rows < 64 && key_of() < ahead.load_end;
            if (next_wanted)
                next_page = ld_meta(p.table + static_cast<long long>(ahead.b) * p.max_pages + (key_of() >> p.page_shift));
        };
        auto next_row = [&] {
            if (!next_wanted) return INT32_MIN;
            return static_cast<unsigned>(next_page) < static_cast<unsigned>(p.num_pages)
                       ? (next_page << p.page_shift) + (key_of() & ((1 << p.page_shift) - 1)) : -p.box_rows;
        };
        if (more) {
            ahead.hi = 0;
            advance();
            if (more) {
                load_tail(ca++, next_row());
                advance();
            }
        }
        int slots = 0;  // of the peer's keys
        for (int b = 0; b * 256 < p.C; ++b) slots += p.C - 256 * b > 128 ? 2 : 1;
        int c = 0;
        bool ok = true;
        while (ok && walk.next()) {
            LatPages pages(p, walk, rank ^ 1, lane);
            for (int j = walk.lo; j < walk.hi; ++j, ++c) {
                const int s = c & 1;
                const bool load = pages.wanted(j, lane), last = (j + 1) * kLatKeys > walk.load_end;
                const int here = __popc(__ballot_sync(0xffffffffu, load)) * p.box_rows * 128, both = pages.both(j), row = pages.take(j, lane);
                const uint32_t dst = sbase + kLatOffK + s * (kLatSlots * kLatPiece) + lane * p.box_rows * 128;
                // S has passed the first four pieces, then all: as keys they are not needed any more
                for (int b = 0; b < 2; ++b) {
                    if (!(ok = wait_warp((b == 0 && kp > 4 ? b_sh : b_sf) + 8 * s, (c >> 1) & 1))) break;
                    if (b == 0 && lane == 0) {
                        if (last) ptx::mbar_arrive_expect_tx(b_vl + 8 * s, here * slots);
                        else if (rank == 0) ptx::mbar_arrive_expect_tx(b_vf + 8 * s, both * slots);
                    }
                    __syncwarp();
                    if (load && b * 256 < p.C) {
                        const int wide = p.C - 256 * b > 128 ? 2 : 1;
                        for (int i = 0; i < wide; ++i)
                            tma_load_2d_pair(dst + (4 * b + wide * (rank ^ 1) + i) * kLatPiece, &tm, last ? b_vl + 8 * s : r_vf + 8 * s, 64 * (4 * b + wide * rank + i), row);
                    }
                    __syncwarp();
                    if (b == 0 && more) {
                        load_tail(ca++, next_row());
                        advance();
                    }
                }
                if (!ok) break;
            }
        }
        // nothing may still be landing in this CTA's memory when it ends
        for (int i = max(0, c - 2); i < c; ++i) wait_warp(b_pv + 16 * (i & 1), (i >> 1) & 1);
    } else if (warp == 5) {
        // ============================================== tensor-core issuer of S
        if (rank == 0) {
            const uint32_t id_s = lat_instr(BF16, kLatKeys, false);
            const uint64_t q_desc = lat_desc(sbase, 16), k_desc = lat_desc(sbase + kLatOffK, 16), t_desc = lat_desc(sbase + kLatOffTail, 16);
            constexpr uint64_t kPieceStep = kLatPiece / 16, kStageStep = kLatSlots * kPieceStep;
            int c = 0, parts = 0;
            bool ok = true;
            while (ok && walk.next()) {
                if (walk.hi == walk.lo) continue;
                if (!(ok = wait_pair_lean(b_qf, parts & 1))) break;
                ++parts;
                for (int j = walk.lo; j < walk.hi; ++j, ++c) {
                    const uint32_t d = tmem + 256 + 64 * (c & 1);
                    const uint64_t kd = k_desc + (c & 1) * kStageStep;
                    // the scores of tile c - 2 were read before its weights were handed over; then in halves as the keys arrive
                    if (c >= 2 && !(ok = wait_pair_lean(b_pf + 8 * (c & 1), ((c >> 1) - 1) & 1))) break;
                    if (!(ok = wait_pair_lean(b_kf + 16 * (c & 1), (c >> 1) & 1))) break;
                    ptx::tc_fence_after_sync();
                    if (tail) mma_pair_k64(d, q_desc + kLatSlots * kPieceStep, t_desc, id_s, 0u);
                    for (int i = 0; i < min(kp, 4); ++i) mma_pair_k64(d, q_desc + i * kPieceStep, kd + i * kPieceStep, id_s, tail || i > 0);
                    if (kp > 4) commit_pair(b_sh + 8 * (c & 1));
                    if (!(ok = wait_pair_lean(b_kf + 16 * (c & 1) + 8, (c >> 1) & 1))) break;
                    ptx::tc_fence_after_sync();
                    for (int i = 4; i < min(kp, kLatSlots); ++i) mma_pair_k64(d, q_desc + i * kPieceStep, kd + i * kPieceStep, id_s, 1u);
                    commit_pair(b_sf + 8 * (c & 1));
                    if (j + 1 == walk.hi) commit_pair(b_qe);
                }
            }
            __syncwarp();
            commit_pair_here(b_drain);
            __syncwarp();
            wait_warp(b_drain, 0);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ====================================== tensor-core issuer of U += P V
        if (rank == 0) {
            const uint64_t v_desc = lat_desc(sbase + kLatOffK, kLatPiece);
            constexpr uint64_t kPieceStep = kLatPiece / 16, kStageStep = kLatSlots * kPieceStep;
            int c = 0, parts = 0, v_phase = 0;
            bool ok = true;
            while (ok && walk.next()) {
                if (walk.hi == walk.lo) continue;
                for (int j = walk.lo; j < walk.hi; ++j, ++c) {
                    if (j == walk.lo && parts > 0 && !(ok = wait_pair_lean(b_oe, (parts - 1) & 1))) break;
                    if ((j + 1) * kLatKeys <= walk.load_end) {
                        if (!(ok = wait_pair_lean(b_vf + 8 * (c & 1), v_phase >> (c & 1) & 1))) break;
                        v_phase ^= 1 << (c & 1);
                    }
                    if (!(ok = wait_pair_lean(b_pf + 8 * (c & 1), (c >> 1) & 1))) break;
                    ptx::tc_fence_after_sync();
                    const uint64_t vd = v_desc + (c & 1) * kStageStep;
                    const uint32_t weights = tmem + 384 + 64 * (c & 1);
                    for (int b = 0; b < 2; ++b) {
                        if (b * 256 < p.C) {
                            const int wide = p.C - 256 * b > 128 ? 2 : 1;
                            const uint32_t id = lat_instr(BF16, 128 * wide, true);
                            const uint64_t vb = vd + 4 * b * kPieceStep;
                            mma_pair_ts_k64(tmem + 128 * b, weights, vb, id, j > walk.lo);
                            mma_pair_ts_k64(tmem + 128 * b, weights + 32, vb + wide * kPieceStep, id, 1u);
                        }
                        commit_pair(b_ke + 16 * (c & 1) + 8 * b);
                    }
                }
                ++parts;
            }
            __syncwarp();
            commit_pair_here(b_drain + 8);
            __syncwarp();
            wait_warp(b_drain + 8, 0);
        }
        __syncwarp();
    } else {
        // ============================================================ queries
        const uint32_t r_qf = in_first_cta(b_qf);
        const int t = tid - 224;
        int parts = 0;
        while (walk.next()) {
            if (walk.hi == walk.lo) continue;
            if (p.q_box && warp == 8) break;  // (one warp's boxes)
            if (parts > 0 && !wait_warp(b_qe, (parts - 1) & 1)) break;
            const int here = max(0, min(64, walk.rows - rank * 64));  // rows
            if (p.q_box) {
                // rows behind the last one are left as they are: no other row's result takes from them
                const int boxes = (here + p.q_box - 1) / p.q_box;     // (whole boxes: H is a multiple of q_box)
                if (lane == 0) arrive_remote_expect(r_qf, boxes * kp * p.q_box * 128);
                __syncwarp();
                for (int i = lane; i < boxes * kp; i += 32) {
                    const int piece = i / boxes, box = i - piece * boxes, r = walk.r0 + rank * 64 + box * p.q_box;
                    tma_load_3d_pair(sbase + piece * kLatPiece + box * p.q_box * 128, &tm_q, r_qf, 64 * piece, r % p.H, walk.rq.q0 + r / p.H);
                }
                __syncwarp();
            } else {
                const int ch = (t & 7) * 8;
#pragma unroll 1
                for (int row = t >> 3; row < 64; row += 8) {
                    const int r = walk.r0 + rank * 64 + row;
                    const bool mine = row < here;
                    const uint16_t* src = p.q + static_cast<long long>(walk.rq.q0 + (mine ? r / p.H : 0)) * p.q_st +
                                          static_cast<long long>(mine ? r % p.H : 0) * p.q_sh + ch;
                    const uint32_t dst = sbase + row * 128 + (((t & 7) ^ (row & 7)) << 4);
                    for (int i = 0; i < kp; ++i) {
                        const bool there = mine && 64 * i + ch < p.W;
                        cp_async16(dst + i * kLatPiece, there ? src + 64 * i : p.q, there);
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                ptx::fence_proxy_async_smem();
                arrive_remote_release(r_qf);
            }
            ++parts;
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA's memory is written or read by the other any more
    if (warp == 5) {
        ptx::tc_fence_after_sync();
        tmem_dealloc_pair(tmem);
    }
}

// The parts of the units that shares cut.  A job is what a softmax warp of a unit held of 32 channels: its lanes' rows, from
// each part.  CTA (x, y): boundary between shares x and x + 1, and eight jobs, a warp each; where few units are cut into
// many parts (SPLIT) one job, whose parts the CTA's warps take in turn and join in shared memory.
// O = sum_s w_s O_s / sum_s w_s with w_s the sum of a part's rounded weights (its O_s is divided by that), LSE from the
// sums of the fp32 weights.
constexpr int kLatJoinWarps = 8;
template <bool BF16, bool SPLIT>
__global__ void __launch_bounds__(32 * kLatJoinWarps) latent_join_kernel(const LatentParams p) {
    constexpr int STEP = SPLIT ? kLatJoinWarps : 1;
    dependents_may_start();
    wait_for_previous();
    const int pairs = static_cast<int>(gridDim.x) + 1, i = blockIdx.x + 1, lane = threadIdx.x & 31, w0 = threadIdx.x >> 5;
    const int4 unit = ld(p.shares + 2 * i), request = ld(p.shares + 2 * i + 1);
    const int share = unit.w;
    const long long at = static_cast<long long>(i) * share;
    if (unit.x >= at || unit.y <= at || at - share > unit.x) return;  // not inside a unit, or not the first boundary inside
    // part of share i - 1 (its first unit or its last), then the first ones of the shares that begin inside
    const int parts = 1 + static_cast<int>(min(static_cast<long long>(pairs - i), (unit.y - at + share - 1) / share));
    const int chunks = lat_chunks(p.C), job = SPLIT ? blockIdx.y : blockIdx.y * kLatJoinWarps + w0;
    const int chunk = job % chunks, warp = job / chunks & 3, rank = job / (4 * chunks);
    const int head_slot = unit.x == at - share ? 0 : 1, row = rank * 64 + (warp & 1) * 32 + lane;
    auto part_of = [&](int j) { return static_cast<long long>(i - 1 + j) * 2 + (j == 0 ? head_slot : 0); };
    const int r = unit.z * kLatRows + row, q0 = request.x, rows = request.y * p.H;
    const bool mine = r < rows;
    if (unit.z * kLatRows + rank * 64 + (warp & 1) * 32 >= rows) return;  // (the whole CTA's, or a warp's own)
    // Two parts of O at a time, the first two on their way while the statistics are read.
    float4 v[2][8];
    auto load = [&](int j0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4* src = p.o_part + lat_part(part_of(min(j0 + j * STEP, parts - 1)), rank, warp, chunk, p.C) + lane;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = ld(src + 32 * e);
        }
    };
    load(SPLIT ? w0 : 0);
    auto stats_of = [&](int j) {
        return mine && j < parts ? ld(p.stats + part_of(j) * kLatRows + row) : make_float2(-INFINITY, -INFINITY);
    };
    float top = -INFINITY, rtop = -INFINITY, l = 0.f, rl = 0.f;
    const int first = SPLIT ? w0 : 0;
#pragma unroll 8
    for (int j = first; j < parts; j += STEP) {
        const float2 a = stats_of(j);
        top = fmaxf(top, a.x), rtop = fmaxf(rtop, a.y);
    }
    const float ref = top == -INFINITY ? 0.f : top, rref = rtop == -INFINITY ? 0.f : rtop;
    float o[32] = {};
    for (int j0 = first; j0 < parts; j0 += 2 * STEP) {
        if (j0 > first) load(j0);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 a = stats_of(j0 + j * STEP);
            const float w = ptx::ex2_approx(a.y - rref);
            l += ptx::ex2_approx(a.x - ref), rl += w;
            const bool use = w != 0.f;  // (a part without a key wrote no O)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[4 * e] = use ? fmaf(v[j][e].x, w, o[4 * e]) : o[4 * e], o[4 * e + 1] = use ? fmaf(v[j][e].y, w, o[4 * e + 1]) : o[4 * e + 1];
                o[4 * e + 2] = use ? fmaf(v[j][e].z, w, o[4 * e + 2]) : o[4 * e + 2], o[4 * e + 3] = use ? fmaf(v[j][e].w, w, o[4 * e + 3]) : o[4 * e + 3];
            }
        }
    }
    const int ch = lat_channel(chunk, warp >> 1, p.C), tok = mine ? q0 + r / p.H : 0, head = r % p.H;
    uint16_t* dst = p.o + static_cast<long long>(tok) * p.o_st + static_cast<long long>(head) * p.o_sh + ch;
    float lse2 = l != 0.f ? ref + log2f(l) : -INFINITY;
    if constexpr (SPLIT) {
        // warp w0 joins channels 4 w0 .. of all warps' results
        __shared__ float4 part_o[kLatJoinWarps][8][32];
        __shared__ float4 part_s[kLatJoinWarps][32];
        part_s[w0][lane] = make_float4(top, rtop, l, rl);
#pragma unroll
        for (int e = 0; e < 8; ++e) part_o[w0][e][lane] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        __syncthreads();
        float4 s[kLatJoinWarps];
        float all = -INFINITY, rall = -INFINITY;
#pragma unroll
        for (int k = 0; k < kLatJoinWarps; ++k) s[k] = part_s[k][lane], all = fmaxf(all, s[k].x), rall = fmaxf(rall, s[k].y);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        l = rl = 0.f;
#pragma unroll
        for (int k = 0; k < kLatJoinWarps; ++k) {
            const float w = s[k].y == -INFINITY ? 0.f : ptx::ex2_approx(s[k].y - rall);
            // (by the sum, not by the maximum, which passes over NaN)
            l += s[k].z == 0.f ? 0.f : s[k].z * ptx::ex2_approx(s[k].x - all);
            rl += s[k].w * w;
            const float4 v = part_o[k][w0][lane];
            sum.x = fmaf(v.x, w, sum.x), sum.y = fmaf(v.y, w, sum.y), sum.z = fmaf(v.z, w, sum.z), sum.w = fmaf(v.w, w, sum.w);
        }
        const float inv = rl != 0.f ? 1.f / rl : 0.f;
        lse2 = l != 0.f ? all + log2f(l) : -INFINITY;
        if (mine && ch + 4 * w0 < p.C)
            *reinterpret_cast<uint2*>(dst + 4 * w0) = make_uint2(pack16(sum.x * inv, sum.y * inv, BF16), pack16(sum.z * inv, sum.w * inv, BF16));
    } else if (mine) {
        const float inv = rl != 0.f ? 1.f / rl : 0.f;
#pragma unroll
        for (int e = 0; e < 32; e += 8)
            if (ch + e < p.C)
                *reinterpret_cast<uint4*>(dst + e) = make_uint4(pack16(o[e] * inv, o[e + 1] * inv, BF16), pack16(o[e + 2] * inv, o[e + 3] * inv, BF16),
                                                                pack16(o[e + 4] * inv, o[e + 5] * inv, BF16), pack16(o[e + 6] * inv, o[e + 7] * inv, BF16));
    }
    if (mine && ch == 0 && (!SPLIT || w0 == 0))
        p.lse[static_cast<long long>(tok) * p.H + head] = lse2 == -INFINITY ? lse2 : lse2 * 0.69314718055994531f;
}

}  // namespace paged
}  // namespace fa
