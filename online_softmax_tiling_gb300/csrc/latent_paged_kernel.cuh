// latent_paged_kernel.cuh - latent attention in its absorbed form over a paged latent cache.
//
// Every head of a request reads the same keys, rows of W = C + R channels, and the values are the
// first C channels of the same rows:
//   O = softmax(scale q c^T) c[:, :C],   W <= 576, C <= 512.
// A key brings 2 W bytes and 2 (W + C) operations per head: with 128 heads and one token 241 per byte,
// below the 286 at which the tensor cores and HBM take the same time, so HBM bounds decoding as
// long as each key is read from it once and enters both products from shared memory.
//
// Mapping.  Packed rows r = i H + g (query i, head g) of a request; a CTA takes 64 of them, and one CTA fills
// an SM: 64 rows of queries (72 KB), two tiles of 64 keys (144 KB), the tile's weights (8 KB).  128 rows would
// leave room for neither the accumulator (512 fp32 columns) beside the scores, nor a second key tile.
// tcgen05.mma.ws with M = 64 spreads 64 rows by N columns over all 128 lanes of tensor memory (lanes 0-63
// hold the first N / 2 columns, lanes 64-127 the others), so 64 x 512 fp32 take 256 columns.
//   * warps 0-3: softmax and epilogue.  Warp w has rows 32 (w & 1) .. and keys 32 (w >> 1) .. of a tile;
//     the two warps of a row exchange its maximum through shared memory;
//   * warp 4: TMA of the key tiles, pages looked up three tiles ahead;
//   * warp 5: tcgen05.mma: S(j + 1) = Q K(j + 1)^T before U += P(j) V(j), so that the tensor core works
//     while the weights of tile j + 1 are computed;
//   * warps 6-7: query rows by cp.async (any strides), for the next unit as soon as the last S of this one is done.
// TMEM: U 0-255, S 256-287 and 288-319.
//
// Weights are 2^(x - ref + 7) in the operands' 16-bit type; ref is the row's maximum when it last moved, and moves only
// where the maximum has grown by more than 2^8 (fp16 holds 2^15), with U rescaled then.  O is divided by the sum of
// the rounded weights, the LSE takes the sum of the fp32 ones.
//
// Sharing out.  All (request, row blocks, tile) of a call, in that order, are dealt out in equal shares to as many
// CTAs as run at once, whatever the lengths.  With more than 64 rows two CTAs (a group) go over the same
// share, one for each row block of a pair, so that a key comes from HBM once.  Parts of a unit go
// through a workspace and are joined by a second launch.
#pragma once

#include "paged_common.cuh"

namespace fa {
namespace paged {

constexpr int kLatRows = 64, kLatKeys = 64;
constexpr int kLatThreads = 256;
constexpr int kLatPieces = 9;                 // 64-channel pieces of a row: W <= 576
constexpr int kLatPiece = 64 * 128;           // 64 rows x 64 16-bit channels, 128-byte swizzle
constexpr int kLatStages = 2;
constexpr int kLatOffK = kLatPieces * kLatPiece;
constexpr int kLatOffP = kLatOffK + kLatStages * kLatPieces * kLatPiece;
constexpr int kLatOffCtl = kLatOffP + kLatPiece;
constexpr int kLatMaxB = 16384;
constexpr float kLatShift = 7.f, kLatLag = 8.f;

struct LatentParams {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    const int* cu_q;
    const int* table;
    const int* lens;
    long long q_st, q_sh, o_st, o_sh;
    int T, B, H, C, W, max_q, max_pages, num_pages, page_shift;
    int members;      // CTAs of a group: 1, or 2 (row blocks 2 i and 2 i + 1)
    int min_share;    // tiles
    int box_rows;
    int causal;
    float scale_log2;
    float* o_part;    // [2 CTAs][64][C]: the parts of a share's first and last unit
    float2* stats;    // [2 CTAs][64]: log2 of the sums of the fp32 and of the rounded weights
    int4* shares;     // [groups + 1]: first unit's begin, end, request, pair; behind the last: the share
};

struct LatCtl {
    uint64_t q_full, q_empty, k_full[kLatStages], k_empty[kLatStages], s_full[2], p_full, pv_done, o_empty, drain;
    uint32_t tmem_base;
    int start[4];                 // request, pair, tile of the share's first unit; tiles of all units
    float top[2][2][kLatRows];    // by tile parity, key half, row
};
static_assert(kLatOffCtl + sizeof(LatCtl) + 1024 <= 232448, "shared memory of a CTA");
constexpr int kLatSmem = kLatOffCtl + static_cast<int>(sizeof(LatCtl)) + 1024;

__device__ __forceinline__ uint64_t lat_desc(uint32_t saddr, uint32_t lbo) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint32_t lat_instr(bool bf16, int n, bool b_mn_major) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           ((static_cast<uint32_t>(n) >> 3) << 17) | ((64u >> 4) << 24);
}
// D (tmem) (+)= A (smem) B (smem)^T, 64 rows over all lanes.
__device__ __forceinline__ void mma_ws(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.ws.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Rows and keys of request b, and its units: pairs of row blocks times tiles of keys (at least one).
struct LatRequest {
    int q0, nq, len, pairs, tiles;
};
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
    r.pairs = (r.nq * p.H + p.members * kLatRows - 1) / (p.members * kLatRows);
    r.tiles = max(1, (r.len + kLatKeys - 1) / kLatKeys);
    return r;
}

// Walks the parts of a CTA's share: for every unit some tiles of its keys.
struct LatWalk {
    const LatentParams& p;
    const int member, f0, f1;
    int f, b, pair, first;
    LatRequest rq;
    // of the current part
    int r0, rows, lo, hi, kend;   // this CTA's rows, and their tiles [lo, hi)
    bool whole, at_start;

    __device__ LatWalk(const LatentParams& p_, const LatCtl* ctl, int member_, int f0_, int f1_)
        : p(p_), member(member_), f0(f0_), f1(f1_), f(f0_), b(ctl->start[0]), pair(ctl->start[1]), first(ctl->start[2]) {
        bool bad = false;
        if (f < f1) rq = lat_request(p, b, bad);
    }
    __device__ int limit(int r) const { return p.causal ? min(rq.len, rq.len - rq.nq + r / p.H + 1) : rq.len; }
    // the next part; false behind the last
    __device__ bool next() {
        if (f >= f1) return false;
        while (pair >= rq.pairs) {  // (units are left, so there is a request that has some)
            if (b + 1 >= p.B) return false;
            bool bad = false;
            ++b, pair = 0;
            rq = lat_request(p, b, bad);
        }
        const int n = min(rq.tiles - first, f1 - f);
        r0 = (pair * p.members + member) * kLatRows;
        rows = max(0, min(kLatRows, rq.nq * p.H - r0));
        kend = rows > 0 ? max(0, limit(r0 + rows - 1)) : 0;
        const int kt = (kend + kLatKeys - 1) / kLatKeys;
        lo = min(first, kt), hi = min(first + n, kt);
        whole = first == 0 && n == rq.tiles;
        at_start = f == f0;
        f += n;
        first = 0;
        ++pair;
        return true;
    }
};

template <bool BF16>
__global__ void __launch_bounds__(kLatThreads, 1)
    latent_paged_kernel(const __grid_constant__ CUtensorMap tm, const LatentParams p) {
    extern __shared__ __align__(16) uint8_t lat_raw[];
    const uint32_t raw = ptx::smem_addr(lat_raw);
    uint8_t* smem = lat_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = ptx::smem_addr(smem);
    LatCtl* ctl = reinterpret_cast<LatCtl*>(smem + kLatOffCtl);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const uint32_t b_qf = ptx::smem_addr(&ctl->q_full), b_qe = ptx::smem_addr(&ctl->q_empty);
    const uint32_t b_kf = ptx::smem_addr(&ctl->k_full[0]), b_ke = ptx::smem_addr(&ctl->k_empty[0]);
    const uint32_t b_sf = ptx::smem_addr(&ctl->s_full[0]), b_pf = ptx::smem_addr(&ctl->p_full);
    const uint32_t b_pv = ptx::smem_addr(&ctl->pv_done), b_oe = ptx::smem_addr(&ctl->o_empty);
    const uint32_t b_drain = ptx::smem_addr(&ctl->drain);
    if (tid == 0) {
        ptx::mbar_init(b_qf, 64);
        ptx::mbar_init(b_qe, 1);
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(b_kf + 8 * s, 1);
            ptx::mbar_init(b_ke + 8 * s, 1);
            ptx::mbar_init(b_sf + 8 * s, 1);
        }
        ptx::mbar_init(b_pf, 128);
        ptx::mbar_init(b_pv, 1);
        ptx::mbar_init(b_oe, 128);
        ptx::mbar_init(b_drain, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tm);
    }
    if (warp == 5) {
        ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    dependents_may_start();
    wait_for_previous();

    // ---- this group's share [f0, f1) of all tiles, in order of request, pair of row blocks, tile
    const int groups = gridDim.x / p.members, group = blockIdx.x / p.members, member = blockIdx.x - group * p.members;
    int f0, f1;
    {
        int* before = reinterpret_cast<int*>(smem);  // (the tiles' memory) tiles before each of a thread's runs of requests
        const int per = (p.B + kLatThreads - 1) / kLatThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
        bool bad = false;
        int own = 0;
        for (int b = b0; b < b1; ++b) {
            const LatRequest r = lat_request(p, b, bad);
            own += r.pairs * r.tiles;
        }
        if (bad) report(kBadData);
        int incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) before[warp] = incl;
        ptx::tc_fence_before_sync();
        __syncthreads();
        ptx::tc_fence_after_sync();
        int run = incl - own, all = 0;
        for (int w = 0; w < kLatThreads / 32; ++w) {
            if (w < warp) run += before[w];
            all += before[w];
        }
        const int share = max((all + groups - 1) / groups, p.min_share);
        f0 = static_cast<int>(min(static_cast<long long>(group) * share, static_cast<long long>(all)));
        f1 = static_cast<int>(min(static_cast<long long>(f0) + share, static_cast<long long>(all)));
        if (f0 < f1 && run <= f0 && f0 < run + own) {
            for (int b = b0; b < b1; ++b) {
                const LatRequest r = lat_request(p, b, bad);
                const int n = r.pairs * r.tiles;
                if (f0 < run + n) {
                    const int rel = f0 - run;
                    ctl->start[0] = b, ctl->start[1] = rel / r.tiles, ctl->start[2] = rel % r.tiles, ctl->start[3] = r.tiles;
                    break;
                }
                run += n;
            }
        }
        ptx::fence_proxy_async_smem();  // (what was read and written here is the key tiles' and queries' memory)
        __syncthreads();
        if (p.shares && member == 0 && tid == 0) {
            int4 u = make_int4(f0, f0, 0, 0);
            if (f0 < f1) u = make_int4(f0 - ctl->start[2], f0 - ctl->start[2] + ctl->start[3], ctl->start[0], ctl->start[1]);
            p.shares[group] = u;
            if (group == 0) p.shares[groups] = make_int4(share, 0, 0, 0);
        }
    }
    const uint32_t tmem = ctl->tmem_base;
    const int kp = (p.W + 63) >> 6;
    LatWalk walk(p, ctl, member, f0, f1);

    if (warp < 4) {
        // ================================================ softmax and epilogue
        const int half = warp >> 1, row = (warp & 1) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t p_row = sbase + kLatOffP + row * 128;
        const int pair_barrier = 1 + (warp & 1);
        int c = 0;  // tiles so far
        bool ok = true;  // (after a wait that ran out nothing is waited for, but every barrier of the pair is still met)
        while (walk.next()) {
            const int r = walk.r0 + row;
            const bool mine = row < walk.rows;
            const int my_limit = mine ? walk.limit(r) : walk.rq.len;
            const int first_limit = walk.limit(walk.r0);  // the least of the block's rows
            const int load_end = min(walk.rq.len, (walk.kend + p.box_rows - 1) / p.box_rows * p.box_rows);
            float ref = -INFINITY, sum = 0.f, rsum = 0.f;  // sums of this thread's keys: fp32 and rounded weights
            for (int j = walk.lo; j < walk.hi; ++j, ++c) {
                ok = ok && wait_warp(b_sf + 8 * (c & 1), (c >> 1) & 1);
                ptx::tc_fence_after_sync();
                const int key0 = j * kLatKeys;
                uint32_t sv[32];
                ptx::tmem_ld_32x32b_x32(tmem + lane_off + 256 + 32 * (c & 1), sv);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) ptx::reg_fence(sv[e]);
                if (key0 + kLatKeys > first_limit) {
                    const int seen = my_limit - key0 - 32 * half;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (e >= seen) sv[e] = __float_as_uint(-INFINITY);
                }
                float top = __uint_as_float(sv[0]);
#pragma unroll
                for (int e = 1; e + 1 < 32; e += 2) top = ptx::fmax3(top, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                top = fmaxf(top, __uint_as_float(sv[31]));
                ctl->top[c & 1][half][row] = top;
                ptx::named_barrier_sync(pair_barrier, 64);
                top = fmaxf(top, ctl->top[c & 1][half ^ 1][row]) * p.scale_log2;
                // U holds the products of the tiles before, and the weights' memory is free
                if (c > 0) ok = ok && wait_warp(b_pv, (c - 1) & 1);
                ptx::tc_fence_after_sync();
                const bool moves = top > ref + kLatLag;  // (the same in both warps of the row)
                if (__any_sync(0xffffffffu, moves)) {
                    float alpha = 1.f;
                    if (moves) {
                        if (ref != -INFINITY) alpha = ptx::ex2_approx(ref - top);
                        ref = top;
                    }
                    sum *= alpha, rsum *= alpha;
                    if (j > walk.lo) {
                        const float2 av = make_float2(alpha, alpha);
                        const int cols = p.C <= 64 ? 32 : p.C <= 128 ? 64 : p.C <= 256 ? 128 : 256;
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
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), fv, nv);
                    const float2 w = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
                    acc = __fadd2_rn(acc, w);
                    pk[e] = pack16(w.x, w.y, BF16);
                    racc = __fadd2_rn(racc, unpack16(pk[e], BF16));
                }
                sum += acc.x + acc.y, rsum += racc.x + racc.y;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p_row + (((4 * half + i) ^ (row & 7)) << 4)),
                                 "r"(pk[4 * i]), "r"(pk[4 * i + 1]), "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3])
                                 : "memory");
                // rows behind the last key that was loaded may hold anything: as values they are zeros
                // (S of this tile is done, so nothing else reads them)
                if (key0 + kLatKeys > load_end) {
                    const uint32_t tile = sbase + kLatOffK + (c & 1) * (kLatPieces * kLatPiece);
                    const int from = max(0, load_end - key0);
                    const int chunks = kLatKeys - from;  // rows
                    for (int i = tid; i < chunks * 8 * kp; i += 128) {
                        const int piece = i / (8 * chunks), at = i - piece * (8 * chunks);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + piece * kLatPiece + from * 128 + at * 16), "r"(0)
                                     : "memory");
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before_sync();
                ptx::mbar_arrive(b_pf);
            }
            // ---- O = U / sum, whole or as a part
            const bool any = walk.hi > walk.lo;
            if (any) {
                ok = ok && wait_warp(b_pv, (c - 1) & 1);
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
            const long long part = static_cast<long long>(blockIdx.x) * 2 + (walk.at_start ? 0 : 1);
            uint16_t* dst = p.o + static_cast<long long>(tok) * p.o_st + static_cast<long long>(head) * p.o_sh;
            float* pdst = p.o_part + (part * kLatRows + row) * p.C;
            if (any || walk.whole) {
                for (int h = 0; h * 256 < p.C; ++h) {
                    const int left = p.C - 256 * h, wide = left <= 64 ? 32 : left <= 128 ? 64 : 128;
#pragma unroll 1
                    for (int x = 0; x < wide; x += 32) {
                        uint32_t ov[32];
                        if (any) {
                            ptx::tmem_ld_32x32b_x32(tmem + lane_off + 128 * h + x, ov);
                            ptx::tmem_wait_ld();
                        }
                        const int d0 = 256 * h + half * wide + x;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float f[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (any) ptx::reg_fence(ov[e + i]); else ov[e + i] = 0;
                                f[i] = __uint_as_float(ov[e + i]) * inv;
                            }
                            if (!mine || d0 + e >= p.C) continue;
                            if (walk.whole) {
                                *reinterpret_cast<uint4*>(dst + d0 + e) = make_uint4(
                                    pack16(f[0], f[1], BF16), pack16(f[2], f[3], BF16), pack16(f[4], f[5], BF16), pack16(f[6], f[7], BF16));
                            } else {
                                *reinterpret_cast<float4*>(pdst + d0 + e) = make_float4(f[0], f[1], f[2], f[3]);
                                *reinterpret_cast<float4*>(pdst + d0 + e + 4) = make_float4(f[4], f[5], f[6], f[7]);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (any) {
                ptx::tc_fence_before_sync();
                ptx::mbar_arrive(b_oe);
            }
            if (mine && half == 0) {
                if (walk.whole)
                    p.lse[static_cast<long long>(tok) * p.H + head] = lse2 * 0.69314718055994531f;
                else
                    p.stats[part * kLatRows + row] =
                        make_float2(lse2, rsum != 0.f ? ref - kLatShift + log2f(rsum) : -INFINITY);
            }
        }
    } else if (warp == 4) {
        // ========================================================== key tiles
        const int boxes = kLatKeys / p.box_rows;   // of a tile
        int c = 0;
        bool ok = true;
        while (ok && walk.next()) {
            const int* trow = p.table + static_cast<long long>(walk.b) * p.max_pages;
            const int load_end = min(walk.rq.len, (walk.kend + p.box_rows - 1) / p.box_rows * p.box_rows);
            auto page_of = [&](int j) {  // this lane's box of tile j: its page, -1 where it is not read
                const int key = j * kLatKeys + lane * p.box_rows;
                return j < walk.hi && lane < boxes && key < load_end ? ld_meta(trow + (key >> p.page_shift)) : -1;
            };
            int page = page_of(walk.lo), page1 = page_of(walk.lo + 1), page2 = page_of(walk.lo + 2);
            for (int j = walk.lo; j < walk.hi; ++j, ++c) {
                const int page3 = page_of(j + 3);
                const int s = c & 1, key = j * kLatKeys + lane * p.box_rows;
                const bool wanted = lane < boxes && key < load_end;
                const bool there = wanted && static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
                if (wanted && !there) report(kBadData);
                const int n = __popc(__ballot_sync(0xffffffffu, there));
                if (c >= kLatStages && !(ok = wait_warp(b_ke + 8 * s, ((c >> 1) - 1) & 1))) break;
                if (lane == 0) {
                    if (n > 0)
                        ptx::mbar_arrive_expect_tx(b_kf + 8 * s, n * kp * p.box_rows * 128);
                    else
                        ptx::mbar_arrive(b_kf + 8 * s);
                }
                __syncwarp();
                if (there) {
                    const int at = (page << p.page_shift) + (key & ((1 << p.page_shift) - 1));
                    const uint32_t dst = sbase + kLatOffK + s * (kLatPieces * kLatPiece) + lane * p.box_rows * 128;
                    for (int i = 0; i < kp; ++i) tma_load_2d(dst + i * kLatPiece, &tm, b_kf + 8 * s, 64 * i, at);
                }
                __syncwarp();
                page = page1, page1 = page2, page2 = page3;
            }
        }
        // nothing may still be landing in this CTA's memory when it ends
        for (int i = max(0, c - kLatStages); i < c; ++i) wait_warp(b_kf + 8 * (i & 1), (i >> 1) & 1);
    } else if (warp == 5) {
        // ================================================== tensor-core issuer
        const uint32_t id_s = lat_instr(BF16, kLatKeys, false);
        const uint64_t q_desc = lat_desc(sbase, 16), k_desc = lat_desc(sbase + kLatOffK, 16);
        const uint64_t p_desc = lat_desc(sbase + kLatOffP, 16), v_desc = lat_desc(sbase + kLatOffK, kLatPiece);
        constexpr uint64_t kPieceStep = kLatPiece / 16, kStageStep = kLatPieces * kPieceStep;
        const int steps = (p.W + 15) >> 4;
        auto issue_s = [&](int c) {
            const uint64_t kd = k_desc + (c & 1) * kStageStep;
            if (ptx::elect_one()) {
                for (int i = 0; i < steps; ++i) {
                    const uint64_t off = (i >> 2) * kPieceStep + 2 * (i & 3);
                    mma_ws(tmem + 256 + 32 * (c & 1), q_desc + off, kd + off, id_s, i > 0);
                }
            }
            __syncwarp();
            ptx::tc_commit_elect(b_sf + 8 * (c & 1));
        };
        auto issue_pv = [&](int c, bool accumulate) {
            const uint64_t vd = v_desc + (c & 1) * kStageStep;
            if (ptx::elect_one()) {
                for (int h = 0; h * 256 < p.C; ++h) {
                    const int left = p.C - 256 * h;
                    const uint32_t id = lat_instr(BF16, left <= 64 ? 64 : left <= 128 ? 128 : 256, true);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_ws(tmem + 128 * h, p_desc + 2 * i, vd + h * 4 * kPieceStep + 128 * i, id, accumulate || i > 0);
                }
            }
            __syncwarp();
        };
        int c = 0, parts = 0;
        bool ok = true;
        while (ok && walk.next()) {
            const int n = walk.hi - walk.lo;
            if (n == 0) continue;
            if (!(ok = wait_warp(b_qf, parts & 1) && wait_warp(b_kf + 8 * (c & 1), (c >> 1) & 1))) break;
            ptx::tc_fence_after_sync();
            issue_s(c);
            if (n == 1) ptx::tc_commit_elect(b_qe);
            for (int i = 0; i < n; ++i, ++c) {
                if (i + 1 < n) {
                    if (!(ok = wait_warp(b_kf + 8 * ((c + 1) & 1), ((c + 1) >> 1) & 1))) break;
                    ptx::tc_fence_after_sync();
                    issue_s(c + 1);  // (its columns were read before the weights of tile c - 1 were handed over)
                    if (i + 2 == n) ptx::tc_commit_elect(b_qe);
                }
                if (!(ok = wait_warp(b_pf, c & 1))) break;
                if (i == 0 && parts > 0 && !(ok = wait_warp(b_oe, (parts - 1) & 1))) break;
                ptx::tc_fence_after_sync();
                issue_pv(c, i > 0);
                ptx::tc_commit_elect(b_ke + 8 * (c & 1));
                ptx::tc_commit_elect(b_pv);
                __syncwarp();
            }
            ++parts;
        }
        ptx::tc_commit_elect(b_drain);
        __syncwarp();
        wait_warp(b_drain, 0);
    } else {
        // ============================================================ queries
        const int t = tid - 192;
        int parts = 0;
        while (walk.next()) {
            if (walk.hi == walk.lo) continue;
            if (parts > 0 && !wait_warp(b_qe, (parts - 1) & 1)) break;
            const int ch = (t & 7) * 8;
#pragma unroll 1
            for (int row = t >> 3; row < kLatRows; row += 8) {
                const int r = walk.r0 + row;
                const bool mine = row < walk.rows;
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
            ptx::mbar_arrive(b_qf);
            ++parts;
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 5) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// The parts of the units that shares cut: a warp per row.  CTA (x, y): boundary between shares x and x + 1, member of
// the group and rows.  O = sum_s w_s O_s / sum_s w_s with w_s the sum of a part's rounded weights (its O_s is divided
// by that), LSE from the sums of the fp32 weights.
constexpr int kLatJoinThreads = 256;
template <bool BF16>
__global__ void __launch_bounds__(kLatJoinThreads) latent_join_kernel(const LatentParams p) {
    dependents_may_start();
    wait_for_previous();
    const int groups = static_cast<int>(gridDim.x) + 1, i = blockIdx.x + 1, lane = threadIdx.x & 31;
    const int4 unit = ld(p.shares + i);
    const int share = ld(p.shares + groups).x;
    const long long at = static_cast<long long>(i) * share;
    if (unit.x >= at || unit.y <= at || at - share > unit.x) return;  // not inside a unit, or not the first boundary inside
    // part of share i - 1 (its first unit or its last), then the first ones of the shares that begin inside
    const int parts = 1 + static_cast<int>(min(static_cast<long long>(groups - i), (unit.y - at + share - 1) / share));
    constexpr int kBlocks = kLatRows / (kLatJoinThreads / 32);
    const int member = blockIdx.y / kBlocks;
    const int row = (blockIdx.y - member * kBlocks) * (kLatJoinThreads / 32) + (threadIdx.x >> 5);
    const int head_slot = unit.x == at - share ? 0 : 1;
    auto slot = [&](int j) {
        return ((static_cast<long long>(i - 1 + j) * p.members + member) * 2 + (j == 0 ? head_slot : 0)) * kLatRows + row;
    };
    bool bad = false;
    const LatRequest rq = lat_request(p, unit.z, bad);
    const int r = (unit.w * p.members + member) * kLatRows + row;
    if (r >= rq.nq * p.H) return;
    const int tok = rq.q0 + r / p.H, head = r % p.H;
    uint16_t* dst = p.o + static_cast<long long>(tok) * p.o_st + static_cast<long long>(head) * p.o_sh;
    for (int c0 = 0; c0 < p.C; c0 += 256) {
        const int c = c0 + lane * 8;
        float top = -INFINITY, rtop = -INFINITY, l = 0.f, rl = 0.f;
        float o[8] = {};
        for (int j0 = 0; j0 < parts; j0 += 32) {
            float2 a = make_float2(-INFINITY, -INFINITY);
            if (j0 + lane < parts) a = ld(p.stats + slot(j0 + lane));
            float next = fmaxf(a.x, top), rnext = fmaxf(a.y, rtop);
#pragma unroll
            for (int x = 16; x; x >>= 1) {
                next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, x));
                rnext = fmaxf(rnext, __shfl_xor_sync(0xffffffffu, rnext, x));
            }
            const float ref = next == -INFINITY ? 0.f : next, rref = rnext == -INFINITY ? 0.f : rnext;
            const float old = ptx::ex2_approx(rtop - rref);
            float sum = ptx::ex2_approx(a.x - ref);
            const float w = ptx::ex2_approx(a.y - rref);
            float rsum = w;
#pragma unroll
            for (int x = 16; x; x >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, x);
                rsum += __shfl_xor_sync(0xffffffffu, rsum, x);
            }
            l = fmaf(l, ptx::ex2_approx(top - ref), sum);
            rl = fmaf(rl, old, rsum);
            top = next, rtop = rnext;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= old;
            const int n = min(32, parts - j0);
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j);
                if (wj == 0.f || c >= p.C) continue;  // (a part without a key wrote no O)
                const float4* src = reinterpret_cast<const float4*>(p.o_part + slot(j0 + j) * p.C + c);
                const float4 u = ld(src), v = ld(src + 1);
                o[0] = fmaf(u.x, wj, o[0]), o[1] = fmaf(u.y, wj, o[1]), o[2] = fmaf(u.z, wj, o[2]), o[3] = fmaf(u.w, wj, o[3]);
                o[4] = fmaf(v.x, wj, o[4]), o[5] = fmaf(v.y, wj, o[5]), o[6] = fmaf(v.z, wj, o[6]), o[7] = fmaf(v.w, wj, o[7]);
            }
        }
        const float inv = rl != 0.f ? 1.f / rl : 0.f;
        if (c < p.C)
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(pack16(o[0] * inv, o[1] * inv, BF16), pack16(o[2] * inv, o[3] * inv, BF16),
                                                            pack16(o[4] * inv, o[5] * inv, BF16), pack16(o[6] * inv, o[7] * inv, BF16));
        if (c == 0) p.lse[static_cast<long long>(tok) * p.H + head] = l != 0.f ? (top + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
}

}  // namespace paged
}  // namespace fa
