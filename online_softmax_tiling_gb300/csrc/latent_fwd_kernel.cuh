// latent_fwd_kernel.cuh - latent attention in its expanded form: prompts of ragged requests, keys of Dn channels per
// head and R more that all heads share, values of Dv channels.
//
//   x_ij = scale (q_i[:Dn] . k_j + q_i[Dn:] . shared_j),  O_i = softmax(x_i) V,   Dn, Dv <= 128, R <= 64
//
// 2 (Dn + R + Dv) operations per visible pair: bound by the tensor cores.  The shared channels are one more
// 64-channel piece of the first product's depth, read from the one copy there is (never laid out per head).
//
// Mapping.  A unit is 512 query rows of one (request, head), two tiles A and B of 256, on a pair of CTAs: tcgen05.mma of both
// (cta_group::2, M = 256), each CTA with 128 rows of a tile and half of every B operand: 64 keys of a key tile of 128 for
// S = Q K^T, half of the value channels (of all keys) for U += P V.  With a depth of 192 the queries take 96 KB; key
// and value halves are 40 KB a tile, so three tiles fit beside them (one CTA alone: one and a half), and per product
// shared memory is read 96 bytes a cycle instead of 128, which left nothing for the loads (75 cycles a step instead of 64).
//   * warps 0-3 / 4-7: softmax of the CTA's rows of tile A / B, a thread per row; weights go to tensor memory;
//   * warp 8: loads (TMA) and the next unit;
//   * warp 9 (of the first CTA): products in the order PV_A(j), S_A(j + 1), PV_B(j), S_B(j + 1), each PV in two
//     halves of 64 keys: while one tile's weights are computed, the tensor cores work for the other.
// TMEM: S_A 0, S_B 128 (16-bit weights over the first 64 columns), U_A 256, U_B 384.
// Units are handed out by the launch itself: a pair that is done takes the next cluster of the grid that has not begun
// (clusterlaunchcontrol), asked for one unit ahead, so that its queries and keys are on their way before the last products of this one.
// (Dealt out in turn, the CTA with the most work had a quarter more than the average.)  They go through heads in groups
// whose keys and values stay in L2, within a group longest first.
// Requests lie behind one another, so a tile may hold the next request's keys: masked as keys; as values they
// are overwritten with zeros (weight 0 times infinity or NaN would reach this request).
#pragma once

#include <type_traits>

#include "pair_ptx.cuh"

namespace fa {
namespace paged {

constexpr int kLfThreads = 320;
constexpr int kLfRows = 512;         // of a unit
constexpr int kLfQPiece = 128 * 128; // 128 rows x 64 channels
constexpr int kLfKPiece = 64 * 128;  // 64 keys x 64 channels
constexpr int kLfVTile = 128 * 128;  // 128 keys x up to 64 channels
constexpr int kLfMaxPieces = 3;      // 64-channel pieces of a query or key
constexpr int kLfStages = 3;
constexpr int kLfStage = kLfMaxPieces * kLfKPiece + kLfVTile;
constexpr int kLfOffK = 2 * kLfMaxPieces * kLfQPiece;
constexpr int kLfOffCtl = kLfOffK + kLfStages * kLfStage;

struct LatentFwdParams {
    uint16_t* o;
    float* lse;
    const int* cu_q;
    const int* cu_k;
    long long o_st, o_sh;
    int T, Tk, B, H, Dn, Dv, max_q;
    int pieces;        // of a key: those of its own channels, then the shared one
    int half_v;        // value channels of a CTA: a multiple of 16, at most 64
    int q_blocks;      // of 512 rows, of the longest request
    int group;         // (request, head) pairs gone through together
    int compact;       // most requests are far shorter than the longest: units by the blocks that there are
    int causal;
    float scale_log2;
};
constexpr int kLfMaxB = 2048;   // requests whose blocks are counted (compact)
struct LfCtl {
    // signalled in the first CTA by both
    uint64_t q_full, k_full[kLfStages], p_half[2], p_full[2], unit_empty[2];
    // in both by the tensor core, by the launch control, or by the CTA's own loads
    uint64_t q_empty, k_empty[kLfStages], v_empty[kLfStages], s_full[2], o_half[2], o_ready[2], unit_full[2], v_full[kLfStages], drain;
    alignas(16) uint4 unit[2];   // answers of the launch control
    uint32_t tmem_base;
    int warp_sum[kLfThreads / 32];
    int before[kLfMaxB + 1];     // compact: blocks before each request
};
constexpr int kLfSmem = kLfOffCtl + static_cast<int>(sizeof(LfCtl)) + 1024;
static_assert(kLfSmem <= 232448, "shared memory of a CTA");

struct LfUnit {
    int q0, nq, k0, nk, head;
    int row0;      // first row of the unit in its request
    int na, nb;    // key tiles that tile A, B sees
    int tiles;     // the larger
    __device__ int n(int x) const { return x ? nb : na; }
};

// Unit u: heads in groups, in a group the last block of every (request, head), then the last but one (a request that has
// fewer has none); compact: head by head the blocks of all requests, each request's from the last.
__device__ __forceinline__ LfUnit lf_unit(const LatentFwdParams& p, const LfCtl* ctl, int u, bool& bad) {
    LfUnit w;
    int b, back;
    if (p.compact) {
        const int all = max(ctl->before[p.B], 1), k = u % all;
        w.head = u / all;
        b = owner_of(ctl->before, p.B, k);
        back = w.head < p.H ? k - ctl->before[b] : p.q_blocks;  // (behind the last unit)
    } else {
        const int heads = p.B * p.H, per = p.group * p.q_blocks, g = u / per, rest = u - g * per;
        const int here = min(p.group, heads - g * p.group), bh = g * p.group + rest % here;
        back = rest / here;
        b = bh / p.H;
        w.head = bh - b * p.H;
    }
    w.q0 = ld_meta(p.cu_q + b), w.k0 = ld_meta(p.cu_k + b);
    w.nq = ld_meta(p.cu_q + b + 1) - w.q0, w.nk = ld_meta(p.cu_k + b + 1) - w.k0;
    if (w.q0 < 0 || w.nq < 0 || w.nq > p.max_q || w.q0 > p.T - w.nq || w.k0 < 0 || w.nk < 0 || w.k0 > p.Tk - w.nk)
        bad = true, w.nq = 0;
    w.row0 = ((w.nq + kLfRows - 1) / kLfRows - 1 - back) * kLfRows;  // (the last block, with the most keys, first; negative: none)
    auto tiles_of = [&](int i0) {
        const int last = min(i0 + 255, w.nq - 1), limit = p.causal ? min(w.nk, last + 1 + w.nk - w.nq) : w.nk;
        return w.row0 < 0 || i0 >= w.nq ? 0 : (max(limit, 0) + 127) / 128;
    };
    w.na = tiles_of(w.row0), w.nb = tiles_of(w.row0 + 256);
    w.tiles = max(w.na, w.nb);
    return w;
}

// Asks for the next cluster of the grid: 16 bytes at `answer` of both CTAs, signalled on `bar` of both.
__device__ __forceinline__ void ask_unit(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], [%1];" ::"r"(answer),
                 "r"(bar)
                 : "memory");
}
// The unit of an answer, -1 where there is none any more.
__device__ __forceinline__ int answered_unit(uint32_t answer) {
    uint32_t yes, x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
        : "=r"(yes), "=r"(x)
        : "r"(answer)
        : "memory");
    return yes ? static_cast<int>(x >> 1) : -1;
}

template <bool BF16>
__global__ void __launch_bounds__(kLfThreads, 1)
    latent_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_s, const __grid_constant__ CUtensorMap tm_v, const LatentFwdParams p) {
    extern __shared__ __align__(16) uint8_t lf_raw[];
    const uint32_t raw = ptx::smem_addr(lf_raw);
    uint8_t* smem = lf_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = ptx::smem_addr(smem);
    LfCtl* ctl = reinterpret_cast<LfCtl*>(smem + kLfOffCtl);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_rank());
    const int KP = p.pieces;

    const uint32_t b_q = ptx::smem_addr(&ctl->q_full), b_qe = ptx::smem_addr(&ctl->q_empty);
    const uint32_t b_kf = ptx::smem_addr(&ctl->k_full[0]), b_ke = ptx::smem_addr(&ctl->k_empty[0]);
    const uint32_t b_vf = ptx::smem_addr(&ctl->v_full[0]), b_ve = ptx::smem_addr(&ctl->v_empty[0]);
    const uint32_t b_sf = ptx::smem_addr(&ctl->s_full[0]), b_ph = ptx::smem_addr(&ctl->p_half[0]), b_pf = ptx::smem_addr(&ctl->p_full[0]);
    const uint32_t b_oh = ptx::smem_addr(&ctl->o_half[0]), b_or = ptx::smem_addr(&ctl->o_ready[0]), b_drain = ptx::smem_addr(&ctl->drain);
    const uint32_t b_uf = ptx::smem_addr(&ctl->unit_full[0]), b_ue = ptx::smem_addr(&ctl->unit_empty[0]);
    const uint32_t answers = ptx::smem_addr(&ctl->unit[0]);
    constexpr int kReaders = 2 * 9 + 1;  // warps that take a unit from an answer: softmax and loader of both, the issuer
    if (tid == 0) {
        ptx::mbar_init(b_q, 2);
        ptx::mbar_init(b_qe, 1);
        for (int s = 0; s < kLfStages; ++s) {
            ptx::mbar_init(b_kf + 8 * s, 2);
            ptx::mbar_init(b_ke + 8 * s, 1);
            ptx::mbar_init(b_vf + 8 * s, 1);
            ptx::mbar_init(b_ve + 8 * s, 1);
        }
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(b_sf + 8 * x, 1);
            ptx::mbar_init(b_ph + 8 * x, 8);
            ptx::mbar_init(b_pf + 8 * x, 8);
            ptx::mbar_init(b_oh + 8 * x, 1);
            ptx::mbar_init(b_or + 8 * x, 1);
            ptx::mbar_init(b_uf + 8 * x, 1);
            ptx::mbar_init(b_ue + 8 * x, kReaders);
        }
        ptx::mbar_init(b_drain, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_s);
        ptx::prefetch_tensormap(&tm_v);
    }
    if (warp == 9) tmem_alloc_pair(ptx::smem_addr(&ctl->tmem_base));
    ptx::tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // barriers and tensor memory of both CTAs are there
    ptx::tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    dependents_may_start();
    wait_for_previous();
    if (p.compact) {
        const int per = (p.B + kLfThreads - 1) / kLfThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
        auto blocks_of = [&](int b) {
            const int q0 = ld_meta(p.cu_q + b), nq = ld_meta(p.cu_q + b + 1) - q0;
            return nq < 0 || nq > p.max_q || q0 < 0 || q0 > p.T - nq ? 1 : (nq + kLfRows - 1) / kLfRows;  // (bad marks: a unit to report them)
        };
        int own = 0;
        for (int b = b0; b < b1; ++b) own += blocks_of(b);
        int incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) ctl->warp_sum[warp] = incl;
        __syncthreads();
        int run = incl - own;
        for (int i = 0; i < warp; ++i) run += ctl->warp_sum[i];
        for (int b = b0; b < b1; ++b) {
            ctl->before[b] = run;
            run += blocks_of(b);
        }
        if (b0 < b1 && b1 == p.B) ctl->before[p.B] = run;
        __syncthreads();
    }

    // The unit behind a role's i-th (the first is the pair's own); -1: none, or the wait ran out.
    const uint32_t r_ue = in_first_cta(b_ue);
    auto unit_after = [&](int i) {
        const int s = i & 1;
        if (!wait_pair(b_uf + 8 * s, (i >> 1) & 1)) return -1;
        const int u = answered_unit(answers + 16 * s);
        ptx::fence_proxy_async_smem();  // (read before the launch control writes there again)
        __syncwarp();
        if (lane == 0) arrive_remote(r_ue + 8 * s);
        return u;
    };
    const int first_unit = static_cast<int>(blockIdx.x >> 1);

    if (warp == 8) {
        // =============================================================== loader
        const uint32_t r_q = in_first_cta(b_q), r_kf = in_first_cta(b_kf);
        int s = 0, wrap = 0;  // stage and times round of the next key tile
        int units = 0;        // whose queries were loaded
        bool ok = true;
        int u = first_unit;
        for (int i = 0; u >= 0; ++i) {
            // the unit after this one: the answer's place is free once all have read the one before last
            if (rank == 0 && i >= 2 && !(ok = wait_pair(b_ue + 8 * (i & 1), ((i >> 1) - 1) & 1))) break;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(b_uf + 8 * (i & 1), 16);
                if (rank == 0) ask_unit(answers + 16 * (i & 1), b_uf + 8 * (i & 1));
            }
            __syncwarp();
            bool bad = false;
            const LfUnit w = lf_unit(p, ctl, u, bad);
            if (w.tiles > 0) {
                if (units > 0 && !(ok = wait_warp(b_qe, (units - 1) & 1))) break;
                const int tiles_q = w.nb > 0 ? 2 : 1;
                if (lane == 0) {
                    arrive_remote_expect(r_q, tiles_q * KP * kLfQPiece);
                    for (int x = 0; x < tiles_q; ++x)
                        for (int d = 0; d < KP; ++d)
                            tma_load_4d_pair(sbase + (x * kLfMaxPieces + d) * kLfQPiece, &tm_q, r_q, d + 1 < KP ? 64 * d : p.Dn,
                                             w.q0 + w.row0 + 256 * x + 128 * rank, w.head, 0);
                }
                ++units;
                for (int j = 0; j < w.tiles; ++j) {
                    const uint32_t stage = sbase + kLfOffK + s * kLfStage;
                    if (wrap > 0 && !(ok = wait_warp(b_ke + 8 * s, (wrap - 1) & 1))) break;
                    if (lane == 0) {
                        arrive_remote_expect(r_kf + 8 * s, KP * kLfKPiece);
                        const int key = w.k0 + 128 * j + 64 * rank;
                        for (int d = 0; d + 1 < KP; ++d) tma_load_4d_pair(stage + d * kLfKPiece, &tm_k, r_kf + 8 * s, 64 * d, key, w.head, 0);
                        tma_load_4d_pair(stage + (KP - 1) * kLfKPiece, &tm_s, r_kf + 8 * s, 0, key, 0, 0);
                    }
                    __syncwarp();
                    if (wrap > 0 && !(ok = wait_warp(b_ve + 8 * s, (wrap - 1) & 1))) break;
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(b_vf + 8 * s, kLfVTile);
                        ptx::tma_load_4d(stage + kLfMaxPieces * kLfKPiece, &tm_v, b_vf + 8 * s, p.half_v * rank, w.k0 + 128 * j, w.head, 0);
                    }
                    __syncwarp();
                    if (++s == kLfStages) s = 0, ++wrap;
                }
                if (!ok) break;
            }
            u = unit_after(i);
        }
        // nothing may still be landing in this CTA's memory when it ends (queries and keys were read by products that are done)
        for (int n = 0; n < kLfStages; ++n) {
            if (--s < 0) s = kLfStages - 1, --wrap;
            if (wrap >= 0) wait_warp(b_vf + 8 * s, wrap & 1);
        }
    } else if (warp == 9) {
        // ====================================================== tensor-core issuer
        if (rank == 0) {
            const uint32_t types = BF16 ? (1u << 7) | (1u << 10) : 0u;
            const uint32_t idesc_s = pr_instr(256, 128, false) | types, idesc_pv = pr_instr(256, 2 * p.half_v, true) | types;
            const uint64_t q_desc = pr_desc(sbase, 16, 1024), k_desc = pr_desc(sbase + kLfOffK, 16, 1024);
            const uint64_t v_desc = pr_desc(sbase + kLfOffK + kLfMaxPieces * kLfKPiece, 16, 1024);
            int sk = 0, wk = 0, sv = 0;  // stage (and times round) of the next key tile; stage of the next value tile
            uint32_t done[2] = {0, 0};   // key tiles of tile A, B so far
            int units = 0;
            bool ok = true;
            auto issue_s = [&](int x, int s, bool last) {
                for (int d = 0; d < KP; ++d)
                    mma_pair_k64(tmem + x * 128, q_desc + (x * kLfMaxPieces + d) * (kLfQPiece / 16), k_desc + s * (kLfStage / 16) + d * (kLfKPiece / 16),
                                 idesc_s, d > 0);
                commit_pair(b_sf + 8 * x);
                if (last) commit_pair(b_ke + 8 * s);
            };
            auto issue_pv = [&](int x, bool last, bool accumulate) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!wait_pair((h ? b_pf : b_ph) + 8 * x, done[x] & 1)) return false;
                    ptx::tc_fence_after_sync();
                    mma_pair_ts_k64(tmem + 256 + x * 128, tmem + x * 128 + 32 * h, v_desc + sv * (kLfStage / 16) + h * 512, idesc_pv, accumulate || h > 0);
                    commit_pair((h ? b_or : b_oh) + 8 * x);
                }
                if (last) commit_pair(b_ve + 8 * sv);
                ++done[x];
                return true;
            };
            int u = first_unit;
            for (int i = 0; ok && u >= 0; ++i) {
                bool bad = false;
                const LfUnit w = lf_unit(p, ctl, u, bad);
                if (w.tiles > 0) {
                    if (!(ok = wait_pair(b_q, units & 1) && wait_pair(b_kf + 8 * sk, wk & 1))) break;
                    ++units;
                    ptx::tc_fence_after_sync();
                    // (S_x overwrites columns that were read before the last weights of the unit before were handed over)
                    if (w.na > 0) issue_s(0, sk, w.nb == 0);
                    if (w.nb > 0) issue_s(1, sk, true);
                    if (w.tiles == 1) commit_pair(b_qe);
                    if (++sk == kLfStages) sk = 0, ++wk;
                    for (int j = 0; ok && j < w.tiles; ++j) {
                        bool k_ready = false;
                        for (int x = 0; ok && x < 2; ++x) {
                            if (j < w.n(x)) ok = issue_pv(x, x == 1 || w.nb <= j, j > 0);
                            if (ok && j + 1 < w.n(x)) {
                                if (!k_ready && !(ok = wait_pair(b_kf + 8 * sk, wk & 1))) break;
                                k_ready = true;
                                ptx::tc_fence_after_sync();
                                const bool last = x == 1 || w.nb <= j + 1;
                                issue_s(x, sk, last);
                                if (j + 2 == w.tiles && last) commit_pair(b_qe);
                            }
                            __syncwarp();
                        }
                        if (++sv == kLfStages) sv = 0;
                        if (j + 1 < w.tiles && ++sk == kLfStages) sk = 0, ++wk;
                    }
                }
                if (ok) u = unit_after(i);
            }
            // nothing of the pair may still run on the tensor cores when it ends
            commit_pair_here(b_drain);
            __syncwarp();
            wait_warp(b_drain, 0);
        }
    } else {
        // ================================================= softmax of tile x
        const int x = warp >> 2, t = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_off + x * 128, u_addr = tmem + lane_off + 256 + x * 128;
        const float c2 = p.scale_log2;
        const float2 c2v = make_float2(c2, c2);
        const uint32_t r_ph = in_first_cta(b_ph + 8 * x), r_pf = in_first_cta(b_pf + 8 * x);
        constexpr float kLimit = BF16 ? 4294967296.f : 32768.f;  // keeps every weight inside the 16-bit type
        uint32_t n = 0;          // key tiles of this query tile so far
        int s0 = 0, w0 = 0;      // stage (and times round) of the unit's first key tile
        bool ok = true;
        int u = first_unit;
        for (int i = 0; ok && u >= 0; ++i) {
            bool bad = false;
            const LfUnit w = lf_unit(p, ctl, u, bad);
            if (bad && tid == 0) report(kBadData);
            const int first_row = w.row0 + 256 * x + 128 * rank, row = first_row + t, T = w.row0 < 0 ? 0 : w.n(x), offset = w.nk - w.nq;
            int sv = s0, wv = w0;  // of the key tile in work
            const bool mine = w.row0 >= 0 && row < w.nq;
            float ref = -INFINITY;                    // reference of the raw scores
            float sum = 0.f, rsum = 0.f;              // of the fp32 and of the rounded weights
            for (int j = 0; j < T; ++j, ++n) {
                if (!(ok = wait_warp(b_sf + 8 * x, n & 1))) break;
                ptx::tc_fence_after_sync();
                // (taken here so that a later wait on this tile's phase is unambiguous)
                if (j > 0 && !(ok = wait_warp(b_oh + 8 * x, (n - 1) & 1))) break;
                const int key0 = j * 128;
                const bool masked = key0 + 128 > w.nk || (p.causal && key0 + 127 > first_row + offset);
                const int seen = (p.causal ? min(w.nk, row + offset + 1) : w.nk) - key0;
                auto load = [&](auto& sv, int c) {  // scores [32 c, ...), masked
                    constexpr int N = sizeof(sv) / 4;
                    if constexpr (N == 64)
                        ptx::tmem_ld_32x32b_x64(s_addr + 32 * c, sv);
                    else
                        ptx::tmem_ld_32x32b_x32(s_addr + 32 * c, sv);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < N; ++e) ptx::reg_fence(sv[e]);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < N; ++e)
                            if (32 * c + e >= seen) sv[e] = __float_as_uint(-INFINITY);
                    }
                };
                // weights 2^(c2 x + nr) of 2 N scores, their sum and the sum of the rounded ones
                auto weigh = [&](const uint32_t* sv, auto count, float nr, uint32_t* pk, float2& s, float2& rs) {
                    const float2 nv = make_float2(nr, nr);
#pragma unroll
                    for (int e = 0; e < decltype(count)::value; ++e) {
                        const float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), c2v, nv);
                        const float2 wt = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
                        s = __fadd2_rn(s, wt);
                        pk[e] = pack16(wt.x, wt.y, BF16);
                        rs = __fadd2_rn(rs, unpack16(pk[e], BF16));
                    }
                };
                using N32 = std::integral_constant<int, 32>;
                using N16 = std::integral_constant<int, 16>;
                auto top_of = [&](int c0, int c1) {
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {
                        uint32_t sv[32];
                        load(sv, c);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) top = ptx::fmax3(top, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                    }
                    return top;
                };
                auto rescale = [&](float alpha) {
                    const float2 av = make_float2(alpha, alpha);
#pragma unroll 1
                    for (int c = 0; c < 2 * p.half_v; c += 16) {
                        uint32_t ov[16];
                        ptx::tmem_ld_32x32b_x16(u_addr + c, ov);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            ptx::reg_fence(ov[e]);
                            ptx::reg_fence(ov[e + 1]);
                            const float2 y = __fmul2_rn(make_float2(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])), av);
                            ov[e] = __float_as_uint(y.x), ov[e + 1] = __float_as_uint(y.y);
                        }
                        ptx::tmem_st_32x32b_x16(u_addr + c, ov);
                    }
                    ptx::tmem_wait_st();
                };
                // this CTA's half of the values is there; those of keys behind the request's last are zeros (written by tile
                // A's warps where A sees the tile)
                if (!(ok = wait_warp(b_vf + 8 * sv, wv & 1))) break;
                const bool zeroed = key0 + 128 > w.nk && (x == 0 || w.na <= j);
                if (zeroed) {
                    const uint32_t tile = sbase + kLfOffK + sv * kLfStage + kLfMaxPieces * kLfKPiece;
                    for (int c = (w.nk - key0) * 8 + t; c < 1024; c += 128)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + c * 16), "r"(0) : "memory");
                    ptx::fence_proxy_async_smem();
                }
                auto hand_over = [&](uint32_t bar) {
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if (zeroed) arrive_remote_release(bar); else arrive_remote(bar);
                    }
                };
                uint32_t pk[32];
                float2 s = make_float2(0.f, 0.f), rs = make_float2(0.f, 0.f);
                bool moved = __any_sync(0xffffffffu, ref == -INFINITY);
                if (!moved) {
                    uint32_t sv[64];
                    load(sv, 0);
                    weigh(sv, N32{}, -ref * c2, pk, s, rs);
                    moved = __any_sync(0xffffffffu, s.x + s.y > kLimit);
                }
                if (moved) {
                    // the tile's maximum; U holds the tiles before (S(j) was issued behind them)
                    const float top = top_of(0, 4);
                    float alpha = 1.f;
                    if (top > ref) {
                        if (ref != -INFINITY) alpha = ptx::ex2_approx((ref - top) * c2);
                        ref = top;
                    }
                    if (j > 0) rescale(alpha);
                    sum *= alpha, rsum *= alpha;
                    s = rs = make_float2(0.f, 0.f);
                    uint32_t sv[64];
                    load(sv, 0);
                    weigh(sv, N32{}, ref == -INFINITY ? 0.f : -ref * c2, pk, s, rs);
                }
                ptx::tmem_st_32x32b_x32(s_addr, pk);
                hand_over(r_ph);
                sum += s.x + s.y, rsum += rs.x + rs.y;
                s = rs = make_float2(0.f, 0.f);
                {
                    uint32_t sv[64];
                    load(sv, 2);
                    weigh(sv, N32{}, ref == -INFINITY ? 0.f : -ref * c2, pk, s, rs);
                }
                if (__any_sync(0xffffffffu, s.x + s.y > kLimit)) {
                    // the first half's weights are under way: U takes them in first
                    const float top = top_of(2, 4);
                    float alpha = 1.f;
                    if (top > ref) {
                        if (ref != -INFINITY) alpha = ptx::ex2_approx((ref - top) * c2);
                        ref = top;
                    }
                    if (!(ok = wait_warp(b_oh + 8 * x, n & 1))) break;
                    ptx::tc_fence_after_sync();
                    rescale(alpha);
                    sum *= alpha, rsum *= alpha;
                    s = rs = make_float2(0.f, 0.f);
#pragma unroll
                    for (int c = 2; c < 4; ++c) {
                        uint32_t sv[32];
                        load(sv, c);
                        weigh(sv, N16{}, ref == -INFINITY ? 0.f : -ref * c2, pk + 16 * (c - 2), s, rs);
                    }
                }
                ptx::tmem_st_32x32b_x32(s_addr + 32, pk);
                hand_over(r_pf);
                sum += s.x + s.y, rsum += rs.x + rs.y;
                if (++sv == kLfStages) sv = 0, ++wv;
            }
            // ---- O = U / sum
            if (ok && T > 0) ok = wait_warp(b_or + 8 * x, (n - 1) & 1);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            const float inv = rsum != 0.f ? 1.f / rsum : 0.f;
            const long long tok = w.q0 + row;
            uint16_t* dst = p.o + tok * p.o_st + static_cast<long long>(w.head) * p.o_sh;
#pragma unroll 1
            for (int c = 0; c < 2 * p.half_v; c += 32) {
                uint32_t ov[32];
                if (T > 0) {
                    ptx::tmem_ld_32x32b_x32(u_addr + c, ov);
                    ptx::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    if (T > 0) ptx::reg_fence(ov[e]); else ov[e] = 0;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    if (!mine || c + e >= p.Dv) continue;
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(ov[e + i]) * inv;
                    *reinterpret_cast<uint4*>(dst + c + e) =
                        make_uint4(pack16(f[0], f[1], BF16), pack16(f[2], f[3], BF16), pack16(f[4], f[5], BF16), pack16(f[6], f[7], BF16));
                }
                __syncwarp();
            }
            if (mine)
                p.lse[tok * p.H + w.head] = sum != 0.f ? (ref * c2 + log2f(sum)) * 0.69314718055994531f : -INFINITY;
            ptx::tc_fence_before_sync();  // (U is overwritten behind this thread's next weights)
            w0 += (s0 + w.tiles) / kLfStages;
            s0 = (s0 + w.tiles) % kLfStages;
            u = unit_after(i);
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA's memory is written or read by the other any more
    if (warp == 9) {
        ptx::tc_fence_after_sync();
        tmem_dealloc_pair(tmem);
    }
}

}  // namespace paged
}  // namespace fa
