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
//   * warps 9 and 10 (of the first CTA): products of tile A / B, in the order PV(k), S(k + 2) for steps k of 64 keys.  (One warp for
//     both left the tensor cores idle between a wait and the products behind it: 384 us for what takes 344 with two.)
// The way from a step's scores over its weights to the next scores (weights 1,000 cycles, the signals between two CTAs
// 300 to 450 each, the products themselves) is longer than what the tensor cores have to do for the other tile
// meanwhile.  So S is held twice, for steps of 64 keys: S(k + 1) is there before the weights of step k are done.  (Steps
// of 128 keys and one S: 4,400 cycles per 128 keys, of which the tensor cores worked 2,560.)  A step takes 1,900 cycles, of which the
// tensor cores work 1,550; the same where tile A, which sees 256 keys less, is done and B goes on alone, which is what the
// rest is lost to: 32 heads, pieces of 4000 and 2516 queries on up to 6000 keys 331 us in a graph, 1.32 PFLOP/s (350 from a cold
// L2); 8192 queries of 16 heads 245 us, 1.40 PFLOP/s.
// Weights are rounded to the operands' 16-bit type, as both operands of a product are of one; O is divided by the sum of the
// rounded ones, the LSE takes the fp32 sum.
// TMEM: S_A 0 and 64, S_B 128 and 192 (16-bit weights over the first 32 columns of each), U_A 256, U_B 384.
// Units are handed out by the launch itself: a pair that is done takes the next cluster of the grid that has not begun
// (clusterlaunchcontrol), asked for one unit ahead, so that its queries and keys are on their way before the last products of this one.
// (Dealt out in turn, the CTA with the most work had a quarter more than the average.)  They go through heads in groups
// whose keys and values stay in L2, within a group longest first.
// Requests lie behind one another, so a tile may hold the next request's keys: masked as keys; as values they
// are overwritten with zeros (weight 0 times infinity or NaN would reach this request).  The warps of one query tile do that for
// both, and both tiles' issuers wait for them: the weights of the other tile say nothing of these values.
#pragma once

#include <type_traits>

#include "pair_ptx.cuh"

namespace fa {
namespace paged {

constexpr int kLfThreads = 352;
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
    uint64_t q_full, k_full[kLfStages], v_full[kLfStages], p_full[4], unit_empty[2];   // p: by tile and step parity
    uint64_t v_ready[kLfStages];   // values of a tile with keys behind its request's last are there, zeros written
    // in both by the tensor core, by the launch control, or by the CTA's own loads
    uint64_t q_empty, k_empty[kLfStages], v_empty[kLfStages], s_full[4], o_ready[4], unit_full[2], v_last[kLfStages], drain[2];
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
    int na, nb;    // steps of 64 keys that tile A, B sees
    int steps, tiles;  // the larger; in key tiles of 128
    __device__ int n(int x) const { return x ? nb : na; }
    // whether step k is the first of a key tile with keys behind the request's last (the last tile alone can be one)
    __device__ bool ends_at(int k) const { return k == 2 * (tiles - 1) && 128 * tiles > nk; }
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
    auto steps_of = [&](int i0) {
        const int last = min(i0 + 255, w.nq - 1), limit = p.causal ? min(w.nk, last + 1 + w.nk - w.nq) : w.nk;
        return w.row0 < 0 || i0 >= w.nq ? 0 : (max(limit, 0) + 63) / 64;
    };
    w.na = steps_of(w.row0), w.nb = steps_of(w.row0 + 256);
    w.steps = max(w.na, w.nb), w.tiles = (w.steps + 1) / 2;
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
    const uint32_t b_sf = ptx::smem_addr(&ctl->s_full[0]), b_pf = ptx::smem_addr(&ctl->p_full[0]);
    const uint32_t b_vl = ptx::smem_addr(&ctl->v_last[0]), b_or = ptx::smem_addr(&ctl->o_ready[0]), b_drain = ptx::smem_addr(&ctl->drain[0]);
    const uint32_t b_vr = ptx::smem_addr(&ctl->v_ready[0]);
    const uint32_t b_uf = ptx::smem_addr(&ctl->unit_full[0]), b_ue = ptx::smem_addr(&ctl->unit_empty[0]);
    const uint32_t answers = ptx::smem_addr(&ctl->unit[0]);
    constexpr int kReaders = 2 * 9 + 2;  // warps that take a unit from an answer: softmax and loader of both, the issuers
    if (tid == 0) {
        ptx::mbar_init(b_q, 2);
        ptx::mbar_init(b_qe, 2);
        for (int s = 0; s < kLfStages; ++s) {
            ptx::mbar_init(b_kf + 8 * s, 2);
            ptx::mbar_init(b_ke + 8 * s, 2);
            ptx::mbar_init(b_vf + 8 * s, 2);
            ptx::mbar_init(b_ve + 8 * s, 2);
            ptx::mbar_init(b_vl + 8 * s, 1);
            ptx::mbar_init(b_vr + 8 * s, 8);
        }
        for (int x = 0; x < 2; ++x) {
            for (int k = 2 * x; k < 2 * x + 2; ++k) {
                ptx::mbar_init(b_sf + 8 * k, 1);
                ptx::mbar_init(b_pf + 8 * k, 8);
                ptx::mbar_init(b_or + 8 * k, 1);
            }
            ptx::mbar_init(b_uf + 8 * x, 1);
            ptx::mbar_init(b_drain + 8 * x, 1);
            ptx::mbar_init(b_ue + 8 * x, kReaders);
        }
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
        ptx::fence_proxy_async_smem();  // (read before the launch control, asked by the first CTA, writes there again)
        __syncwarp();
        if (lane == 0) arrive_remote_release(r_ue + 8 * s);
        return u;
    };
    const int first_unit = static_cast<int>(blockIdx.x >> 1);

    if (warp == 8) {
        // =============================================================== loader
        const uint32_t r_q = in_first_cta(b_q), r_kf = in_first_cta(b_kf), r_vf = in_first_cta(b_vf);
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
            if (w.steps > 0) {
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
                        for (int h = 0; h < 2; ++h) {  // its half of each step's keys
                            const int key = w.k0 + 128 * j + 64 * h + 32 * rank;
                            const uint32_t to = stage + h * (kLfKPiece / 2);
                            for (int d = 0; d + 1 < KP; ++d) tma_load_4d_pair(to + d * kLfKPiece, &tm_k, r_kf + 8 * s, 64 * d, key, w.head, 0);
                            tma_load_4d_pair(to + (KP - 1) * kLfKPiece, &tm_s, r_kf + 8 * s, 0, key, 0, 0);
                        }
                    }
                    __syncwarp();
                    if (wrap > 0 && !(ok = wait_warp(b_ve + 8 * s, (wrap - 1) & 1))) break;
                    const uint32_t to = stage + kLfMaxPieces * kLfKPiece;
                    if (lane == 0) {
                        if (128 * (j + 1) > w.nk) {  // softmax warps wait for it and write zeros into it: v_ready says that it is there
                            ptx::mbar_arrive_expect_tx(b_vl + 8 * s, kLfVTile);
                            ptx::tma_load_4d(to, &tm_v, b_vl + 8 * s, p.half_v * rank, w.k0 + 128 * j, w.head, 0);
                            arrive_remote(r_vf + 8 * s);
                        } else {
                            arrive_remote_expect(r_vf + 8 * s, kLfVTile);
                            tma_load_4d_pair(to, &tm_v, r_vf + 8 * s, p.half_v * rank, w.k0 + 128 * j, w.head, 0);
                        }
                    }
                    __syncwarp();
                    if (++s == kLfStages) s = 0, ++wrap;
                }
                if (!ok) break;
            }
            u = unit_after(i);
        }
        // (everything that was loaded was read by products, or waited for, before the pair ends)
    } else if (warp == 9 || warp == 10) {
        // ============================================ tensor-core issuer of tile x
        if (rank == 0) {
            const int x = warp - 9;
            const uint32_t types = BF16 ? (1u << 7) | (1u << 10) : 0u;
            const uint32_t idesc_s = pr_instr(256, 64, false) | types, idesc_pv = pr_instr(256, 2 * p.half_v, true) | types;
            const uint64_t qd = pr_desc(sbase + x * kLfMaxPieces * kLfQPiece, 16, 1024);
            const uint64_t k_desc = pr_desc(sbase + kLfOffK, 16, 1024), v_desc = pr_desc(sbase + kLfOffK + kLfMaxPieces * kLfKPiece, 16, 1024);
            const uint32_t s_cols = tmem + x * 128, u_cols = tmem + 256 + x * 128, bars = 16 * x;
            // of the key tile that S is at, and of the value tile: stage, parity, descriptor
            int sk = 0, sv = 0;
            uint32_t wk = 0, wv = 0, n = 0;   // n: steps so far
            uint64_t kd = k_desc, vd = v_desc;
            uint32_t ready_phase = 0;  // bit s: parity of the next tile in stage s that v_ready speaks of
            int units = 0;
            bool ok = true;
            // S of the unit's step s.  Key and value tiles are passed on by both issuers, by the one whose tile does
            // not see them too.
            auto issue_s = [&](int s, int mine, int steps) {
                if (!(s & 1) && !wait_pair_lean(b_kf + 8 * sk, wk)) return false;
                if (s < mine) {
                    ptx::tc_fence_after_sync();
                    const uint32_t odd = (n + s) & 1;
                    const uint64_t b = kd + (s & 1) * (kLfKPiece / 32);
                    if (KP == 3) {
                        mma_pair_k192(s_cols + 64 * odd, qd, b, idesc_s);
                    } else {
                        for (int c = 0; c < KP; ++c) mma_pair_k64(s_cols + 64 * odd, qd + c * (kLfQPiece / 16), b + c * (kLfKPiece / 16), idesc_s, c > 0);
                    }
                    commit_pair(b_sf + bars + 8 * odd);
                }
                if ((s & 1) || s + 1 == steps) {
                    commit_pair(b_ke + 8 * sk);
                    kd += kLfStage / 16;
                    if (++sk == kLfStages) sk = 0, wk ^= 1, kd = k_desc;
                }
                if (s + 1 == steps) commit_pair(b_qe);
                return true;
            };
            int u = first_unit;
            for (int i = 0; ok && u >= 0; ++i) {
                bool bad = false;
                const LfUnit w = lf_unit(p, ctl, u, bad);
                const int mine = w.n(x), steps = w.steps;
                if (steps > 0) {
                    if (!(ok = wait_pair_lean(b_q, units & 1))) break;
                    ++units;
                    ptx::tc_fence_after_sync();
                    // (S overwrites columns that were read, and weights whose product was issued, before)
                    for (int s = 0; ok && s < min(2, steps); ++s) ok = issue_s(s, mine, steps);
                    for (int k = 0; ok && k < steps; ++k) {
                        if (!(k & 1)) {
                            if (!(ok = wait_pair_lean(b_vf + 8 * sv, wv))) break;
                            if (w.ends_at(k)) {
                                if (!(ok = wait_pair_lean(b_vr + 8 * sv, (ready_phase >> sv) & 1))) break;
                                ready_phase ^= 1u << sv;
                            }
                        }
                        if (k < mine) {
                            const uint32_t odd = (n + k) & 1;
                            if (!(ok = wait_pair_lean(b_pf + bars + 8 * odd, ((n + k) >> 1) & 1))) break;
                            ptx::tc_fence_after_sync();
                            mma_pair_ts_k64(u_cols, s_cols + 64 * odd, vd + (k & 1) * (64 * 128 / 16), idesc_pv, k > 0);
                            commit_pair(b_or + bars + 8 * odd);
                        }
                        if ((k & 1) || k + 1 == steps) {
                            commit_pair(b_ve + 8 * sv);
                            vd += kLfStage / 16;
                            if (++sv == kLfStages) sv = 0, wv ^= 1, vd = v_desc;
                        }
                        if (k + 2 < steps) ok = issue_s(k + 2, mine, steps);
                    }
                    n += mine;
                }
                if (ok) u = unit_after(i);
            }
            __syncwarp();
            // nothing of the pair may still run on the tensor cores when it ends
            commit_pair_here(b_drain + 8 * x);
            __syncwarp();
            wait_warp(b_drain + 8 * x, 0);
        }
    } else if (warp < 8) {
        // ================================================= softmax of tile x
        const int x = warp >> 2, t = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t u_addr = tmem + lane_off + 256 + x * 128;
        const float c2 = p.scale_log2;
        const float2 c2v = make_float2(c2, c2);
        constexpr float kLimit = BF16 ? 4294967296.f : 32768.f;  // keeps every weight inside the 16-bit type
        // Weights in fp16 are 2^7 times as large: they keep 11 bits down to 2^-21 of the reference, and only below 2^-32 of it are
        // they lost (100,000 keys of 2^-25 would be 0.3% of a row; as many of 2^-32 are 2^-15).
        constexpr float kShift = BF16 ? 0.f : 7.f;
        uint32_t n = 0;          // steps of this query tile so far
        int s0 = 0;              // stage of the unit's first key tile
        uint32_t last_phase = 0; // bit s: parity of the next tile in stage s with keys behind its request's last
        bool ok = true;
        int u = first_unit;
        for (int i = 0; ok && u >= 0; ++i) {
            bool bad = false;
            const LfUnit w = lf_unit(p, ctl, u, bad);
            if (bad && tid == 0) report(kBadData);
            const int first_row = w.row0 + 256 * x + 128 * rank, row = first_row + t, T = w.n(x), offset = w.nk - w.nq;
            const bool mine = w.row0 >= 0 && row < w.nq;
            float ref = -INFINITY;                    // reference of the raw scores
            float sum = 0.f, rsum = 0.f;              // of the fp32 and of the rounded weights
            for (int k = 0; k < T; ++k, ++n) {
                const uint32_t at = 16 * x + 8 * (n & 1), s_addr = tmem + lane_off + x * 128 + 64 * (n & 1);
                const int key0 = 64 * k;
                // Values of keys behind the request's last: zeros, for both query tiles, by A's warps where A sees the step; done while
                // the scores are on their way (behind the weights short prompts take 12.9 us in a graph, here 11.9).
                if (w.ends_at(k) && x == (w.na > k ? 0 : 1)) {
                    const int st = (s0 + k / 2) % kLfStages;
                    if (!(ok = wait_warp(b_vl + 8 * st, (last_phase >> st) & 1))) break;
                    const uint32_t tile = sbase + kLfOffK + st * kLfStage + kLfMaxPieces * kLfKPiece;
                    for (int c = (w.nk - key0) * 8 + t; c < 128 * 8; c += 128)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + c * 16), "r"(0) : "memory");
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_remote_release(in_first_cta(b_vr + 8 * st));
                }
                if (!(ok = wait_warp(b_sf + at, (n >> 1) & 1))) break;
                ptx::tc_fence_after_sync();
                const bool masked = key0 + 64 > w.nk || (p.causal && key0 + 63 > first_row + offset);
                const int seen = (p.causal ? min(w.nk, row + offset + 1) : w.nk) - key0;
                auto load = [&](uint32_t(&sv)[64]) {
                    ptx::tmem_ld_32x32b_x64(s_addr, sv);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 64; ++e) ptx::reg_fence(sv[e]);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (e >= seen) sv[e] = __float_as_uint(-INFINITY);
                    }
                };
                uint32_t sv[64], pk[32];
                float2 s, rs;
                // weights 2^(c2 (x - ref) + kShift), their sum and the sum of the rounded ones
                auto weigh = [&] {
                    const float nr = ref == -INFINITY ? 0.f : fmaf(-ref, c2, kShift);
                    const float2 nv = make_float2(nr, nr);
                    float2 a[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, b[2] = {a[0], a[0]};
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), c2v, nv);
                        const float2 wt = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
                        a[e & 1] = __fadd2_rn(a[e & 1], wt);
                        pk[e] = pack16(wt.x, wt.y, BF16);
                        b[e & 1] = __fadd2_rn(b[e & 1], unpack16(pk[e], BF16));
                    }
                    s = __fadd2_rn(a[0], a[1]), rs = __fadd2_rn(b[0], b[1]);
                };
                load(sv);
                bool moved = __any_sync(0xffffffffu, ref == -INFINITY);
                if (!moved) {
                    weigh();
                    // (all weights are positive: their sum bounds each)
                    moved = __any_sync(0xffffffffu, s.x + s.y > kLimit);
                }
                if (moved) {
                    // The step's maximum becomes the reference; U, which holds the steps before once the last product is done, is
                    // rescaled.
                    load(sv);
                    float top = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 64; e += 2) top = ptx::fmax3(top, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                    float alpha = 1.f;
                    if (top > ref) {
                        if (ref != -INFINITY) alpha = ptx::ex2_approx((ref - top) * c2);
                        ref = top;
                    }
                    weigh();
                    if (k > 0) {
                        if (!(ok = wait_warp(b_or + 16 * x + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1))) break;
                        ptx::tc_fence_after_sync();
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
                    }
                    sum *= alpha, rsum *= alpha;
                }
                ptx::tmem_st_32x32b_x32(s_addr, pk);
                sum += s.x + s.y, rsum += rs.x + rs.y;
                ptx::tmem_wait_st();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_remote(in_first_cta(b_pf + at));
            }
            // ---- O = U / sum
            if (ok && T > 0) ok = wait_warp(b_or + 16 * x + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1);
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
                    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(ov[e + k]) * inv;
                    *reinterpret_cast<uint4*>(dst + c + e) =
                        make_uint4(pack16(f[0], f[1], BF16), pack16(f[2], f[3], BF16), pack16(f[4], f[5], BF16), pack16(f[6], f[7], BF16));
                }
                __syncwarp();
            }
            if (mine)
                p.lse[tok * p.H + w.head] = sum != 0.f ? (ref * c2 + (log2f(sum) - kShift)) * 0.69314718055994531f : -INFINITY;
            ptx::tc_fence_before_sync();  // (U is overwritten behind this thread's next weights)
            if (w.tiles > 0 && 128 * w.tiles > w.nk) last_phase ^= 1u << (s0 + w.tiles - 1) % kLfStages;
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
