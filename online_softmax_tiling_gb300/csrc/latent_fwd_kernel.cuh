// latent_fwd_kernel.cuh - latent attention in its expanded form: prompts of ragged requests, keys of Dn channels per
// head and R more that all heads share, values of Dv channels.
//
//   x_ij = scale (q_i[:Dn] . k_j + q_i[Dn:] . shared_j),  O_i = softmax(x_i) V,   Dn, Dv <= 128, R <= 64
//
// 2 (Dn + R + Dv) operations per visible pair: bound by the tensor cores.  The shared channels are one more
// 64-channel piece of the first product's depth, read from the one copy there is (never laid out per head).
//
// Mapping: that of the fused forward kernel.  A persistent CTA per SM walks units of 256 query rows of one
// (request, head), two tiles A and B of 128: softmax of A in warps 0-3 and of B in warps 4-7 (a thread per row), loader
// warp 8, tensor-core issuer warp 9 in the order PV_A(j), S_A(j + 1), PV_B(j), S_B(j + 1), each PV in two halves of
// 64 keys.  TMEM: S_A 0, S_B 128 (16-bit weights over the first 64 columns), U_A 256, U_B 384.
// With a depth of 192 the queries take 96 KB and a key tile 48: two of them and two value tiles would not fit beside
// the queries, so keys and values share one ring of eight 16 KB slots, each with barriers of its own: a slot
// holds 64 channels of 128 keys, or 64 keys of all value channels (the half that a PV step reads), and is free as soon as
// its last product is done.
// Requests lie behind one another, so a tile may hold the next request's keys: masked as keys; as values they
// are overwritten with zeros (weight 0 times infinity or NaN would reach this request).
// Units go through heads in groups whose keys and values stay in L2, within a group longest first.
#pragma once

#include <type_traits>

#include "paged_common.cuh"

namespace fa {
namespace paged {

constexpr int kLfThreads = 320;
constexpr int kLfSlot = 128 * 128;   // 16 KB
constexpr int kLfSlots = 8;
constexpr int kLfMaxPieces = 3;      // 64-channel pieces of a query or key
constexpr int kLfOffCtl = 2 * kLfMaxPieces * kLfSlot + kLfSlots * kLfSlot;

struct LatentFwdParams {
    uint16_t* o;
    float* lse;
    const int* cu_q;
    const int* cu_k;
    long long o_st, o_sh;
    int T, Tk, B, H, Dn, Dv, max_q;
    int pieces;        // of a key: those of its own channels, then the shared one
    int wide_v;        // Dv > 64
    int q_blocks;      // of 256 rows, of the longest request
    int group;         // (request, head) pairs gone through together
    int units;
    int causal;
    float scale_log2;
};
struct LfCtl {
    uint64_t q_full, q_empty, full[kLfSlots], empty[kLfSlots], s_full[2], p_half[2], p_full[2], o_half[2], o_ready[2], drain;
    uint32_t tmem_base;
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

__device__ __forceinline__ LfUnit lf_unit(const LatentFwdParams& p, int u, bool& bad) {
    LfUnit w;
    const int heads = p.B * p.H, per = p.group * p.q_blocks, g = u / per, rest = u - g * per;
    const int here = min(p.group, heads - g * p.group), back = rest / here, bh = g * p.group + rest - back * here;
    const int b = bh / p.H;
    w.head = bh - b * p.H;
    w.q0 = ld_meta(p.cu_q + b), w.k0 = ld_meta(p.cu_k + b);
    w.nq = ld_meta(p.cu_q + b + 1) - w.q0, w.nk = ld_meta(p.cu_k + b + 1) - w.k0;
    if (w.q0 < 0 || w.nq < 0 || w.nq > p.max_q || w.q0 > p.T - w.nq || w.k0 < 0 || w.nk < 0 || w.k0 > p.Tk - w.nk)
        bad = true, w.nq = 0;
    w.row0 = ((w.nq + 255) / 256 - 1 - back) * 256;  // (the last block, with the most keys, first; negative: none)
    auto tiles_of = [&](int i0) {
        const int last = min(i0 + 127, w.nq - 1), limit = p.causal ? min(w.nk, last + 1 + w.nk - w.nq) : w.nk;
        return w.row0 < 0 || i0 >= w.nq ? 0 : (max(limit, 0) + 127) / 128;
    };
    w.na = tiles_of(w.row0), w.nb = tiles_of(w.row0 + 128);
    w.tiles = max(w.na, w.nb);
    return w;
}
// Units of a CTA: c, then 2 G - 1 - c, 2 G + c, ...
__device__ __forceinline__ int lf_unit_id(int r) {
    const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    return r * G + ((r & 1) ? G - 1 - c : c);
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
    const int KP = p.pieces, VP = p.wide_v ? 2 : 1, per_tile = KP + VP;
    const uint32_t ring = sbase + 2 * kLfMaxPieces * kLfSlot;

    const uint32_t b_q = ptx::smem_addr(&ctl->q_full), b_qe = ptx::smem_addr(&ctl->q_empty);
    const uint32_t b_full = ptx::smem_addr(&ctl->full[0]), b_empty = ptx::smem_addr(&ctl->empty[0]);
    const uint32_t b_sf = ptx::smem_addr(&ctl->s_full[0]), b_ph = ptx::smem_addr(&ctl->p_half[0]), b_pf = ptx::smem_addr(&ctl->p_full[0]);
    const uint32_t b_oh = ptx::smem_addr(&ctl->o_half[0]), b_or = ptx::smem_addr(&ctl->o_ready[0]), b_drain = ptx::smem_addr(&ctl->drain);
    if (tid == 0) {
        ptx::mbar_init(b_q, 1);
        ptx::mbar_init(b_qe, 1);
        for (int s = 0; s < kLfSlots; ++s) {
            ptx::mbar_init(b_full + 8 * s, 1);
            ptx::mbar_init(b_empty + 8 * s, 1);
        }
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(b_sf + 8 * x, 1);
            ptx::mbar_init(b_ph + 8 * x, 128);
            ptx::mbar_init(b_pf + 8 * x, 128);
            ptx::mbar_init(b_oh + 8 * x, 1);
            ptx::mbar_init(b_or + 8 * x, 1);
        }
        ptx::mbar_init(b_drain, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_s);
        ptx::prefetch_tensormap(&tm_v);
    }
    if (warp == 9) {
        ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    dependents_may_start();
    wait_for_previous();

    // Pieces in the ring, numbered from the unit's first: K(0), V(0), K(1), V(1), ...  With slots for 8 of 5 per tile V(j)
    // comes a whole tile ahead, K(j + 1) while S_B(j) and PV_A(j) run.
    auto k_piece = [&](int j) { return j * per_tile; };
    auto v_piece = [&](int j) { return j * per_tile + KP; };

    if (warp == 8) {
        // =============================================================== loader
        int n = 0;      // pieces so far
        int units = 0;  // whose queries were loaded
        bool ok = true;
        auto slot_free = [&](int i) { return i < kLfSlots || wait_warp(b_empty + 8 * (i % kLfSlots), (i / kLfSlots - 1) & 1); };
        for (int r = 0; ok; ++r) {
            const int u = lf_unit_id(r);
            if (u >= p.units) break;
            bool bad = false;
            const LfUnit w = lf_unit(p, u, bad);
            if (w.tiles == 0) continue;
            if (units > 0 && !(ok = wait_warp(b_qe, (units - 1) & 1))) break;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(b_q, (w.n(1) > 0 ? 2 : 1) * KP * kLfSlot);
                for (int x = 0; x < (w.n(1) > 0 ? 2 : 1); ++x)
                    for (int i = 0; i < KP; ++i)
                        ptx::tma_load_4d(sbase + (x * kLfMaxPieces + i) * kLfSlot, &tm_q, b_q, i + 1 < KP ? 64 * i : p.Dn,
                                         w.q0 + w.row0 + 128 * x, w.head, 0);
            }
            ++units;
            for (int j = 0; ok && j < w.tiles; ++j) {
                const int key = w.k0 + j * 128;
                for (int i = 0; i < per_tile; ++i, ++n) {
                    if (!(ok = slot_free(n))) break;
                    const uint32_t bar = b_full + 8 * (n % kLfSlots), dst = ring + (n % kLfSlots) * kLfSlot;
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(bar, kLfSlot);
                        if (i + 1 < KP) {
                            ptx::tma_load_4d(dst, &tm_k, bar, 64 * i, key, w.head, 0);
                        } else if (i < KP) {
                            ptx::tma_load_4d(dst, &tm_s, bar, 0, key, 0, 0);
                        } else {
                            // two boxes of 64 keys x 64 channels: both channel groups of a half, or both halves
                            const int h = i - KP;
                            ptx::tma_load_4d(dst, &tm_v, bar, 0, key + 64 * h, w.head, 0);
                            ptx::tma_load_4d(dst + kLfSlot / 2, &tm_v, bar, VP == 2 ? 64 : 0, key + (VP == 2 ? 64 * h : 64), w.head, 0);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        // nothing may still be landing in this CTA's memory when it ends
        if (units > 0) wait_warp(b_q, (units - 1) & 1);
        for (int i = max(0, n - kLfSlots); i < n; ++i) wait_warp(b_full + 8 * (i % kLfSlots), (i / kLfSlots) & 1);
    } else if (warp == 9) {
        // ====================================================== tensor-core issuer
        const uint32_t types = BF16 ? (1u << 7) | (1u << 10) : 0u;
        const uint32_t idesc_s = pr_instr(128, 128, false) | types, idesc_pv = pr_instr(128, 64 * VP, true) | types;
        constexpr uint64_t kStep = kLfSlot / 16;
        const uint64_t q_desc = pr_desc(sbase, 16, 1024), k_desc = pr_desc(ring, 16, 1024), v_desc = pr_desc(ring, kLfSlot / 2, 1024);
        int base = 0;        // pieces of the units before
        uint32_t done[2] = {0, 0};  // key tiles of tile A, B so far
        int units = 0;
        bool ok = true;
        auto full = [&](int i) { return wait_warp(b_full + 8 * (i % kLfSlots), (i / kLfSlots) & 1); };
        // S_x of the key tile whose first piece is i; the first product with it waits for its pieces, the last frees them
        auto issue_s = [&](int x, int i, bool first, bool last) {
            for (int d = 0; d < KP; ++d) {
                const int at = i + d;
                if (first) {
                    if (!full(at)) return false;
                    ptx::tc_fence_after_sync();
                }
                ptx::mma_ss_k64(tmem + x * 128, q_desc + (x * kLfMaxPieces + d) * kStep, k_desc + (at % kLfSlots) * kStep, idesc_s, d > 0);
                if (last) ptx::tc_commit_elect(b_empty + 8 * (at % kLfSlots));
            }
            ptx::tc_commit_elect(b_sf + 8 * x);
            return true;
        };
        auto issue_pv = [&](int x, int i, bool first, bool last, bool accumulate) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = VP == 2 ? i + h : i;
                if (first && (h == 0 || VP == 2) && !full(at)) return false;
                if (!wait_warp((h ? b_pf : b_ph) + 8 * x, done[x] & 1)) return false;
                ptx::tc_fence_after_sync();
                ptx::mma_ts_k64(tmem + 256 + x * 128, tmem + x * 128 + 32 * h,
                                v_desc + (at % kLfSlots) * kStep + (VP == 1 && h ? kStep / 2 : 0), idesc_pv, accumulate || h > 0);
                ptx::tc_commit_elect((h ? b_or : b_oh) + 8 * x);
                if (last && (h == 1 || VP == 2)) ptx::tc_commit_elect(b_empty + 8 * (at % kLfSlots));
            }
            ++done[x];
            return true;
        };
        for (int r = 0; ok; ++r) {
            const int u = lf_unit_id(r);
            if (u >= p.units) break;
            bool bad = false;
            const LfUnit w = lf_unit(p, u, bad);
            if (w.tiles == 0) continue;
            if (!(ok = wait_warp(b_q, units & 1))) break;
            ++units;
            ptx::tc_fence_after_sync();
            // (S_x overwrites columns that were read before the last weights of the unit before were handed over)
            for (int x = 0; ok && x < 2; ++x)
                if (w.n(x) > 0) ok = issue_s(x, base, x == 0 || w.n(0) == 0, x == 1 || w.n(1) == 0);
            if (w.tiles == 1) ptx::tc_commit_elect(b_qe);
            for (int j = 0; ok && j < w.tiles; ++j) {
                const int kn = base + k_piece(j + 1), vn = base + v_piece(j);
                for (int x = 0; ok && x < 2; ++x) {
                    const bool other_v = w.n(x ^ 1) > j, other_k = w.n(x ^ 1) > j + 1;
                    if (j < w.n(x)) ok = issue_pv(x, vn, x == 0 || !other_v, x == 1 || !other_v, j > 0);
                    if (ok && j + 1 < w.n(x)) {
                        ok = issue_s(x, kn, x == 0 || !other_k, x == 1 || !other_k);
                        if (j + 2 == w.tiles && (x == 1 || !other_k)) ptx::tc_commit_elect(b_qe);
                    }
                    __syncwarp();
                }
            }
            base += w.tiles * per_tile;
        }
        // nothing of this CTA may still run on the tensor core when it ends
        ptx::tc_commit_elect(b_drain);
        __syncwarp();
        wait_warp(b_drain, 0);
    } else {
        // ================================================= softmax of tile x
        const int x = warp >> 2, t = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_off + x * 128, u_addr = tmem + lane_off + 256 + x * 128;
        const float c2 = p.scale_log2;
        const float2 c2v = make_float2(c2, c2);
        constexpr float kLimit = BF16 ? 4294967296.f : 32768.f;  // keeps every weight inside the 16-bit type
        uint32_t n = 0;   // key tiles of this query tile so far
        int base = 0;     // pieces of the units before
        bool ok = true;
        for (int r = 0; ok; ++r) {
            const int u = lf_unit_id(r);
            if (u >= p.units) break;
            bool bad = false;
            const LfUnit w = lf_unit(p, u, bad);
            if (bad && tid == 0) report(kBadData);
            if (w.row0 < 0) continue;
            const int first_row = w.row0 + 128 * x, row = first_row + t, T = w.n(x), offset = w.nk - w.nq;
            const bool mine = row < w.nq;
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
                    for (int c = 0; c < 64 * VP; c += 16) {
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
                // values of keys behind the request's last: zeros (by tile A's warps where A sees the tile)
                if (key0 + 128 > w.nk && (x == 0 || w.n(0) <= j)) {
                    const int from = w.nk - key0, vn = base + v_piece(j);
                    for (int i = 0; i < VP; ++i) {
                        const int at = vn + i;
                        if (!(ok = ok && wait_warp(b_full + 8 * (at % kLfSlots), (at / kLfSlots) & 1))) break;
                        // 1024 16-byte pieces: of 64 keys, twice (channel groups of half i, or both halves)
                        for (int c = t; c < 1024; c += 128) {
                            const int key = ((c >> 3) & 63) + 64 * (VP == 2 ? i : c >> 9);
                            if (key >= from)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ring + (at % kLfSlots) * kLfSlot + c * 16), "r"(0)
                                             : "memory");
                        }
                    }
                    if (!ok) break;
                    ptx::fence_proxy_async_smem();
                }
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
                ptx::tmem_wait_st();
                ptx::tc_fence_before_sync();
                ptx::mbar_arrive(b_ph + 8 * x);
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
                ptx::tmem_wait_st();
                ptx::tc_fence_before_sync();
                ptx::mbar_arrive(b_pf + 8 * x);
                sum += s.x + s.y, rsum += rs.x + rs.y;
            }
            // ---- O = U / sum
            if (ok && T > 0) ok = wait_warp(b_or + 8 * x, (n - 1) & 1);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            const float inv = rsum != 0.f ? 1.f / rsum : 0.f;
            const long long tok = w.q0 + row;
            uint16_t* dst = p.o + tok * p.o_st + static_cast<long long>(w.head) * p.o_sh;
#pragma unroll 1
            for (int c = 0; c < 64 * VP; c += 32) {
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
            base += w.tiles * per_tile;
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace paged
}  // namespace fa
