// paged_prompt_wide_kernel.cuh - attention over the paged 8-bit cache for many
// query rows per key head, 128 < d <= 256.
//
// Two pieces of 1258 and 2000 queries over 3404 and 6000 keys, 16 query and 2 key heads, d 256:
// 268 us, 0.83 PFLOP/s of visible pairs (the few-row kernel 1085; with the scales read by
// the widening warps 300, page numbers looked up one by one 324).  Both of 2000 over 6000: 369.
//
// The mathematics is that of paged_prompt_kernel.cuh.  An accumulator of 128 rows
// takes half of TMEM here, so a unit is one tile of 128 packed rows, and the
// tensor core is kept busy by two key tiles in flight instead of two row tiles:
//   * TMEM (512 columns): Q 0 (128 columns of fp16 pairs), S_0 128 and S_1 192
//     (64 keys each, fp32; the fp16 weights overwrite the first 32 columns), U 256;
//   * Q as the first operand from TMEM leaves S = Q K^T half the reads of
//     shared memory, whose other half the widening's stores take: per 64
//     keys 1,024 cycles of products, 512 of operand reads, 512 of stores;
//   * warps 0-3: softmax, thread t owns row t;
//   * warps 4-11 / 12-19: widen tiles of 64 keys of K / of V to fp16 in shared
//     memory (128-byte swizzle, three stages), two tiles ahead in registers: a tile's
//     products are shorter than a read of its codes takes;
//   * warp 20: issues S(0), S(1), then per key tile j PV(j), S(j+2);
//   * warp 21: the scales, eight tiles at a time.
#pragma once

#include "paged_prompt_kernel.cuh"

namespace fa {
namespace paged {

constexpr int kPwRows = 128, kPwKeys = 64, kPwD = 256;
constexpr int kPwThreads = 704;
constexpr int kPwStages = 3, kPwMeta = 8;
constexpr int kPwSub = kPwKeys * 128;              // 64 rows x 64 fp16 columns, swizzled
constexpr int kPwTileBytes = kPwKeys * kPwD * 2;
constexpr int kPwOffV = kPwStages * kPwTileBytes, kPwOffCtl = 2 * kPwOffV;
constexpr int kPwSmem = kPwOffCtl + 1024 + 1024;

// The widening warps run at most kPwStages tiles ahead of S, the softmax at most two behind it.
static_assert(kPwMeta >= kPwStages + 2 && kPwMeta == 8, "");

struct PwCtl {
    uint64_t q_full, k_full[kPwStages], k_empty[kPwStages], v_full[kPwStages], v_empty[kPwStages], s_full[2], p_full[2],
        o_ready, drain;
    uint32_t tmem_base;
    PrGroup meta[kPwMeta][4];
};
static_assert(sizeof(PwCtl) <= 1024, "");

// First operand in TMEM, second K-major in shared memory, 64 channels: 4 steps.
__device__ __forceinline__ void pw_mma_ts_channels64(uint32_t d_tmem, uint32_t a_tmem, uint64_t b0, uint32_t idesc,
                                                     uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p0, p1;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p0, %4, 0;\n\t"
        "setp.eq.b32 p1, %4, %4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p0;\n\t"
        "add.u32 a, %1, 8;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p1;\n\t"
        "add.u32 a, %1, 16;\n\tadd.s64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p1;\n\t"
        "add.u32 a, %1, 24;\n\tadd.s64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p1;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b0), "r"(idesc), "r"(accumulate)
        : "memory");
}

__global__ void __launch_bounds__(kPwThreads, 1)
    paged_prompt_wide_kernel(const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ v_codes, const PagedParams p,
                             const bool bf16) {
    extern __shared__ __align__(16) uint8_t pw_raw[];
    const uint32_t raw = ptx::smem_addr(pw_raw);
    uint8_t* smem = pw_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = ptx::smem_addr(smem);
    PwCtl* ctl = reinterpret_cast<PwCtl*>(smem + kPwOffCtl);
    const int tid = threadIdx.x, warp = tid >> 5;

    dependents_may_start();
    wait_for_previous();
    // ---- the unit: row blocks from the last to the first, then request, head, range
    int u = blockIdx.x;
    const int split = u % p.splits;
    u /= p.splits;
    const int h = u % p.Hk;
    u /= p.Hk;
    int b = u % p.B, rb = p.row_blocks - 1 - u / p.B;
    if (p.packed && !find_block<kPwThreads>(p, kPwRows, u, b, rb)) return;
    int q0, nq, len;
    bool bad = false;
    request_of(p, b, q0, nq, len, bad);
    if (len < 0 || len > (p.max_pages << p.page_shift)) bad = true, len = 0;
    if (bad && tid == 0) report(kBadData);
    const int rows = nq * p.G, r0 = rb * kPwRows;
    if (r0 >= rows) return;
    auto row_limit = [&](int r) { return p.causal ? min(len, len - nq + r / p.G + 1) : len; };
    // key tiles that the last row sees, of them the range's [k0, k0 + T)
    const int all = (max(row_limit(min(r0 + kPwRows, rows) - 1), 0) + kPwKeys - 1) / kPwKeys;
    const int per = (all + p.splits - 1) / p.splits, k0 = min(split * per, all), T = min(k0 + per, all) - k0;

    const uint32_t b_q = ptx::smem_addr(&ctl->q_full), b_drain = ptx::smem_addr(&ctl->drain);
    const uint32_t b_kf = ptx::smem_addr(&ctl->k_full[0]), b_ke = ptx::smem_addr(&ctl->k_empty[0]);
    const uint32_t b_vf = ptx::smem_addr(&ctl->v_full[0]), b_ve = ptx::smem_addr(&ctl->v_empty[0]);
    const uint32_t b_sf = ptx::smem_addr(&ctl->s_full[0]), b_pf = ptx::smem_addr(&ctl->p_full[0]);
    const uint32_t b_or = ptx::smem_addr(&ctl->o_ready);
    if (tid == 0) {
        ptx::mbar_init(b_q, kPwRows);
        for (int s = 0; s < kPwStages; ++s) {
            ptx::mbar_init(b_kf + 8 * s, 257);
            ptx::mbar_init(b_ke + 8 * s, 1);
            ptx::mbar_init(b_vf + 8 * s, 256);
            ptx::mbar_init(b_ve + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(b_sf + 8 * s, 1);
            ptx::mbar_init(b_pf + 8 * s, kPwRows);
        }
        ptx::mbar_init(b_or, 1);
        ptx::mbar_init(b_drain, 1);
        ptx::fence_mbar_init();
    }
    if (warp == 20) {
        ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;

    if (warp < 4) {
        // ================================================= softmax
        const int r = r0 + tid;
        const bool mine = r < rows;
        const int qi = mine ? r / p.G : 0, hq = h * p.G + (mine ? r - qi * p.G : 0);
        const long long tok = q0 + qi;
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t u_addr = tmem + lane_off + 256;
        // ---- the query row, fp16 in TMEM
        float unit = 1.f;
        {
            const uint16_t* src = p.q + tok * p.q_st + static_cast<long long>(hq) * p.q_sh;
            float s = 1.f;
            if (bf16) {
                float amax = 0.f;
                for (int c = 0; c < kPwD / 8; ++c) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (mine && c * 8 < p.d) v = ld(reinterpret_cast<const uint4*>(src + c * 8));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = unpack16(w[e], true);
                        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
                const int e = amax > 0.f && amax < INFINITY
                                  ? max(-120, min(100, 14 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127))) : 0;
                s = pow2(e);
                unit = pow2(-e);
            }
#pragma unroll 1
            for (int c = 0; c < kPwD / 32; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (mine && c * 32 + i * 8 < p.d) v = ld(reinterpret_cast<const uint4*>(src + c * 32 + i * 8));
                    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
                }
                if (bf16) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 f = unpack16(w[e], true);
                        w[e] = pack_half2(f.x * s, f.y * s);
                    }
                }
                __syncwarp();
                ptx::tmem_st_32x32b_x16(tmem + lane_off + c * 16, w);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            ptx::mbar_arrive(b_q);
        }
        const float mul = unit * p.scale_log2;
        const int limit = mine ? row_limit(r) : len;
        const int first_limit = row_limit(r0);  // the least of the tile's rows
        float ref = -INFINITY, sum = 0.f;
        bool ok = true;
        for (int j = 0; j < T; ++j) {
            const uint32_t s_addr = tmem + lane_off + 128 + (j & 1) * 64;
            if (!(ok = wait_warp(b_sf + 8 * (j & 1), (j >> 1) & 1))) break;
            ptx::tc_fence_after_sync();
            const PrGroup* meta = ctl->meta[j % kPwMeta];
            const int key0 = (k0 + j) * kPwKeys;
            const bool edge = key0 + kPwKeys > first_limit;
            const int seen = limit - key0;  // keys of this tile the row sees
            // largest x + ev of the tile
            auto tile_top = [&] {
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t sv[16];
                    ptx::tmem_ld_32x32b_x16(s_addr + c * 16, sv);
                    ptx::tmem_wait_ld();
                    float m = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        ptx::reg_fence(sv[e]);
                        if (!edge || c * 16 + e < seen) m = fmaxf(m, __uint_as_float(sv[e]));
                    }
                    const PrGroup mt = meta[c];
                    top = fmaxf(top, fmaf(m, mul * mt.ks, mt.ev));
                }
                return top;
            };
            // packed weights against ref; their sum (bounds each) and the sum that
            // counts for the row (without the value scales)
            auto weights_of = [&](auto masked, uint32_t(&pk)[32], float& bound, float& add) {
                const float sub = (ref == -INFINITY ? 0.f : ref) - kPrShift;
                bound = add = 0.f;
                uint32_t sv[32];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g % 2 == 0) {
                        ptx::tmem_ld_32x32b_x32(s_addr + g * 16, sv);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ptx::reg_fence(sv[e]);
                    }
                    const PrGroup mt = meta[g];
                    const float f = mul * mt.ks, o = mt.ev - sub;
                    const float2 fv = make_float2(f, f), ov = make_float2(o, o);
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[16 * (g & 1) + 2 * e]),
                                                          __uint_as_float(sv[16 * (g & 1) + 2 * e + 1])), fv, ov);
                        if constexpr (decltype(masked)::value) {
                            if (16 * g + 2 * e >= seen) y.x = -INFINITY;
                            if (16 * g + 2 * e + 1 >= seen) y.y = -INFINITY;
                        }
                        const float2 w = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
                        acc = __fadd2_rn(acc, w);
                        pk[8 * g + e] = pack_half2(w.x, w.y);
                    }
                    const float both = acc.x + acc.y;
                    bound += both;
                    add = fmaf(both, mt.rv, add);
                }
            };
            uint32_t pk[32];
            float bound, add;
            auto weights = [&] {
                if (edge)
                    weights_of(std::true_type{}, pk, bound, add);
                else
                    weights_of(std::false_type{}, pk, bound, add);
            };
            weights();
            // (taken in every tile, so that no wait on this phase is ambiguous; S(j+1)
            // runs meanwhile)
            if (j > 0 && !(ok = wait_warp(b_or, (j - 1) & 1))) break;
            ptx::tc_fence_after_sync();
            // (every branch around tcgen05.ld / st is uniform over the warp)
            if (__any_sync(0xffffffffu, ref == -INFINITY || bound > kPrLimit)) {
                const float top = tile_top();
                float alpha = 1.f;
                if (top > ref) {
                    if (ref != -INFINITY) alpha = ptx::ex2_approx(ref - top);
                    ref = top;
                }
                if (j > 0) {
                    const float2 av = make_float2(alpha, alpha);
#pragma unroll 1
                    for (int c = 0; c < p.d / 16; ++c) {
                        uint32_t ov[16];
                        ptx::tmem_ld_32x32b_x16(u_addr + c * 16, ov);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            ptx::reg_fence(ov[e]);
                            ptx::reg_fence(ov[e + 1]);
                            const float2 y = __fmul2_rn(make_float2(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])), av);
                            ov[e] = __float_as_uint(y.x), ov[e + 1] = __float_as_uint(y.y);
                        }
                        ptx::tmem_st_32x32b_x16(u_addr + c * 16, ov);
                    }
                }
                sum *= alpha;
                weights();
            }
            ptx::tmem_st_32x32b_x32(s_addr, pk);
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            ptx::mbar_arrive(b_pf + 8 * (j & 1));
            sum += add;
        }
        // ---- O = U / sum
        if (ok && T > 0) ok = wait_warp(b_or, (T - 1) & 1);
        if (ok) {
            ptx::tc_fence_after_sync();
            const float inv = sum != 0.f ? 1.f / sum : 0.f;
            const float lse2 = sum != 0.f ? ref - kPrShift + log2f(sum) : -INFINITY;
            const long long grow = tok * p.Hq + hq;
#pragma unroll 1
            for (int c = 0; c < kPwD / 32; ++c) {
                uint32_t ov[32];
                if (T > 0) {
                    ptx::tmem_ld_32x32b_x32(u_addr + c * 32, ov);
                    ptx::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    if (T > 0) ptx::reg_fence(ov[e]); else ov[e] = 0;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    if (!mine || c * 32 + e >= p.d) continue;
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(ov[e + i]) * inv;
                    if (p.splits > 1) {
                        float4* dst = reinterpret_cast<float4*>(p.o_part + (grow * p.splits + split) * p.d + c * 32 + e);
                        dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                        dst[1] = make_float4(f[4], f[5], f[6], f[7]);
                    } else {
                        *reinterpret_cast<uint4*>(p.o + tok * p.o_st + static_cast<long long>(hq) * p.o_sh + c * 32 + e) =
                            make_uint4(pack16(f[0], f[1], bf16), pack16(f[2], f[3], bf16), pack16(f[4], f[5], bf16),
                                       pack16(f[6], f[7], bf16));
                    }
                }
                __syncwarp();
            }
            if (mine) {
                if (p.splits > 1)
                    p.lse_part[grow * p.splits + split] = lse2;
                else
                    p.lse[grow] = lse2 * 0.69314718055994531f;
            }
        }
    } else if (warp < 20) {
        // ==================================== widen K (is_v = 0) or V tiles
        const int is_v = warp >= 12, ct = (tid - 128) & 255, lane = tid & 31;
        const uint8_t* codes = is_v ? v_codes : k_codes;
        const uint32_t b_full = is_v ? b_vf : b_kf, b_empty = is_v ? b_ve : b_ke;
        // thread ct takes row row0 of each of the tile's four groups of 16 keys, 16
        // channels of it.  Eight neighbouring threads hold four pieces of an even and of
        // an odd row: with the swizzle their stores go to eight different chunks.
        const int sub = (ct >> 3) & 3, piece = ct & 3, ch = sub * 4 + piece, row0 = ((ct >> 5) << 1) | ((ct >> 2) & 1);
        const uint32_t dst_row = sbase + (is_v ? kPwOffV : 0) + sub * kPwSub + row0 * 128;
        const uint32_t dst0 = dst_row + (((2 * piece) ^ (row0 & 7)) << 4), dst1 = dst_row + (((2 * piece + 1) ^ (row0 & 7)) << 4);
        const int P1 = (1 << p.page_shift) - 1;
        const int* trow = p.table + static_cast<long long>(b) * p.max_pages;
        const uint8_t* mine = codes + (static_cast<long long>(h << p.page_shift) + row0) * p.d + ch * 16;
        const long long page_bytes = (static_cast<long long>(p.Hk) << p.page_shift) * p.d;
        const bool ch_on = ch * 16 < p.d;
        bool bad_page = false;
        // Page numbers: lane l of a warp holds that of the l-th group of 16 keys of eight
        // tiles; the next eight tiles' are on their way.
        int pages = 0, next_pages = 0;
        auto lookup = [&](int j) { return ld_meta(trow + (min((k0 + j) * kPwKeys + 16 * lane, len - 1) >> p.page_shift)); };
        // The codes a thread holds of a tile on its way; bad table entries read nothing
        // and are reported at the end.
        struct Held {
            uint4 v[4];
        } even, odd;
        auto load = [&](Held& t, int j) {  // j = 0, 1, 2, ...
            if (j % 8 == 0) pages = next_pages, next_pages = lookup(j + 8);
            const int key0 = (k0 + j) * kPwKeys;
            int at[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) at[k] = __shfl_sync(0xffffffffu, pages, (j % 8) * 4 + k);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool there = static_cast<unsigned>(at[k]) < static_cast<unsigned>(p.num_pages);
                bad_page |= !there;
                t.v[k] = make_uint4(0, 0, 0, 0);
                if (there && key0 + 16 * k + row0 < len && ch_on)
                    t.v[k] = ldg_codes(mine + static_cast<long long>(at[k]) * page_bytes + ((key0 + 16 * k) & P1) * p.d);
            }
        };
        int s = 0, phase = 1;  // (a first pass over the stages finds them empty)
        auto store = [&](Held& t, int j) {
            if (j >= kPwStages && !wait_warp(b_empty + 8 * s, phase)) return false;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                pr_widen16(dst0 + s * kPwTileBytes + 16 * k * 128, dst1 + s * kPwTileBytes + 16 * k * 128, t.v[k]);
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(b_full + 8 * s);
            if (++s == kPwStages) s = 0, phase ^= 1;
            if (j + 2 < T) load(t, j + 2);
            return true;
        };
        if (T > 0) {  // (then len > 0)
            next_pages = lookup(0);
            load(even, 0);
            if (T > 1) load(odd, 1);
        }
        for (int j = 0; j < T; j += 2) {
            if (!store(even, j)) break;
            if (j + 1 < T && !store(odd, j + 1)) break;
        }
        if (bad_page) report(kBadData);
    } else if (warp == 21) {
        // ========== scales: lane l holds those of the l-th group of 16 keys of eight tiles
        const int lane = tid & 31;
        const int* trow = p.table + static_cast<long long>(b) * p.max_pages;
        auto lookup = [&](int j) { return ld_meta(trow + (min((k0 + j) * kPwKeys + 16 * lane, len - 1) >> p.page_shift)); };
        int page = 0;
        float ks = 1.f, vs = 1.f;
        bool on = false;
        auto load = [&](int j) {
            on = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages) && (k0 + j) * kPwKeys + 16 * lane < len;
            if (on) ks = ld(p.k_scale + page * p.Hk + h), vs = ld(p.v_scale + page * p.Hk + h);
        };
        if (T > 0) {
            page = lookup(0);
            load(0);
            page = lookup(8);
        }
        PrGroup mine;
        int s = 0, phase = 1;
        for (int j = 0; j < T; ++j) {
            if (j % 8 == 0) {
                const float v = fminf(fmaxf(vs, 0x1p-60f), 0x1p60f);
                mine = on ? PrGroup{fminf(fmaxf(ks, 0x1p-60f), 0x1p60f), log2f(v), 1.f / v} : PrGroup{1.f, -INFINITY, 1.f};
                load(j + 8);
                page = lookup(j + 16);
            }
            if (j >= kPwStages && !wait_warp(b_ke + 8 * s, phase)) break;
            if (lane >> 2 == j % 8) ctl->meta[j % kPwMeta][lane & 3] = mine;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(b_kf + 8 * s);
            if (++s == kPwStages) s = 0, phase ^= 1;
        }
    } else {
        // ============================================== tensor-core issuer
        constexpr uint32_t idesc_s = pr_instr(kPwRows, kPwKeys, false);
        const uint32_t idesc_pv = pr_instr(kPwRows, p.d, true);
        constexpr uint64_t kStep = kPwTileBytes / 16;
        const uint64_t k_desc = pr_desc(sbase, 16, 1024), v_desc = pr_desc(sbase + kPwOffV, kPwSub, 1024);
        int ks = 0, kphase = 0;  // K's next stage
        auto issue_s = [&](int j) {
            if (!wait_warp(b_kf + 8 * ks, kphase)) return false;
            ptx::tc_fence_after_sync();
            for (int c = 0; c * 64 < p.d; ++c)
                pw_mma_ts_channels64(tmem + 128 + (j & 1) * 64, tmem + c * 32, k_desc + ks * kStep + c * (kPwSub / 16), idesc_s,
                                     c > 0 ? 1u : 0u);
            ptx::tc_commit_elect(b_sf + 8 * (j & 1));
            ptx::tc_commit_elect(b_ke + 8 * ks);
            if (++ks == kPwStages) ks = 0, kphase ^= 1;
            return true;
        };
        bool ok = T > 0 && wait_warp(b_q, 0);
        ptx::tc_fence_after_sync();
        if (ok) ok = issue_s(0);
        if (ok && T > 1) ok = issue_s(1);
        int vs = 0, vphase = 0;
        for (int j = 0; ok && j < T; ++j) {
            if (!(ok = wait_warp(b_vf + 8 * vs, vphase))) break;
            if (!(ok = wait_warp(b_pf + 8 * (j & 1), (j >> 1) & 1))) break;
            ptx::tc_fence_after_sync();
            ptx::mma_ts_k64(tmem + 256, tmem + 128 + (j & 1) * 64, v_desc + vs * kStep, idesc_pv, j > 0 ? 1u : 0u);
            ptx::tc_commit_elect(b_or);
            ptx::tc_commit_elect(b_ve + 8 * vs);
            if (++vs == kPwStages) vs = 0, vphase ^= 1;
            if (j + 2 < T) ok = issue_s(j + 2);
            __syncwarp();
        }
        // nothing of this CTA may still run on the tensor core when it ends
        ptx::tc_commit_elect(b_drain);
        __syncwarp();
        wait_warp(b_drain, 0);
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 20) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace paged
}  // namespace fa
