// paged_prompt_kernel.cuh - attention over the paged 8-bit cache for many
// query rows per key head (prompts and pieces of them), d <= 128.
//
// Three pieces of 1288 to 2048 queries over up to 8192 keys, 32 query and 8 key heads,
// d 128: 454 us, 1.09 PFLOP/s of visible pairs.  Of 3,840 cycles per key tile the products
// take 2,750 (2,048 at their full rate: the widened tiles are written to the shared
// memory that S = Q K^T reads without a pause), waits for weights 800, for K and V
// 290 (without the widening 410 us, without widening and softmax 349).
//
// The mathematics is that of paged_fwd_kernel.cuh: weights 2^(x_j + ev_j) with
// ev_j the exponent of the value page's scale, so that both products run on
// the codes themselves, widened to fp16 (exact).  Here the work is bound by
// the tensor cores, so it goes to tcgen05:
//   * packed rows r = i G + g (query i, head g of the group) of one key head;
//     a unit is 256 of them, two tiles A and B of 128, over one range of keys;
//   * warps 0-3 / 4-7: softmax of tile A / B.  Thread t owns row t (= TMEM
//     lane t).  At the start it reads its query row and writes it to shared
//     memory as fp16 (bf16 rows scaled by a power of two, which keeps every
//     bit above 2^-38 of the row's largest value), at the end it divides and
//     stores its row;
//   * warps 8-11 / 12-15: widen tiles of 128 keys of K / of V from the pages
//     to fp16 in shared memory (128-byte swizzle), one tile ahead in registers:
//     16-byte reads of 16 codes, two 16-byte stores.  Per key and channel that
//     is 2 conversions for 4 * 256 products, so it hides behind the MMAs;
//   * warp 16: issues tcgen05.mma, per key tile j in the order PV_A(j),
//     S_A(j+1), PV_B(j), S_B(j+1): while one tile's softmax runs, the tensor
//     core works for the other.  P V runs in two halves of 64 keys, the first
//     while the weights of the second are computed.
//   * registers: 20 warps are launched with 96 a thread, which the widening
//     ones keep; softmax threads rise to 128 with what the issuer's group gives
//     up (32768 + 24576 + 3072 of the 61440 launched);
//   * TMEM (512 columns): S_A 0, S_B 128 (fp32; the fp16 weights overwrite the
//     first 64 columns), U_A 256, U_B 384.
// Weights are 2^(x + ev - ref + 8), first against the reference that earlier
// tiles left: their sum over 64 keys bounds each of them, and only where it passes 2^15
// (fp16 ends at 2^16) the tile's maximum is taken, ref moves there and U is
// rescaled.  64 equal weights of 2^8 do not pass it, so rows of flat scores stay on
// the fast path; a weight keeps 11 bits down to 2^-22 of the reference.
#pragma once

#include <type_traits>

#include "paged_common.cuh"
#include "paged_fwd_kernel.cuh"

namespace fa {
namespace paged {

constexpr int kPrTile = 128;               // rows of a tile, keys of a key tile
constexpr int kPrRows = 2 * kPrTile;       // packed rows of a unit
constexpr int kPrThreads = 640;
constexpr int kPrSoftmaxRegs = 128, kPrIssueRegs = 24;
constexpr int kPrSub = 128 * 128;          // 128 rows x 64 fp16 columns, swizzled
constexpr int kPrMeta = 4;                 // key tiles whose scales are kept
constexpr float kPrShift = 8.f, kPrLimit = 32768.f;

template <int D>
struct PrCfg {
    static_assert(D == 64 || D == 128, "");
    static constexpr int kTileBytes = kPrTile * D * 2;
    static constexpr int kStages = 2;
    static constexpr int kOffK = 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffCtl = kOffV + kStages * kTileBytes;
    static constexpr int kSmem = kOffCtl + 1024 + 1024;
};

struct PrGroup {          // scales of 16 keys
    float ks, ev, rv;     // K's; log2 and reciprocal of V's (ev = -inf: no such keys)
};
struct PrCtl {
    uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_half[2], p_full[2], o_half[2], o_ready[2], drain;
    uint32_t tmem_base;
    PrGroup meta[kPrMeta][8];
};

// Shared-memory matrix descriptor for tcgen05.mma: 128-byte swizzle, start
// address, leading and stride byte offsets in 16-byte units, version 1.
__device__ __forceinline__ uint64_t pr_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor, kind::f16: fp16 operands, fp32 sums.
__host__ __device__ constexpr uint32_t pr_instr(int m, int n, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((static_cast<uint32_t>(n) >> 3) << 17) |
           ((static_cast<uint32_t>(m) >> 4) << 24);
}

// 16 codes that this SM reads once: not kept in L1, whose memory the tiles take.
__device__ __forceinline__ uint4 ldg_codes(const uint8_t* a) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(a) : "memory");
    return v;
}

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// 16 codes to fp16, stored at two 16-byte chunks of a swizzled row.
__device__ __forceinline__ void pr_widen16(uint32_t dst0, uint32_t dst1, const uint4& v) {
    const uint32_t c[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[2 * i] = e4m3x2_to_half2(c[i] & 0xFFFFu), h[2 * i + 1] = e4m3x2_to_half2(c[i] >> 16);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst0), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst1), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]) : "memory");
}

// The request and row block of the u-th block of `size` rows that the launch serves (false:
// there are not so many).  A thread counts a run of consecutive requests', the
// CTA sums up.
template <int THREADS>
__device__ __forceinline__ bool find_block(const PagedParams& p, int size, int u, int& b, int& rb) {
    __shared__ int warp_sums[THREADS / 32], found[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + THREADS - 1) / THREADS, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    auto blocks_of = [&](int i) {
        int q0, nq, len;
        bool bad = false;
        request_of(p, i, q0, nq, len, bad);
        return (nq * p.G + size - 1) / size;
    };
    int own = 0;
    for (int i = b0; i < b1; ++i) own += blocks_of(i);
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (tid == 0) found[0] = -1;
    if (lane == 31) warp_sums[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += warp_sums[w];
    int at = sum - own;  // blocks before the thread's first request
    if (at <= u && u < sum) {
        for (int i = b0; i < b1; ++i) {
            const int n = blocks_of(i);
            if (u < at + n) {
                found[0] = i, found[1] = at + n - 1 - u;  // (with the causal mask the last has the most keys)
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    b = found[0], rb = found[1];
    return b >= 0;
}

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1)
    paged_prompt_kernel(const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ v_codes, const PagedParams p,
                        const bool bf16) {
    using C = PrCfg<D>;
    extern __shared__ __align__(16) uint8_t pr_raw[];
    const uint32_t raw = ptx::smem_addr(pr_raw);
    uint8_t* smem = pr_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = ptx::smem_addr(smem);
    PrCtl* ctl = reinterpret_cast<PrCtl*>(smem + C::kOffCtl);
    const int tid = threadIdx.x, warp = tid >> 5;

    dependents_may_start();
    wait_for_previous();
    // ---- the unit: row blocks from the last (with the causal mask the one
    // with the most keys) to the first, then request, head, range
    int u = blockIdx.x;
    const int split = u % p.splits;
    u /= p.splits;
    const int h = u % p.Hk;
    u /= p.Hk;
    int b = u % p.B, rb = p.row_blocks - 1 - u / p.B;
    if (p.packed && !find_block<kPrThreads>(p, kPrRows, u, b, rb)) return;
    int q0, nq, len;
    bool bad = false;
    request_of(p, b, q0, nq, len, bad);
    if (len < 0 || len > (p.max_pages << p.page_shift)) bad = true, len = 0;
    if (bad && tid == 0) report(kBadData);
    const int rows = nq * p.G, r0 = rb * kPrRows;
    if (r0 >= rows) return;
    auto row_limit = [&](int r) { return p.causal ? min(len, len - nq + r / p.G + 1) : len; };
    // key tiles that a tile's last row sees, of them the range's [k0, k0 + T)
    auto tiles_of_rows = [&](int x) {
        if (r0 + x * kPrTile >= rows) return 0;
        return (max(row_limit(min(r0 + x * kPrTile + kPrTile, rows) - 1), 0) + kPrTile - 1) / kPrTile;
    };
    const int all_a = tiles_of_rows(0), all_b = tiles_of_rows(1), all = max(all_a, all_b);
    const int per = (all + p.splits - 1) / p.splits, k0 = min(split * per, all), k1 = min(k0 + per, all);
    const int TA = max(0, min(k1, all_a) - k0), TB = max(0, min(k1, all_b) - k0), T = max(TA, TB);

    const uint32_t b_q = ptx::smem_addr(&ctl->q_full), b_drain = ptx::smem_addr(&ctl->drain);
    const uint32_t b_kf = ptx::smem_addr(&ctl->k_full[0]), b_ke = ptx::smem_addr(&ctl->k_empty[0]);
    const uint32_t b_vf = ptx::smem_addr(&ctl->v_full[0]), b_ve = ptx::smem_addr(&ctl->v_empty[0]);
    const uint32_t b_sf = ptx::smem_addr(&ctl->s_full[0]), b_pf = ptx::smem_addr(&ctl->p_full[0]);
    const uint32_t b_or = ptx::smem_addr(&ctl->o_ready[0]);
    const uint32_t b_ph = ptx::smem_addr(&ctl->p_half[0]), b_oh = ptx::smem_addr(&ctl->o_half[0]);
    if (tid == 0) {
        ptx::mbar_init(b_q, 2 * kPrTile);
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(b_kf + 8 * s, 128);
            ptx::mbar_init(b_ke + 8 * s, 1);
            ptx::mbar_init(b_vf + 8 * s, 128);
            ptx::mbar_init(b_ve + 8 * s, 1);
            ptx::mbar_init(b_sf + 8 * s, 1);
            ptx::mbar_init(b_ph + 8 * s, kPrTile);
            ptx::mbar_init(b_pf + 8 * s, kPrTile);
            ptx::mbar_init(b_oh + 8 * s, 1);
            ptx::mbar_init(b_or + 8 * s, 1);
        }
        ptx::mbar_init(b_drain, 1);
        ptx::fence_mbar_init();
    }
    if (warp == 16) {
        ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;

    if (warp < 8) {
        // ================================================= softmax of tile x
        regs_inc<kPrSoftmaxRegs>();
        const int x = warp >> 2, t = tid & 127;
        const int r = r0 + x * kPrTile + t;
        const int TX = x ? TB : TA;
        const bool mine = r < rows;
        const int qi = mine ? r / p.G : 0, hq = h * p.G + (mine ? r - qi * p.G : 0);
        const long long tok = q0 + qi;
        // ---- the query row, fp16 in shared memory
        float unit = 1.f;
        {
            const uint16_t* src = p.q + tok * p.q_st + static_cast<long long>(hq) * p.q_sh;
            const uint32_t dst = sbase + x * C::kTileBytes + t * 128;
            float amax = 0.f;
            float s = 1.f;
            if (bf16) {
                for (int c = 0; c < D / 8; ++c) {
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
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (mine && c * 8 < p.d) v = ld(reinterpret_cast<const uint4*>(src + c * 8));
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
                if (bf16) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = unpack16(w[e], true);
                        w[e] = pack_half2(f.x * s, f.y * s);
                    }
                }
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (c >> 3) * kPrSub + (((c & 7) ^ (t & 7)) << 4)),
                             "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(b_q);
        }
        const float mul = unit * p.scale_log2;
        const int limit = mine ? row_limit(r) : len;
        const int first_limit = row_limit(min(r0 + x * kPrTile, rows - 1));  // the least of the tile's rows
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_off + x * 128, u_addr = tmem + lane_off + 256 + x * 128;
        float ref = -INFINITY, sum = 0.f;
        bool ok = true;
        for (int j = 0; j < TX; ++j) {
            if (!(ok = wait_warp(b_sf + 8 * x, j & 1))) break;
            ptx::tc_fence_after_sync();
            // (taken here so that a later wait on this tile's phase is unambiguous)
            if (j > 0 && !(ok = wait_warp(b_oh + 8 * x, (j - 1) & 1))) break;
            const PrGroup* meta = ctl->meta[j % kPrMeta];
            const int key0 = (k0 + j) * kPrTile;
            const bool edge = key0 + kPrTile > first_limit;
            const int seen = limit - key0;  // keys of this tile the row sees
            // largest x + ev of keys [64 hf, 64 hf + 64) of the tile
            auto half_top = [&](int hf) {
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
                    uint32_t sv[32];
                    ptx::tmem_ld_32x32b_x32(s_addr + c * 32, sv);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) ptx::reg_fence(sv[e]);
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c * 32 + e >= seen) sv[e] = __float_as_uint(-INFINITY);
                    }
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float m = __uint_as_float(sv[16 * g]);
#pragma unroll
                        for (int e = 1; e + 1 < 16; e += 2)
                            m = ptx::fmax3(m, __uint_as_float(sv[16 * g + e]), __uint_as_float(sv[16 * g + e + 1]));
                        m = fmaxf(m, __uint_as_float(sv[16 * g + 15]));
                        const PrGroup mt = meta[2 * c + g];
                        top = fmaxf(top, fmaf(m, mul * mt.ks, mt.ev));
                    }
                }
                return top;
            };
            // packed weights of those keys against ref; their sum (bounds each) and
            // the sum that counts for the row (without the value scales)
            auto half_weights_of = [&](auto masked, int hf, uint32_t(&pk)[32], float& bound, float& add) {
                const float sub = (ref == -INFINITY ? 0.f : ref) - kPrShift;
                bound = add = 0.f;
                uint32_t sv[32];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g % 2 == 0) {
                        ptx::tmem_ld_32x32b_x32(s_addr + hf * 64 + g * 16, sv);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ptx::reg_fence(sv[e]);
                    }
                    const PrGroup mt = meta[4 * hf + g];
                    const float f = mul * mt.ks, o = mt.ev - sub;
                    const float2 fv = make_float2(f, f), ov = make_float2(o, o);
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[16 * (g & 1) + 2 * e]),
                                                          __uint_as_float(sv[16 * (g & 1) + 2 * e + 1])), fv, ov);
                        if constexpr (decltype(masked)::value) {
                            if (hf * 64 + 16 * g + 2 * e >= seen) y.x = -INFINITY;
                            if (hf * 64 + 16 * g + 2 * e + 1 >= seen) y.y = -INFINITY;
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
            auto half_weights = [&](int hf, uint32_t(&pk)[32], float& bound, float& add) {
                if (edge)
                    half_weights_of(std::true_type{}, hf, pk, bound, add);
                else
                    half_weights_of(std::false_type{}, hf, pk, bound, add);
            };
            // U of the tiles before (and the sum) to a moved reference
            auto rescale = [&](float alpha) {
                const float2 av = make_float2(alpha, alpha);
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
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
            };
            uint32_t pk[32];
            float bound, add;
            half_weights(0, pk, bound, add);
            // (every branch around tcgen05.ld / st is uniform over the warp)
            if (__any_sync(0xffffffffu, ref == -INFINITY || bound > kPrLimit)) {
                // the tile's maximum; U holds the products of the tiles before
                // (S(j) was issued behind them)
                const float top = fmaxf(half_top(0), half_top(1));
                float alpha = 1.f;
                if (top > ref) {
                    if (ref != -INFINITY) alpha = ptx::ex2_approx(ref - top);
                    ref = top;
                }
                if (j > 0) rescale(alpha);
                sum *= alpha;
                half_weights(0, pk, bound, add);
            }
            ptx::tmem_st_32x32b_x32(s_addr, pk);
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            ptx::mbar_arrive(b_ph + 8 * x);
            sum += add;
            half_weights(1, pk, bound, add);
            if (__any_sync(0xffffffffu, bound > kPrLimit)) {
                // the first half's weights are under way: U takes them in first
                const float top = half_top(1);
                float alpha = 1.f;
                if (top > ref) {
                    if (ref != -INFINITY) alpha = ptx::ex2_approx(ref - top);
                    ref = top;
                }
                if (!(ok = wait_warp(b_oh + 8 * x, j & 1))) break;
                ptx::tc_fence_after_sync();
                rescale(alpha);
                sum *= alpha;
                half_weights(1, pk, bound, add);
            }
            ptx::tmem_st_32x32b_x32(s_addr + 32, pk);
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            ptx::mbar_arrive(b_pf + 8 * x);
            sum += add;
        }
        // ---- O = U / sum
        if (ok && TX > 0) ok = wait_warp(b_or + 8 * x, (TX - 1) & 1);
        if (ok) {
            ptx::tc_fence_after_sync();
            const float inv = sum != 0.f ? 1.f / sum : 0.f;
            const float lse2 = sum != 0.f ? ref - kPrShift + log2f(sum) : -INFINITY;
            const long long grow = tok * p.Hq + hq;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t ov[32];
                if (TX > 0) {
                    ptx::tmem_ld_32x32b_x32(u_addr + c * 32, ov);
                    ptx::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    if (TX > 0) ptx::reg_fence(ov[e]); else ov[e] = 0;
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
    } else if (warp < 16) {
        // ==================================== widen K (is_v = 0) or V tiles
        const int is_v = warp >= 12, ct = tid & 127;
        const uint8_t* codes = is_v ? v_codes : k_codes;
        const uint32_t tiles = sbase + (is_v ? C::kOffV : C::kOffK);
        const uint32_t b_full = is_v ? b_vf : b_kf, b_empty = is_v ? b_ve : b_ke;
        // thread ct takes rows row0 + RPP k of a tile, 16 channels (one piece) of
        // each.  Eight neighbouring threads hold four pieces of an even and of an
        // odd row: with the swizzle their stores go to eight different chunks.
        constexpr int PIECES = D / 16, RPP = 128 / PIECES, NV = kPrTile / RPP;
        const int ch = D == 64 ? ct & 3 : (ct & 3) | ((ct >> 1) & 4);
        const int row0 = D == 64 ? ct >> 2 : ((ct >> 4) << 1) | ((ct >> 2) & 1);
        const uint32_t dst_row = tiles + (ch >> 2) * kPrSub + row0 * 128;
        const uint32_t dst0 = dst_row + (((2 * (ch & 3)) ^ (row0 & 7)) << 4), dst1 = dst_row + (((2 * (ch & 3) + 1) ^ (row0 & 7)) << 4);
        const int P1 = (1 << p.page_shift) - 1;
        const int* trow = p.table + static_cast<long long>(b) * p.max_pages;
        // (pages hold whole groups of 16 keys, so a row's place in its group is the thread's own)
        const uint8_t* mine = codes + (static_cast<long long>(h << p.page_shift) + (row0 & 15)) * p.d + ch * 16;
        const long long page_bytes = (static_cast<long long>(p.Hk) << p.page_shift) * p.d;
        const bool ch_on = ch * 16 < p.d;
        // Page numbers run two tiles ahead and codes one: all loads of a tile are
        // independent of one another (bad table entries read nothing, reported at the end).
        // Lane g of a warp holds the page of the tile's g-th group of 16 keys.
        int pages = 0;
        bool bad_page = false;
        const int lane = ct & 31;
        auto load_pages = [&](int j) {
            if (lane < 8) pages = ld_meta(trow + (min((k0 + j) * kPrTile + 16 * lane, len - 1) >> p.page_shift));
        };
        uint4 v[NV];
        PrGroup mg = {1.f, -INFINITY, 1.f};
        auto load = [&](int j) {
            const int key0 = (k0 + j) * kPrTile;
            int page[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k) page[k] = __shfl_sync(0xffffffffu, pages, (row0 + RPP * k) >> 4);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int key = key0 + row0 + RPP * k;
                const bool there = static_cast<unsigned>(page[k]) < static_cast<unsigned>(p.num_pages);
                bad_page |= !there;
                v[k] = make_uint4(0, 0, 0, 0);
                if (there && key < len && ch_on)
                    v[k] = ldg_codes(mine + static_cast<long long>(page[k]) * page_bytes + ((key0 + (row0 & 16) + RPP * k) & P1) * p.d);
            }
            if (!is_v && ct < 8) {  // scales of the tile's eight groups of 16 keys
                mg = {1.f, -INFINITY, 1.f};
                if (static_cast<unsigned>(pages) < static_cast<unsigned>(p.num_pages) && key0 + 16 * ct < len) {
                    const int ph = pages * p.Hk + h;
                    const float vs = fminf(fmaxf(ld(p.v_scale + ph), 0x1p-60f), 0x1p60f);
                    mg = {fminf(fmaxf(ld(p.k_scale + ph), 0x1p-60f), 0x1p60f), log2f(vs), 1.f / vs};
                }
            }
        };
        if (T > 0) {  // (then len > 0)
            load_pages(0);
            load(0);
            load_pages(1);
        }
        for (int j = 0; j < T; ++j) {
            const int s = j & 1;
            if (j >= 2 && !wait_warp(b_empty + 8 * s, ((j >> 1) - 1) & 1)) break;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                pr_widen16(dst0 + s * C::kTileBytes + RPP * k * 128, dst1 + s * C::kTileBytes + RPP * k * 128, v[k]);
            if (!is_v && ct < 8) ctl->meta[j % kPrMeta][ct] = mg;
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(b_full + 8 * s);
            if (j + 1 < T) {
                load(j + 1);
                load_pages(j + 2);
            }
        }
        if (bad_page) report(kBadData);
    } else {
        regs_dec<kPrIssueRegs>();
        if (warp == 16) {
        // ============================================== tensor-core issuer
        constexpr uint32_t idesc_s = pr_instr(kPrTile, kPrTile, false), idesc_pv = pr_instr(kPrTile, D, true);
        constexpr uint64_t kStep = C::kTileBytes / 16;
        const uint64_t q_desc = pr_desc(sbase, 16, 1024), k_desc = pr_desc(sbase + C::kOffK, 16, 1024);
        const uint64_t v_desc = pr_desc(sbase + C::kOffV, kPrSub, 1024);
        auto issue_s = [&](int x, int s) {
            if constexpr (D == 128)
                ptx::mma_ss_k128(tmem + x * 128, q_desc + x * kStep, k_desc + s * kStep, idesc_s, 0u);
            else
                ptx::mma_ss_k64(tmem + x * 128, q_desc + x * kStep, k_desc + s * kStep, idesc_s, 0u);
            ptx::tc_commit_elect(b_sf + 8 * x);
        };
        auto issue_pv = [&](int x, int j, int s) {
            const uint64_t vd = v_desc + s * kStep;
            if (!wait_warp(b_ph + 8 * x, j & 1)) return false;
            ptx::tc_fence_after_sync();
            ptx::mma_ts_k64(tmem + 256 + x * 128, tmem + x * 128, vd, idesc_pv, j > 0 ? 1u : 0u);
            ptx::tc_commit_elect(b_oh + 8 * x);
            if (!wait_warp(b_pf + 8 * x, j & 1)) return false;
            ptx::tc_fence_after_sync();
            ptx::mma_ts_k64(tmem + 256 + x * 128, tmem + x * 128 + 32, vd + 512, idesc_pv, 1u);
            ptx::tc_commit_elect(b_or + 8 * x);
            return true;
        };
        bool ok = T > 0 && wait_warp(b_q, 0) && wait_warp(b_kf, 0);
        if (ok) {
            ptx::tc_fence_after_sync();
            if (TA > 0) issue_s(0, 0);
            if (TB > 0) issue_s(1, 0);
            ptx::tc_commit_elect(b_ke);
        }
        for (int j = 0; ok && j < T; ++j) {
            const int s = j & 1, n = s ^ 1;
            if (!(ok = wait_warp(b_vf + 8 * s, (j >> 1) & 1))) break;
            bool k_ready = false;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int TX = x ? TB : TA;
                if (j >= TX) continue;
                if (!(ok = issue_pv(x, j, s))) break;
                if (j + 1 < TX) {
                    if (!k_ready && !(ok = wait_warp(b_kf + 8 * n, ((j + 1) >> 1) & 1))) break;
                    k_ready = true;
                    ptx::tc_fence_after_sync();
                    issue_s(x, n);
                }
            }
            if (!ok) break;
            if (j + 1 < T) ptx::tc_commit_elect(b_ke + 8 * n);
            ptx::tc_commit_elect(b_ve + 8 * s);
            __syncwarp();
        }
        // nothing of this CTA may still run on the tensor core when it ends
        ptx::tc_commit_elect(b_drain);
        __syncwarp();
        wait_warp(b_drain, 0);
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 16) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace paged
}  // namespace fa
