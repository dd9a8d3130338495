// kv_page_select.cuh - which pages one query per request should read.
//
// For whole-number queries qi and a page's whole-number channel bounds lo, hi
// (in units of 4 scales) sum_c max(qi lo, qi hi) = sum_c max(qi, 0) hi + min(qi, 0) lo
// bounds q . k over the page's keys from above.  Queries and bounds fit 8 bits,
// so four products are one instruction, the sum is exact in 32 bits (at most
// 256 * 127 * 112 < 2^24: exact in fp32 too), and the factor is a power of two:
// scores carry no rounding, and their order does not depend on how the sum is
// split.
// A cluster takes one (request, key head): its CTAs score shares of the pages
// into the first one's shared memory (as order-preserving 32-bit keys, counted
// by their top 8 bits on the way); that one finds the key of the
// num_selected-th best by histograms of 8 bits at a time, and writes the indices above
// it, and the first of those equal to it, in ascending order.
// What bounds it: 2 d + 4 bytes per page and head from HBM when there are many
// requests; for one the dependent reads (table, then bounds), which is why
// a group of lanes has four pages on their way at a time.  One request of 1024 pages
// and 8 heads: 7.7 us (25 with one CTA per head and a page at a time); 32 requests of up
// to 512 pages: 14.5 us.
#pragma once

#include "paged_common.cuh"

namespace fa {
namespace paged {

constexpr int kSelectThreads = 256;
constexpr int kSelectMaxPages = 32768;
constexpr int kSelectMaxCluster = 8;
constexpr int kSelectAhead = 4;    // pages a group of lanes has on their way

struct SelectParams {
    const uint16_t* q;
    long long q_st, q_sh;
    const int8_t* bounds;
    const float* k_scale;
    const int* table;
    const int* lens;
    int Hk, G, d, num_pages, page_shift, max_pages, keep;
    int cluster;      // CTAs that share a row's pages
    int* selected;
    int* count;
};

// fp32 -> uint32 in the same order
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <bool BF16>
__global__ void __launch_bounds__(kSelectThreads, 4) kv_page_select_kernel(const SelectParams p) {
    extern __shared__ __align__(16) uint32_t sel_smem[];
    // [G][d/4] words of max(qi, 0), then of min(qi, 0); [G] units; [pages] keys
    const int dw = p.d >> 2;
    uint32_t* qpos = sel_smem;
    uint32_t* qneg = qpos + p.G * dw;
    float* unit = reinterpret_cast<float*>(qneg + p.G * dw);
    uint32_t* keys = reinterpret_cast<uint32_t*>(unit + p.G);
    __shared__ uint32_t hist[2][256];
    __shared__ uint32_t pick, need;
    __shared__ int warp_n[2][kSelectThreads / 32];
    constexpr int kWarps = kSelectThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x % p.cluster, unit_at = blockIdx.x / p.cluster;
    const int h = unit_at % p.Hk, b = unit_at / p.Hk;
    static_assert(kSelectThreads == 256, "a thread per bin");
    hist[0][tid] = 0;
    dependents_may_start();
    wait_for_previous();
    int len = ld_meta(p.lens + b);
    if (len < 0 || len > (p.max_pages << p.page_shift)) {
        if (tid == 0 && rank == 0) report(kBadData);
        len = min(max(len, 0), p.max_pages << p.page_shift);
    }
    const int n = (len + (1 << p.page_shift) - 1) >> p.page_shift;
    int* out = p.selected + static_cast<long long>(unit_at) * p.keep;
    if (n <= p.keep) {  // all of them
        if (rank != 0) return;
        for (int i = tid; i < p.keep; i += kSelectThreads) out[i] = i < n ? i : -1;
        if (tid == 0) p.count[unit_at] = n;
        return;
    }
    // the first CTA's shared memory may be written once all of them have started
    if (p.cluster > 1) cluster_arrive();
    // LG lanes (16, or 8 for d <= 128) score one page: 16 channels per lane
    const int LG = p.d <= 128 ? 8 : 16, sub = tid % LG;
    const int per_pass = kSelectThreads / LG;
    const bool on = sub * 16 < p.d;
    const int share = (n + p.cluster - 1) / p.cluster, j_end = min(n, (rank + 1) * share);
    const int* trow = p.table + static_cast<long long>(b) * p.max_pages;
    bool bad_page = false;
    int page[kSelectAhead];
    float ks[kSelectAhead];
    int4 lo[kSelectAhead], hi[kSelectAhead];
    auto load_pages = [&](int j0) {
#pragma unroll
        for (int i = 0; i < kSelectAhead; ++i) {
            const int j = j0 + tid / LG + i * per_pass;
            page[i] = j < j_end ? ld_meta(trow + j) : 0;
        }
    };
    auto load_bounds = [&](int j0) {
#pragma unroll
        for (int i = 0; i < kSelectAhead; ++i) {
            const bool there = static_cast<unsigned>(page[i]) < static_cast<unsigned>(p.num_pages);
            bad_page |= !there;
            ks[i] = 0.f;
            lo[i] = hi[i] = make_int4(0, 0, 0, 0);
            if (there && j0 + tid / LG + i * per_pass < j_end) {
                const long long ph = static_cast<long long>(page[i]) * p.Hk + h;
                ks[i] = ld(p.k_scale + ph);
                if (on) {
                    const int4* bd = reinterpret_cast<const int4*>(p.bounds + ph * 2 * p.d) + sub;
                    lo[i] = ld(bd);
                    hi[i] = ld(bd + (p.d >> 4));
                }
            }
        }
    };
    load_pages(rank * share);  // (their latency passes while the queries are rounded)
    // queries to whole numbers, one warp per head of the group
    for (int g = warp; g < p.G; g += kWarps) {
        const uint16_t* q = p.q + static_cast<long long>(b) * p.q_st + static_cast<long long>(h * p.G + g) * p.q_sh;
        float f[8];
        const bool on = lane * 8 < p.d;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (on) v = ld(reinterpret_cast<const uint4*>(q + lane * 8));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack16(u[i], BF16);
            f[2 * i] = x.x, f[2 * i + 1] = x.y;
            a = fmaxf(a, fmaxf(fabsf(x.x), fabsf(x.y)));   // fmaxf passes NaN over
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const float s = pow2(query_unit_exp(a)), inv = 1.f / s;
        uint32_t pos[2] = {0, 0}, neg[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = f[e] != f[e] ? 0.f : fminf(fmaxf(f[e] * inv, -127.f), 127.f);
            const int i = __float2int_rn(x);
            pos[e >> 2] |= static_cast<uint32_t>(max(i, 0) & 255) << (8 * (e & 3));
            neg[e >> 2] |= static_cast<uint32_t>(min(i, 0) & 255) << (8 * (e & 3));
        }
        if (on) {
            *reinterpret_cast<uint2*>(qpos + g * dw + lane * 2) = make_uint2(pos[0], pos[1]);
            *reinterpret_cast<uint2*>(qneg + g * dw + lane * 2) = make_uint2(neg[0], neg[1]);
        }
        if (lane == 0) unit[g] = 4.f * s;
    }
    load_bounds(rank * share);
    __syncthreads();

    uint32_t keys_at = ptx::smem_addr(keys), hist_at = ptx::smem_addr(hist[0]);
    if (p.cluster > 1) {  // those of the cluster's first CTA
        asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(keys_at) : "r"(keys_at));
        asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(hist_at) : "r"(hist_at));
        cluster_wait();
    }
    for (int j0 = rank * share; j0 < j_end; j0 += per_pass * kSelectAhead) {
        if (j0 != rank * share) load_bounds(j0);
        const int j1 = j0 + per_pass * kSelectAhead;
        if (j1 < j_end) load_pages(j1);
        float best[kSelectAhead];
#pragma unroll
        for (int i = 0; i < kSelectAhead; ++i) best[i] = -INFINITY;
        for (int g = 0; g < p.G; ++g) {
            uint4 a = make_uint4(0, 0, 0, 0), c = a;
            if (on) {
                a = *reinterpret_cast<const uint4*>(qpos + g * dw + sub * 4);
                c = *reinterpret_cast<const uint4*>(qneg + g * dw + sub * 4);
            }
            const float u = unit[g];
#pragma unroll
            for (int i = 0; i < kSelectAhead; ++i) {
                int acc = 0;
                acc = __dp4a(hi[i].x, static_cast<int>(a.x), acc);
                acc = __dp4a(hi[i].y, static_cast<int>(a.y), acc);
                acc = __dp4a(hi[i].z, static_cast<int>(a.z), acc);
                acc = __dp4a(hi[i].w, static_cast<int>(a.w), acc);
                acc = __dp4a(lo[i].x, static_cast<int>(c.x), acc);
                acc = __dp4a(lo[i].y, static_cast<int>(c.y), acc);
                acc = __dp4a(lo[i].z, static_cast<int>(c.z), acc);
                acc = __dp4a(lo[i].w, static_cast<int>(c.w), acc);
                acc += __shfl_xor_sync(0xffffffffu, acc, 1);
                acc += __shfl_xor_sync(0xffffffffu, acc, 2);
                acc += __shfl_xor_sync(0xffffffffu, acc, 4);
                if (LG == 16) acc += __shfl_xor_sync(0xffffffffu, acc, 8);
                best[i] = fmaxf(best[i], static_cast<float>(acc) * (u * ks[i]));
            }
        }
#pragma unroll
        for (int i = 0; i < kSelectAhead; ++i) {
            const int j = j0 + tid / LG + i * per_pass;
            if (sub == 0 && j < j_end) {
                const uint32_t key = j == n - 1 ? 0xFFFFFFFFu : ordered(best[i] + 0.f);  // -0 counts as 0
                if (p.cluster > 1) {
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(keys_at + 4 * j), "r"(key) : "memory");
                    asm volatile("red.shared::cluster.add.u32 [%0], 1;" ::"r"(hist_at + 4 * (key >> 24)) : "memory");
                } else {
                    keys[j] = key;
                    atomicAdd(&hist[0][key >> 24], 1);
                }
            }
        }
    }
    if (bad_page) report(kBadData);
    if (p.cluster > 1) {
        cluster_sync();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }

    // the key of the keep-th best: 8 bits at a time from the top
    uint32_t prefix = 0, mask = 0, left = p.keep;
    for (int shift = 24; shift >= 0; shift -= 8) {
        const int buf = (shift >> 3) & 1 ^ 1;  // 24: 0, 16: 1, 8: 0, 0: 1
        if (shift < 24) {
            for (int j = tid; j < n; j += kSelectThreads)
                if ((keys[j] & mask) == prefix) atomicAdd(&hist[buf][(keys[j] >> shift) & 255], 1);
            __syncthreads();
        }
        hist[buf ^ 1][tid] = 0;  // the other buffer is for the next 8 bits
        if (warp == 0) {
            // counts of 8 bins per lane, summed from the top
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = hist[buf][255 - (lane * 8 + e)], sum += c[e];
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            uint32_t run = incl - sum;
            if (run < left && incl >= left) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (run < left && run + c[e] >= left) pick = 255 - (lane * 8 + e), need = left - run;
                    run += c[e];
                }
            }
        }
        __syncthreads();
        prefix |= pick << shift;
        mask |= 255u << shift;
        left = need;
    }
    // indices above that key, and the first `left` equal to it, in order
    int base = 0, base_eq = 0;
    for (int j0 = 0; j0 < n; j0 += kSelectThreads) {
        const int j = j0 + tid;
        const uint32_t k = j < n ? keys[j] : 0;
        const bool above = j < n && k > prefix, equal = j < n && k == prefix;
        const uint32_t m_eq = __ballot_sync(0xffffffffu, equal), m_ab = __ballot_sync(0xffffffffu, above);
        if (lane == 0) warp_n[0][warp] = __popc(m_ab), warp_n[1][warp] = __popc(m_eq);
        __syncthreads();
        int ab = base, eq = base_eq, ab_all = base, eq_all = base_eq;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) ab += warp_n[0][i], eq += warp_n[1][i];
            ab_all += warp_n[0][i], eq_all += warp_n[1][i];
        }
        const uint32_t lt = (1u << lane) - 1u;
        ab += __popc(m_ab & lt);
        eq += __popc(m_eq & lt);
        const bool take = above || (equal && eq < static_cast<int>(left));
        if (take) out[ab + min(eq, static_cast<int>(left))] = j;
        base = ab_all, base_eq = eq_all;
        __syncthreads();
    }
    if (tid == 0) p.count[unit_at] = p.keep;
}

}  // namespace paged
}  // namespace fa
