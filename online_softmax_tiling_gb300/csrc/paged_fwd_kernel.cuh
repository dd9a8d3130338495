// paged_fwd_kernel.cuh - attention over the paged 8-bit cache for few query
// rows per key head (decoding, short drafts, and head widths that the
// prompt kernel does not serve).
//
// Mathematics.  A value is code * 2^ev with ev constant over a page, so with
// weights w_j = 2^(x_j + ev_j) (x_j the scaled score in the base-2 domain)
//   O = sum_j w_j v8_j / sum_j w_j 2^-ev_j,   LSE = ln2 log2(sum_j w_j 2^-ev_j):
// the codes enter the second product as they are, and the running maximum is
// that of x_j + ev_j, the largest contribution to O.  Weights are scaled by a
// further 2^14 and rounded to fp16 (their fp32 values are summed): a weight
// keeps 11 bits down to 2^-28 of the row's largest contribution.  Scores are
// fp16 products with fp32 sums: e4m3 codes are exact in fp16, and a 16-bit query row is
// scaled by a power of two (its largest value to [2^14, 2^15)), which leaves
// out nothing above 2^-38 of that value.
//
// Mapping.  The G query heads of a key head (times the request's new tokens)
// are packed rows; a CTA takes 8, 16 or 32 of them and a range of keys.  Its four (or eight)
// warps take 32-key chunks in turn (16-key ones for d > 128), each
// with a TMA ring, a running softmax and an accumulator of its own; nothing
// is shared until the end, where their partial results are joined in
// shared memory.  The CTAs of 2, 4, 8 or 16 key ranges are a cluster and join
// theirs over distributed shared memory, without a workspace or a second
// launch; other counts go through a workspace and a merge.  For many keys
// (EVEN) the chunks of all requests and heads, in order, are dealt out in equal shares
// to as many CTAs as run at once: lengths as unequal as they like keep every SM
// busy to the end, and a CTA's fixed time (about 5 us) is paid once or twice instead of per
// range.  A share's first and last unit may be parts of one; the parts are
// joined by a second launch.  64 requests of 5000 to 16384 keys, 32 query and 8 key
// heads, d 128: 229 us, 6.1 TB/s (248 with two ranges per row); one request of 4096
// keys: 8.6 us (10.1 with 16 CTAs of four warps).  Reads are what bounds this kernel (2 d bytes per key and
// head against 4 G d operations), so mma.sync is the tensor path that fits:
// tcgen05 would take codes widened in shared memory, 128 rows at a time, for
// 4 to 16 rows of work.  Codes go from the swizzled tile into registers by
// 16-byte reads free of bank conflicts (lane (g, t) reads key g, channels
// 32 t ..; for V keys 2t, 2t+1, 2t+8, 2t+9, channels 16 g ..): channel and key
// orders inside a product are free as long as both operands agree, so the
// fragments need no shuffles.  With 16 or 32 rows the queries are the products'
// first operand (M = rows); with 8 the codes are (M = keys, then channels, and
// N = 8 rows), which takes half the mma instructions and accumulators and turns
// the 8 x 8 blocks of weights with movmatrix in between.
#pragma once

#include "paged_common.cuh"

namespace fa {
namespace paged {

constexpr float kWeightShift = 14.f;
constexpr int kDecMaxCluster = 16;

struct PagedParams {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    const int* cu_q;
    const int* table;
    const int* lens;
    const int* sel;
    const int* sel_count;
    const float* k_scale;
    const float* v_scale;
    long long q_st, q_sh, o_st, o_sh;
    int T, B, Hq, Hk, G, d, max_q, max_pages, num_sel, num_pages, page_shift;
    int rows_from, rows_to;  // requests of other counts of packed rows are another launch's
    int row_blocks;   // per request and key head
    int packed;       // only as many row blocks as there are, found by find_block
    int splits;       // key ranges per row block
    int in_cluster;   // the ranges are the CTAs of a cluster, which join their results themselves
    int box_rows;
    int causal;
    float scale_log2;
    float* o_part;    // [T * Hq][splits][d], or [2 CTAs][rows][d] (even shares)
    float* lse_part;  // [T * Hq][splits], or [2 CTAs][rows]; log2 units
    int4* shares;     // even shares: each CTA's first unit (first and last + 1 chunk, request, head)
};
constexpr int kEvenMaxB = 1024;  // requests whose chunk counts a CTA sums up

// Rows and keys of request b; marks that cannot be leave it without rows, and so
// does a count of rows that another launch serves.
__device__ __forceinline__ void request_of(const PagedParams& p, int b, int& q0, int& nq, int& len, bool& bad) {
    q0 = b, nq = 1;
    if (p.cu_q) {
        q0 = ld_meta(p.cu_q + b);
        nq = ld_meta(p.cu_q + b + 1) - q0;
        if (q0 < 0 || nq < 0 || nq > p.max_q || q0 > p.T - nq) bad = true, nq = 0;
        if (nq * p.G < p.rows_from || nq * p.G > p.rows_to) nq = 0;
    }
    len = ld_meta(p.lens + b);
}

template <int D, int R>
struct DecCfg {
    static constexpr int kKeys = D == 256 ? 16 : 32;    // keys per chunk
    static constexpr int kMinCtas = D == 256 || R == 32 ? 2 : 3;  // per SM
    static constexpr int kTiles = kKeys / 16;
    static constexpr int kStages = D == 64 ? 4 : D == 128 ? 2 : 3;
    static constexpr int kHalf = kKeys * D;             // K or V of a chunk
    static constexpr int kRing = kStages * 2 * kHalf;   // of one warp
    static constexpr int kSub = D == 256 ? 2 : 1;       // 128-byte column groups
    static constexpr int kSteps = D / 16;               // k16 steps of q k^T
    static constexpr int kCols = D / 8;                 // n8 tiles of P V
    static constexpr int kPieces = D / 8;               // 16-byte pieces of a query row
    static constexpr int kRowsPass = 32 / kPieces;      // query rows a warp reads at once
    static constexpr int kAccPad = D + 8;
};
// Bytes of shared memory: rings (the warps' partial results reuse them), the
// queries in fragment order, barriers.
template <int D, int R, bool EVEN, int W>
constexpr int dec_smem() {
    using C = DecCfg<D, R>;
    const int ring = W * C::kRing;
    const int join = W * (R * C::kAccPad + R * 2) * 4 + R * D * 4;
    return (ring > join ? ring : join) + R * C::kSteps * 32 + W * C::kStages * 8 + (EVEN ? (kEvenMaxB + 1) * 4 : 0) + 1024;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// What CTA `rank` of the cluster has at the shared address `a` of this one.
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t a, uint32_t rank) {
    float2 v;
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [r];\n\t}"
                 : "=f"(v.x), "=f"(v.y) : "r"(a), "r"(rank) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a, uint32_t rank) {
    float4 v;
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a), "r"(rank) : "memory");
    return v;
}

// Transposes an 8 x 8 block of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// R: rows of a CTA's block (8, 16 or 32).  W: warps, 4, or 8 in one CTA per SM where
// few CTAs have little to do each (one request of 4096 keys: a cluster of 8 such
// CTAs instead of 16 of four warps).  EVEN: equal shares of all chunks
// (one row block per request).
template <int D, int R, bool EVEN, int W>
__global__ void __launch_bounds__(32 * W, (W == 4 ? DecCfg<D, R>::kMinCtas : 1))
    paged_fwd_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const PagedParams p, const bool bf16) {
    using C = DecCfg<D, R>;
    constexpr int kDecWarps = W, kDecThreads = 32 * W;
    constexpr bool kTurned = R == 8;    // codes first, rows as N
    constexpr int MT = R / 16;          // 16-row tiles (not kTurned)
    constexpr int NST = C::kStages, KEYS = C::kKeys, NT = C::kTiles;
    extern __shared__ __align__(16) uint8_t dec_raw[];
    const uint32_t raw = ptx::smem_addr(dec_raw);
    uint8_t* smem = dec_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = ptx::smem_addr(smem);
    constexpr int kRings = kDecWarps * C::kRing;
    constexpr int kJoin = kDecWarps * (R * C::kAccPad + R * 2) * 4;
    constexpr int kJoinAll = kJoin + R * D * 4;  // and the CTA's joined result
    constexpr int kOffQ = kRings > kJoinAll ? kRings : kJoinAll;
    constexpr int kOffBar = kOffQ + R * C::kSteps * 32;
    uint4* qfrag = reinterpret_cast<uint4*>(smem + kOffQ);  // [MT][step][lane], or 8-byte [step][lane]
    __shared__ float row_unit[R];                           // 2^-e of each row's query scaling
    __shared__ __align__(8) float2 cta_stat[R];             // this CTA's maximum and sum of each row
    __shared__ int failed;                                  // a wait of this CTA ran out
    int* tab = reinterpret_cast<int*>(smem + kOffBar + kDecWarps * NST * 8);  // EVEN: chunks before each request

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;

    // (nothing here touches what the kernel before this one may still write)
    const uint32_t ring = sbase + warp * C::kRing;
    const uint32_t bars = sbase + kOffBar + warp * NST * 8;
    if (lane == 0) {
        for (int s = 0; s < NST; ++s) ptx::mbar_init(bars + 8 * s, 1);
        ptx::fence_mbar_init();
    }
    if (tid == 0) {
        failed = 0;
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    __syncwarp();
    dependents_may_start();
    wait_for_previous();
    // ---- EVEN: this CTA's share [f, f1) of all chunks, in order of request, head, chunk
    int f = 0, f0 = 0, f1 = 0;
    if constexpr (EVEN) {
        __shared__ int warp_sum[kDecWarps];
        const int per_thread = (p.B + kDecThreads - 1) / kDecThreads;
        const int b0 = min(tid * per_thread, p.B), b1 = min(b0 + per_thread, p.B);
        auto chunks_of = [&](int b) {
            int q, n, l;
            bool bad = false;
            request_of(p, b, q, n, l, bad);
            if (l < 0 || l > (p.max_pages << p.page_shift)) bad = true, l = 0;
            if (bad) report(kBadData);
            if (n == 0) return 0;
            if (p.sel) l = min(p.num_sel, (l + (1 << p.page_shift) - 1) >> p.page_shift) << p.page_shift;
            return (l + KEYS - 1) / KEYS * p.Hk;
        };
        int mine_sum = 0;
        for (int b = b0; b < b1; ++b) {
            const int n = chunks_of(b);
            tab[b] = n;
            mine_sum += n;
        }
        int incl = mine_sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int run = incl - mine_sum;
        for (int w = 0; w < warp; ++w) run += warp_sum[w];
        for (int b = b0; b < b1; ++b) {
            const int n = tab[b];
            tab[b] = run;
            run += n;
        }
        if (tid == kDecThreads - 1) tab[p.B] = run;
        __syncthreads();
        const int all = tab[p.B], G = static_cast<int>(gridDim.x), share = (all + G - 1) / G;
        f = f0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * share, static_cast<long long>(all)));
        f1 = min(f + share, all);
        if (tid == 0) {
            if (blockIdx.x == 0) p.shares[G] = make_int4(share, 0, 0, 0);
            if (f == f1) p.shares[blockIdx.x] = make_int4(f, f, 0, 0);
        }
        // rows of requests without a key
        for (int b = blockIdx.x; b < p.B; b += G) {
            if (tab[b + 1] != tab[b]) continue;
            int q, n, l;
            bool bad = false;
            request_of(p, b, q, n, l, bad);
            const int d4 = p.d >> 2;
            for (int i = tid; i < n * p.Hq * d4; i += kDecThreads) {
                const int row = i / d4, c = (i - row * d4) * 4, tok = row / p.Hq, hq = row - tok * p.Hq;
                *reinterpret_cast<uint2*>(p.o + (q + tok) * p.o_st + hq * p.o_sh + c) = make_uint2(0, 0);
                if (c == 0) p.lse[static_cast<long long>(q + tok) * p.Hq + hq] = -INFINITY;
            }
        }
    }
    int base = 0;  // chunks this warp has taken before this unit (phases of its ring)
    do {
    // unit: range fastest (a cluster's CTAs), then row block (they read the same keys), head, request
    int split = 0, rb = 0, h, b, first = 0, last = 0;
    bool whole = !EVEN;
    if constexpr (EVEN) {
        if (f >= f1) break;
        b = owner_of(tab, p.B, f);
        const int n = (tab[b + 1] - tab[b]) / p.Hk, rel = f - tab[b];
        h = rel / n;
        first = rel - h * n;
        last = min(n, first + f1 - f);
        whole = first == 0 && last == n;
        if (tid == 0 && f == f0)
            p.shares[blockIdx.x] = make_int4(f - first, f - first + n, b, h);
        f += last - first;
    } else {
        int u = blockIdx.x;
        split = u % p.splits;
        u /= p.splits;
        rb = u % p.row_blocks;
        u /= p.row_blocks;
        h = u % p.Hk, b = u / p.Hk;
    }

    int q0, nq, len;
    bool bad = false;
    request_of(p, b, q0, nq, len, bad);
    // This warp's chunks are chunk0 + k step, whatever the length (ranges are
    // interleaved, a share is contiguous): the pages of the first 32 are looked up
    // while the length is still on its way.
    const int chunk0 = EVEN ? first + warp : split * kDecWarps + warp, step = EVEN ? kDecWarps : p.splits * kDecWarps;
    int early[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const long long lp = (static_cast<long long>(chunk0 + lane * step) * KEYS + i * 16) >> p.page_shift;
        early[i] = 0;
        if (!p.sel && lp < p.max_pages) early[i] = ld_meta(p.table + static_cast<long long>(b) * p.max_pages + lp);
    }
    // the query rows, on their way while the lengths and pages are looked up
    constexpr int kQPass = (R + kDecWarps * C::kRowsPass - 1) / (kDecWarps * C::kRowsPass);
    const int piece = lane % C::kPieces, sub_row = lane / C::kPieces;
    const int r0 = rb * R;
    uint4 qv[kQPass];
#pragma unroll
    for (int i = 0; i < kQPass; ++i) {
        const int r = (i * kDecWarps + warp) * C::kRowsPass + sub_row, pr = r0 + r;
        qv[i] = make_uint4(0, 0, 0, 0);
        if (r < R && pr < nq * p.G && piece * 8 < p.d) {
            const int tok = pr / p.G, hg = pr - tok * p.G;
            qv[i] = ld(reinterpret_cast<const uint4*>(
                p.q + static_cast<long long>(q0 + tok) * p.q_st + static_cast<long long>(h * p.G + hg) * p.q_sh + piece * 8));
        }
    }
    if (len < 0 || (len >> p.page_shift) > p.max_pages || len > (p.max_pages << p.page_shift)) bad = true, len = 0;
    if (bad && tid == 0) report(kBadData);
    const int rows = nq * p.G;                 // packed rows of the request: r = i G + g
    if (!EVEN && r0 >= rows) return;
    const int my_rows = min(R, rows - r0);
    // keys the last row of the block sees; places the range covers (with a
    // selection, places in the concatenated selected pages)
    const int last_i = (r0 + my_rows - 1) / p.G;
    const int kend = p.causal ? min(len, len - nq + last_i + 1) : len;
    int places = max(kend, 0);
    if (p.sel) {
        int n = ld_meta(p.sel_count + b * p.Hk + h);
        if (n < 0 || n > p.num_sel) {
            if (tid == 0) report(kBadData);
            n = 0;
        }
        places = n << p.page_shift;
    }
    const int chunks = (places + KEYS - 1) / KEYS;
    const int end = EVEN ? min(last, chunks) : chunks;
    const int mine = end > chunk0 ? (end - chunk0 + step - 1) / step : 0;  // chunks of this warp

    // What a warp needs of its next chunks, per 16-key tile: lane i holds that
    // of chunk 32 n + i (refilled one block ahead).
    struct Meta {
        int row[NT];      // first row of the tile in the cache's tensor map, -1: none
        int pos[NT];      // position of the tile's first key
        float ks[NT], ev[NT], rv[NT];  // scales: of K; log2 and reciprocal of V's
    };
    // pages first, so that the boxes can be issued; then the scales
    auto fetch = [&](int k, bool looked_up) {
        Meta m;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            m.row[i] = -1, m.pos[i] = len;
            const int place = k < mine ? (chunk0 + k * step) * KEYS + i * 16 : places;
            if (place >= places) continue;
            int lp = place >> p.page_shift;
            const int off = place & ((1 << p.page_shift) - 1);
            if (p.sel) lp = ld_meta(p.sel + static_cast<long long>(b * p.Hk + h) * p.num_sel + lp);
            const int pos = (lp << p.page_shift) + off;
            if (lp < 0 || lp >= p.max_pages) {
                report(kBadData);
            } else if (pos < len) {
                const int page = looked_up && !p.sel ? early[i] : ld_meta(p.table + static_cast<long long>(b) * p.max_pages + lp);
                if (page < 0 || page >= p.num_pages) {
                    report(kBadData);
                } else {
                    m.row[i] = ((page * p.Hk + h) << p.page_shift) + off;
                    m.pos[i] = pos;
                }
            }
        }
        return m;
    };
    auto fetch_scales = [&](Meta& m) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int ph = max(m.row[i], 0) >> p.page_shift;
            m.ks[i] = fminf(fmaxf(ld(p.k_scale + ph), 0x1p-60f), 0x1p60f);
            const float vs = fminf(fmaxf(ld(p.v_scale + ph), 0x1p-60f), 0x1p60f);
            m.ev[i] = log2f(vs);
            m.rv[i] = 1.f / vs;
        }
    };
    // boxes of a chunk into stage s; every chunk completes its phase (missing
    // tiles are masked, so their stage may hold anything)
    auto issue = [&](const int (&row)[NT], int s) {
        const uint32_t kd = ring + s * 2 * C::kHalf, vd = kd + C::kHalf, bar = bars + 8 * s;
        if (lane != 0) return;
        const int tiles_per_box = p.box_rows >> 4;
        uint32_t bytes = 0;
        for (int i = 0; i < NT; i += tiles_per_box)
            if (row[i] >= 0) bytes += 2 * p.box_rows * D;
        if (bytes == 0) {
            ptx::mbar_arrive(bar);
            return;
        }
        ptx::mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if ((i & (tiles_per_box - 1)) || row[i] < 0) continue;
#pragma unroll
            for (int c = 0; c < C::kSub; ++c) {
                constexpr int kRowBytes = D > 128 ? 128 : D;  // of a row in one column group
                tma_load_2d(kd + c * KEYS * 128 + i * 16 * kRowBytes, &tm_k, bar, 128 * c, row[i]);
                tma_load_2d(vd + c * KEYS * 128 + i * 16 * kRowBytes, &tm_v, bar, 128 * c, row[i]);
            }
        }
    };
    Meta cur = fetch(lane, true), nxt = cur;
    auto row_of = [&](int k, int (&row)[NT]) {  // k in the current or the next block
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int a = __shfl_sync(0xffffffffu, cur.row[i], k & 31);
            const int c = __shfl_sync(0xffffffffu, nxt.row[i], k & 31);
            row[i] = (k >> 5) & 1 ? c : a;
        }
    };
    // (blocks alternate between cur and nxt by parity of k / 32)
#pragma unroll
    for (int s = 0; s < NST; ++s) {
        if (s < mine) {
            int row[NT];
            row_of(s, row);
            issue(row, (base + s) % NST);
        }
    }
    fetch_scales(cur);
    if (mine > 32) {
        nxt = fetch(32 + lane, false);
        fetch_scales(nxt);
    }

    // queries: rows scaled to fp16 and stored in fragment order
#pragma unroll
    for (int i = 0; i < kQPass; ++i) {
        const int r = (i * kDecWarps + warp) * C::kRowsPass + sub_row;
        const uint32_t u4[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
        float f[8], a = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 x = unpack16(u4[e], bf16);
            f[2 * e] = x.x, f[2 * e + 1] = x.y;
            a = fmaxf(a, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
#pragma unroll
        for (int o = C::kPieces / 2; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        // power of two that takes the largest value to [2^14, 2^15)
        const int e = a > 0.f && a < INFINITY ? max(-120, min(100, 14 - (static_cast<int>(__float_as_uint(a) >> 23) - 127))) : 0;
        const float s = pow2(e);
        if (r >= R) continue;
        if (piece == 0) row_unit[r] = pow2(-e);
        // channel c -> step, word half, lane quarter: within 128 channels
        // lane quarter t holds 32 t .. 32 t + 31 (d = 64: 16 t .. 16 t + 15)
        constexpr int CPL = D == 64 ? 16 : 32;
        const int c = piece * 8, cg = c / 128, cc = c % 128, t = cc / CPL, w = (cc % CPL) / 4;
        const int mt = r / 16, rr = r % 16;
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {  // two words of four channels
            const int step = cg * 8 + w + e2;
            if constexpr (kTurned) {
                reinterpret_cast<uint2*>(qfrag)[step * 32 + r * 4 + t] =
                    make_uint2(pack_half2(f[4 * e2] * s, f[4 * e2 + 1] * s), pack_half2(f[4 * e2 + 2] * s, f[4 * e2 + 3] * s));
            } else {
                uint32_t* dst = reinterpret_cast<uint32_t*>(qfrag + (mt * C::kSteps + step) * 32 + (rr & 7) * 4 + t);
                dst[rr >> 3] = pack_half2(f[4 * e2] * s, f[4 * e2 + 1] * s);
                dst[2 + (rr >> 3)] = pack_half2(f[4 * e2 + 2] * s, f[4 * e2 + 3] * s);
            }
        }
    }
    __syncthreads();

    // the rows a lane holds: g and g + 8 of each tile, or 2 t and 2 t + 1
    constexpr int NR = kTurned ? 1 : MT;
    auto row_at = [&](int m, int e) { return kTurned ? 2 * t4 + e : 16 * m + 8 * e + g; };
    float mul[NR][2];      // score -> base-2 units
    int limit[NR][2];      // keys the row sees
    int min_limit = len;
#pragma unroll
    for (int m = 0; m < NR; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row_at(m, e);
            mul[m][e] = row_unit[r] * p.scale_log2;
            limit[m][e] = r < my_rows ? (p.causal ? min(len, len - nq + (r0 + r) / p.G + 1) : len) : 0;
            if (r < my_rows) min_limit = min(min_limit, limit[m][e]);
        }
    min_limit = __reduce_min_sync(0xffffffffu, min_limit);  // every row of the block sees keys below it

    // accumulators: n8 tiles of channels, or m16 tiles of channels by 8 rows
    constexpr int NA = kTurned ? D / 16 : C::kCols;
    float acc[NR][NA][4];
    float mx[NR][2], sum[NR][2];
#pragma unroll
    for (int m = 0; m < NR; ++m) {
#pragma unroll
        for (int c = 0; c < NA; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][c][e] = 0.f;
        mx[m][0] = mx[m][1] = -INFINITY;
        sum[m][0] = sum[m][1] = 0.f;
    }
    uint2 qt[kTurned ? C::kSteps : 1];
    if constexpr (kTurned) {
#pragma unroll
        for (int i = 0; i < C::kSteps; ++i) qt[i] = reinterpret_cast<const uint2*>(qfrag)[i * 32 + lane];
    }

    bool ok = true;
    int k = 0;
    for (; k < mine; ++k) {
        const int s = (base + k) % NST;
        if (!(ok = wait_warp(bars + 8 * s, ((base + k) / NST) & 1))) break;
        const uint32_t ks_base = ring + s * 2 * C::kHalf, vs_base = ks_base + C::kHalf;
        int pos[NT], row[NT];
        float kf[NT], ev[NT], rv[NT];
        const bool odd = (k >> 5) & 1;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            pos[i] = __shfl_sync(0xffffffffu, odd ? nxt.pos[i] : cur.pos[i], k & 31);
            row[i] = __shfl_sync(0xffffffffu, odd ? nxt.row[i] : cur.row[i], k & 31);
            kf[i] = __shfl_sync(0xffffffffu, odd ? nxt.ks[i] : cur.ks[i], k & 31);
            ev[i] = __shfl_sync(0xffffffffu, odd ? nxt.ev[i] : cur.ev[i], k & 31);
            rv[i] = __shfl_sync(0xffffffffu, odd ? nxt.rv[i] : cur.rv[i], k & 31);
        }
        // ---- scores.  Rows first: n8 tile j holds keys 8 j + ... of rows g, g + 8;
        // codes first: m16 tile i holds keys 16 i + g and + 8 of rows 2 t, 2 t + 1
        constexpr int NS = kTurned ? NT : 2 * NT;
        float sc[NR][NS][4];
#pragma unroll
        for (int m = 0; m < NR; ++m)
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[m][j][e] = 0.f;
#pragma unroll
        for (int cg = 0; cg < C::kSub; ++cg) {
#pragma unroll
            for (int half = 0; half < (D == 64 ? 1 : 2); ++half) {
                uint4 kw[2 * NT];
#pragma unroll
                for (int j = 0; j < 2 * NT; ++j) {
                    const int key = 8 * j + g;
                    if constexpr (D == 64)
                        kw[j] = lds128(ks_base + key * 64 + ((t4 ^ ((key >> 1) & 3)) << 4));
                    else
                        kw[j] = lds128(ks_base + cg * KEYS * 128 + key * 128 + (((2 * t4 + half) ^ (key & 7)) << 4));
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int step = cg * 8 + half * 4 + w;
                    if constexpr (kTurned) {
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const uint4 &k0 = kw[2 * i], &k1 = kw[2 * i + 1];
                            const uint32_t x = w == 0 ? k0.x : w == 1 ? k0.y : w == 2 ? k0.z : k0.w;
                            const uint32_t y = w == 0 ? k1.x : w == 1 ? k1.y : w == 2 ? k1.z : k1.w;
                            mma_f16(sc[0][i], e4m3x2_to_half2(x & 0xFFFFu), e4m3x2_to_half2(y & 0xFFFFu), e4m3x2_to_half2(x >> 16),
                                    e4m3x2_to_half2(y >> 16), qt[step].x, qt[step].y);
                        }
                    } else {
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint4 a = qfrag[(m * C::kSteps + step) * 32 + lane];
#pragma unroll
                        for (int j = 0; j < 2 * NT; ++j) {
                            const uint32_t x = w == 0 ? kw[j].x : w == 1 ? kw[j].y : w == 2 ? kw[j].z : kw[j].w;
                            mma_f16(sc[m][j], a.x, a.y, a.z, a.w, e4m3x2_to_half2(x & 0xFFFFu), e4m3x2_to_half2(x >> 16));
                        }
                    }
                    }
                }
            }
        }
        // ---- weights.  Element e of a score tile: row e >> 1 and key e & 1 of the
        // lane's, or row e & 1 and key e >> 1 where the codes come first
        uint32_t pa[NR][NT][4];
        bool edge = false;
#pragma unroll
        for (int i = 0; i < NT; ++i) edge |= row[i] < 0 || pos[i] + 16 > min_limit;
#pragma unroll
        for (int m = 0; m < NR; ++m) {
            float top[2] = {mx[m][0], mx[m][1]};
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = kTurned ? j : j / 2, r = kTurned ? e & 1 : e >> 1;
                    const int key = kTurned ? g + 8 * (e >> 1) : 8 * (j & 1) + 2 * t4 + (e & 1);
                    float x = fmaf(sc[m][j][e], mul[m][r] * kf[i], ev[i]);
                    if (edge && (row[i] < 0 || pos[i] + key >= limit[m][r])) x = -INFINITY;
                    sc[m][j][e] = x;
                    top[r] = fmaxf(top[r], x);
                }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int o = kTurned ? 4 : 1; o < (kTurned ? 32 : 4); o *= 2)
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], o));
            const float ref[2] = {top[0] == -INFINITY ? 0.f : top[0] - kWeightShift,
                                  top[1] == -INFINITY ? 0.f : top[1] - kWeightShift};
            if (__any_sync(0xffffffffu, top[0] != mx[m][0] || top[1] != mx[m][1])) {
                const float al[2] = {ptx::ex2_approx(mx[m][0] - (top[0] == -INFINITY ? 0.f : top[0])),
                                     ptx::ex2_approx(mx[m][1] - (top[1] == -INFINITY ? 0.f : top[1]))};
#pragma unroll
                for (int c = 0; c < NA; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][c][e] *= al[kTurned ? e & 1 : e >> 1];
                sum[m][0] *= al[0], sum[m][1] *= al[1];
                mx[m][0] = top[0], mx[m][1] = top[1];
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if constexpr (kTurned) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = ptx::ex2_approx(sc[m][i][e] - ref[e & 1]);
                    sum[m][0] = fmaf(w[0] + w[2], rv[i], sum[m][0]);
                    sum[m][1] = fmaf(w[1] + w[3], rv[i], sum[m][1]);
                    pa[m][i][0] = transpose8x8(pack_half2(w[0], w[1]));  // keys 2t, 2t + 1 of row g
                    pa[m][i][1] = transpose8x8(pack_half2(w[2], w[3]));  // keys 2t + 8, 2t + 9
                } else {
                    float w[8];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[4 * j + e] = ptx::ex2_approx(sc[m][2 * i + j][e] - ref[e >> 1]);
                    sum[m][0] = fmaf((w[0] + w[1]) + (w[4] + w[5]), rv[i], sum[m][0]);
                    sum[m][1] = fmaf((w[2] + w[3]) + (w[6] + w[7]), rv[i], sum[m][1]);
                    pa[m][i][0] = pack_half2(w[0], w[1]);
                    pa[m][i][1] = pack_half2(w[2], w[3]);
                    pa[m][i][2] = pack_half2(w[4], w[5]);
                    pa[m][i][3] = pack_half2(w[6], w[7]);
                }
            }
        }
        // ---- U += P V, 16 keys at a time
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (edge && row[i] < 0) continue;
#pragma unroll
            for (int cg = 0; cg < C::kSub; ++cg) {
                constexpr int WORDS = D == 64 ? 2 : 4;   // 4-channel words per key and lane
                uint32_t vw[4][WORDS];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = 16 * i + 8 * (e >> 1) + 2 * t4 + (e & 1);
                    if constexpr (D == 64) {
                        const uint2 v = lds64(vs_base + key * 64 + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
                        vw[e][0] = v.x, vw[e][1] = v.y;
                    } else {
                        const uint4 v = lds128(vs_base + cg * KEYS * 128 + key * 128 + ((g ^ (key & 7)) << 4));
                        vw[e][0] = v.x, vw[e][1] = v.y, vw[e][2] = v.z, vw[e][3] = v.w;
                    }
                    // what lies behind the last key carries no weight and may be anything, NaN too
                    if (edge && pos[i] + key - 16 * i >= len)
#pragma unroll
                        for (int w = 0; w < WORDS; ++w) vw[e][w] = 0;
                }
#pragma unroll
                for (int w = 0; w < WORDS; ++w) {
                    // pairs of keys (2t, 2t+1) and (2t+8, 2t+9) of each of four channels
                    const uint32_t l0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), l1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
                    const uint32_t h0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), h1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
                    const uint32_t b0[4] = {e4m3x2_to_half2(l0 & 0xFFFFu), e4m3x2_to_half2(l0 >> 16),
                                            e4m3x2_to_half2(l1 & 0xFFFFu), e4m3x2_to_half2(l1 >> 16)};
                    const uint32_t b1[4] = {e4m3x2_to_half2(h0 & 0xFFFFu), e4m3x2_to_half2(h0 >> 16),
                                            e4m3x2_to_half2(h1 & 0xFFFFu), e4m3x2_to_half2(h1 >> 16)};
                    if constexpr (kTurned) {
                        // rows (channels) 2 c and 2 c + 1 of the lane's, 8 c apart in the tile
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            mma_f16(acc[0][cg * 8 + 2 * w + c], b0[2 * c], b0[2 * c + 1], b1[2 * c], b1[2 * c + 1], pa[0][i][0], pa[0][i][1]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int m = 0; m < MT; ++m)
                                mma_f16(acc[m][cg * 16 + 4 * w + c], pa[m][i][0], pa[m][i][1], pa[m][i][2], pa[m][i][3], b0[c], b1[c]);
                    }
                }
            }
        }
        __syncwarp();
        // the stage is read: load the chunk NST further on
        if (k + NST < mine) {
            int nrow[NT];
            row_of(k + NST, nrow);
            issue(nrow, s);
        }
        // chunk k was the last of its block: refill that block two further on
        if ((k & 31) == 31) {
            Meta m = fetch(k + 33 + lane, false);
            fetch_scales(m);
            if (odd) nxt = m; else cur = m;
        }
    }
    if (!ok) {  // let copies in flight land before the CTA ends
        if (lane == 0) failed = 1;
        for (const int until = min(k + NST, mine); k < until; ++k) wait_warp(bars + 8 * ((base + k) % NST), ((base + k) / NST) & 1);
    }

    // ---- join the warps' partial results
#pragma unroll
    for (int m = 0; m < NR; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int o = kTurned ? 4 : 1; o < (kTurned ? 32 : 4); o *= 2)
                sum[m][r] += __shfl_xor_sync(0xffffffffu, sum[m][r], o);
    __syncthreads();  // every ring is drained: its memory takes the partial results
    if (EVEN && failed) break;  // (the phases of its ring are lost)
    float* part = reinterpret_cast<float*>(smem);
    constexpr int kPartWarp = R * C::kAccPad + R * 2;
    {
        float* mypart = part + warp * kPartWarp;
        float* stat = mypart + R * C::kAccPad;
#pragma unroll
        for (int m = 0; m < NR; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int rr = row_at(m, r);
                if ((kTurned ? g : t4) == 0) stat[2 * rr] = mx[m][r], stat[2 * rr + 1] = sum[m][r];
                constexpr int N = D == 64 ? 8 : 16;  // channels in a row of this lane
#pragma unroll
                for (int cg = 0; cg < C::kSub; ++cg) {
                    if constexpr (kTurned) {
#pragma unroll
                        for (int n = 0; n < N; n += 4)
                            *reinterpret_cast<float4*>(mypart + rr * C::kAccPad + cg * 128 + N * g + n) =
                                make_float4(acc[m][cg * 8 + n / 2][r], acc[m][cg * 8 + n / 2][2 + r],
                                            acc[m][cg * 8 + n / 2 + 1][r], acc[m][cg * 8 + n / 2 + 1][2 + r]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int ch = cg * 128 + N * (2 * t4 + j);
#pragma unroll
                            for (int n = 0; n < N; n += 4)
                                *reinterpret_cast<float4*>(mypart + rr * C::kAccPad + ch + n) =
                                    make_float4(acc[m][cg * 16 + n][2 * r + j], acc[m][cg * 16 + n + 1][2 * r + j],
                                                acc[m][cg * 16 + n + 2][2 * r + j], acc[m][cg * 16 + n + 3][2 * r + j]);
                        }
                    }
                }
            }
    }
    __syncthreads();
    for (int r = warp; r < my_rows; r += kDecWarps) {
        float m4[kDecWarps], top = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            m4[w] = part[w * kPartWarp + R * C::kAccPad + 2 * r];
            top = fmaxf(top, m4[w]);
        }
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            m4[w] = ptx::ex2_approx(m4[w] - ref);
            l = fmaf(part[w * kPartWarp + R * C::kAccPad + 2 * r + 1], m4[w], l);
        }
        const float inv = p.in_cluster ? 1.f : l != 0.f ? 1.f / l : 0.f;  // (NaN stays)
        const float lse2 = p.in_cluster ? 0.f : l != 0.f ? top - kWeightShift + log2f(l) : -INFINITY;
        const int pr = r0 + r, i = pr / p.G, hq = h * p.G + pr - i * p.G;
        const long long tok = q0 + i;
        const long long grow = tok * p.Hq + hq;
        // a part of the row's result: its place in the workspace
        const long long at = EVEN ? (2ll * blockIdx.x + (first > 0 ? 0 : 1)) * R + r : grow * p.splits + split;
        const bool partial = EVEN ? !whole : p.splits > 1;
        for (int c = lane * 4; c < p.d; c += 128) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(part + w * kPartWarp + r * C::kAccPad + c);
                o.x = fmaf(x.x, m4[w], o.x), o.y = fmaf(x.y, m4[w], o.y);
                o.z = fmaf(x.z, m4[w], o.z), o.w = fmaf(x.w, m4[w], o.w);
            }
            o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
            if (p.in_cluster)
                *reinterpret_cast<float4*>(smem + kJoin + (r * D + c) * 4) = o;
            else if (partial)
                *reinterpret_cast<float4*>(p.o_part + at * p.d + c) = o;
            else
                *reinterpret_cast<uint2*>(p.o + tok * p.o_st + static_cast<long long>(hq) * p.o_sh + c) =
                    make_uint2(pack16(o.x, o.y, bf16), pack16(o.z, o.w, bf16));
        }
        if (lane == 0) {
            if (p.in_cluster)
                cta_stat[r] = make_float2(top, l);
            else if (partial)
                p.lse_part[at] = lse2;
            else
                p.lse[grow] = lse2 * 0.69314718055994531f;
        }
    }
    if constexpr (EVEN) {
        // the next unit's boxes may land where partial results were written and read
        ptx::fence_proxy_async_smem();
        __syncthreads();
        base += mine;
        continue;
    }
    if (!p.in_cluster) return;

    // ---- join the cluster's CTAs: each takes its share of the block's outputs
    // from all of them
    cluster_sync();
    // S lanes share four channels of a row, one for each CTA's result
    const int S = p.splits, n4 = p.d >> 2, n = my_rows * n4, from = tid & (S - 1);
    for (int i0 = 0; i0 < n; i0 += kDecThreads) {
        const int i = i0 + (split * kDecThreads + tid) / S;
        float2 st = make_float2(-INFINITY, 0.f);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const int r = min(i, n - 1) / n4, c = (min(i, n - 1) - r * n4) * 4;
        if (i < n) {
            st = ld_cluster_f2(ptx::smem_addr(&cta_stat[r]), from);
            o = ld_cluster_f4(sbase + kJoin + (r * D + c) * 4, from);
        }
        float top = st.x;
        for (int x = 1; x < S; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float w = ptx::ex2_approx(st.x - (top == -INFINITY ? 0.f : top));
        float l = st.y * w;
        o.x *= w, o.y *= w, o.z *= w, o.w *= w;
        for (int x = 1; x < S; x *= 2) {
            l += __shfl_xor_sync(0xffffffffu, l, x);
            o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
            o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
        }
        if (i >= n || from != 0) continue;
        const float inv = l != 0.f ? 1.f / l : 0.f;
        const int pr = r0 + r, iq = pr / p.G, hq = h * p.G + pr - iq * p.G;
        const long long tok = q0 + iq;
        *reinterpret_cast<uint2*>(p.o + tok * p.o_st + static_cast<long long>(hq) * p.o_sh + c) =
            make_uint2(pack16(o.x * inv, o.y * inv, bf16), pack16(o.z * inv, o.w * inv, bf16));
        if (c == 0)
            p.lse[tok * p.Hq + hq] = l != 0.f ? (top - kWeightShift + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    cluster_sync();  // the others have read this CTA's results
    } while (EVEN);
}

// Joins the parts of a unit that shares cut: CTA i - 1 of this grid looks at
// the boundary before share i, and takes the unit if it is the first in it.
// A warp takes a row at a time: lane j the weight of part j, four channels of every part.
constexpr int kJoinThreads = 256;
template <int R>
__global__ void __launch_bounds__(kJoinThreads) paged_even_join_kernel(const PagedParams p, const bool bf16) {
    dependents_may_start();
    wait_for_previous();
    const int G = static_cast<int>(gridDim.x) + 1, i = blockIdx.x + 1, lane = threadIdx.x & 31;
    const int4 unit = ld(p.shares + i);  // first chunk, last + 1, request, head
    const int share = ld(p.shares + G).x;
    const long long at = static_cast<long long>(i) * share;
    if (unit.x >= at || unit.y <= at || at - share > unit.x) return;
    // share i - 1's last unit, then the first ones of the shares that begin inside
    const int parts = 1 + static_cast<int>(min(static_cast<long long>(G - i), (unit.y - at + share - 1) / share));
    auto slot = [&](int j) { return j == 0 ? 2ll * (i - 1) + 1 : 2ll * (i + j - 1); };
    int q0, nq, len;
    bool bad = false;
    request_of(p, unit.z, q0, nq, len, bad);
    const int my_rows = min(R, nq * p.G);
    for (int r = threadIdx.x >> 5; r < my_rows; r += kJoinThreads / 32) {
        const int tok = q0 + r / p.G, hq = unit.w * p.G + r % p.G;
        for (int c0 = 0; c0 < p.d; c0 += 128) {
            const int c = c0 + lane * 4;
            float top = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j0 = 0; j0 < parts; j0 += 32) {
                const float a = j0 + lane < parts ? ld(p.lse_part + slot(j0 + lane) * R + r) : -INFINITY;
                float next = fmaxf(a, top);
#pragma unroll
                for (int x = 16; x; x >>= 1) next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, x));
                const float ref = next == -INFINITY ? 0.f : next, old = ptx::ex2_approx(top - ref);
                const float w = ptx::ex2_approx(a - ref);
                float sum = w;
#pragma unroll
                for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                top = next;
                l = fmaf(l, old, sum);
                o.x *= old, o.y *= old, o.z *= old, o.w *= old;
                const int n = min(32, parts - j0);
#pragma unroll 4
                for (int j = 0; j < n; ++j) {
                    const float wj = __shfl_sync(0xffffffffu, w, j);
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c < p.d) x = ld(reinterpret_cast<const float4*>(p.o_part + (slot(j0 + j) * R + r) * p.d + c));
                    o.x = fmaf(x.x, wj, o.x), o.y = fmaf(x.y, wj, o.y), o.z = fmaf(x.z, wj, o.z), o.w = fmaf(x.w, wj, o.w);
                }
            }
            const float inv = l != 0.f ? 1.f / l : 0.f;
            if (c < p.d)
                *reinterpret_cast<uint2*>(p.o + tok * p.o_st + hq * p.o_sh + c) =
                    make_uint2(pack16(o.x * inv, o.y * inv, bf16), pack16(o.z * inv, o.w * inv, bf16));
            if (c == 0) p.lse[static_cast<long long>(tok) * p.Hq + hq] = l != 0.f ? (top + log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
    }
}

// O = sum_s 2^(lse_s - lse) O_s, LSE = log-sum over the ranges of a row.
// One warp per row of q.
constexpr int kMergeWarps = 4;
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const PagedParams p, const bool bf16) {
    dependents_may_start();
    wait_for_previous();
    const long long row = static_cast<long long>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long tok = row / p.Hq;
    const int hq = static_cast<int>(row - tok * p.Hq);
    // rows before the first query and behind the last were not computed
    if (tok >= p.T || (p.cu_q && (tok < ld_meta(p.cu_q) || tok >= ld_meta(p.cu_q + p.B)))) return;
    const float* ls = p.lse_part + row * p.splits;
    float a0 = lane < p.splits ? ld(ls + lane) : -INFINITY, a1 = lane + 32 < p.splits ? ld(ls + lane + 32) : -INFINITY;
    float top = fmaxf(a0, a1);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    a0 = ptx::ex2_approx(a0 - ref), a1 = ptx::ex2_approx(a1 - ref);
    float l = a0 + a1;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l != 0.f ? 1.f / l : 0.f;
    if (lane == 0) p.lse[row] = l != 0.f ? (top + log2f(l)) * 0.69314718055994531f : -INFINITY;
    const float* op = p.o_part + row * p.splits * p.d;
    for (int c0 = 0; c0 < p.d; c0 += 128) {
        const int c = c0 + lane * 4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < p.splits; ++s) {
            const float w = __shfl_sync(0xffffffffu, s < 32 ? a0 : a1, s & 31);
            if (w == 0.f || c >= p.d) continue;
            const float4 x = ld(reinterpret_cast<const float4*>(op + s * p.d + c));
            o.x = fmaf(x.x, w, o.x), o.y = fmaf(x.y, w, o.y), o.z = fmaf(x.z, w, o.z), o.w = fmaf(x.w, w, o.w);
        }
        if (c < p.d)
            *reinterpret_cast<uint2*>(p.o + tok * p.o_st + static_cast<long long>(hq) * p.o_sh + c) =
                make_uint2(pack16(o.x * inv, o.y * inv, bf16), pack16(o.z * inv, o.w * inv, bf16));
    }
}

}  // namespace paged
}  // namespace fa
