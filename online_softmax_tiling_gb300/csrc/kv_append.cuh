// kv_append.cuh - new keys and values quantised into their pages.
//
// Per page and head the scale is a power of two, s = 2^e with e the smallest
// exponent for which every finite |x| <= 448 s; code = round_e4m3(x / s).
// Dividing by a power of two is exact, so the only rounding is the one to
// e4m3, and a page whose scale grows is rounded again only where its codes
// fall below the normal range.
//
// A run is the tokens of one page that a call brings (consecutive rows, slots
// ascending by one); an item is one run of one head of K or of V.  A CTA looks
// through a chunk of slots, finds the runs that begin there and takes them for
// one (head, K or V); a run of a few tokens (a decode step) is one warp's item,
// a longer one is the CTA's.  Either way the team holds the item's 16-bit
// values in registers between the maximum and the rounding, so HBM is read
// once and written once.
// What bounds it: HBM for prompts (4 d bytes read and 2 d written per token
// and head), launch and two dependent reads for a decode step.
#pragma once

#include "paged_common.cuh"

namespace fa {
namespace paged {

constexpr int kAppendThreads = 256;
constexpr int kAppendMaxChunk = 64;  // slots a CTA looks through for beginnings of runs
constexpr int kAppendShortRows = 4;  // rows per thread of a one-warp item

struct AppendParams {
    const uint16_t* x[2];       // k, v: [T, Hk, d] 16-bit
    long long st[2], sh[2];     // token and head strides, elements
    uint8_t* codes[2];          // [num_pages, Hk, P, d]
    float* scale[2];            // [num_pages, Hk]
    int8_t* bounds;             // [num_pages, Hk, 2, d] or null (K only)
    const int* slots;
    int T, Hk, d, num_pages, page_shift, chunk;
};

// bounds of a code: floor and ceiling of code / 4 (NaN counts as 0)
__device__ __forceinline__ void code_bounds(float c, int& lo, int& hi) {
    const float q = (c != c) ? 0.f : c * 0.25f;
    lo = min(lo, __float2int_rd(q));
    hi = max(hi, __float2int_ru(q));
}

// One item by a team of TH threads: n tokens from row t into place `place` of
// `page`.  NL: rows of the run each thread holds.
template <int TH, int NL, bool BF16>
__device__ __forceinline__ void append_item(const AppendParams& p, int t, int n, int page, int place,
                                            int h, int w, int tid, float* red, int* blo, int* bhi) {
    const int P = 1 << p.page_shift;
    auto sync = [] { if constexpr (TH == 32) __syncwarp(); else __syncthreads(); };
    const int LR = p.d >> 3;               // threads per row, 8 channels each
    const int rows = TH / LR;              // rows per pass
    const int r0 = tid / LR, c8 = (tid - r0 * LR) * 8;
    const bool on = r0 < rows;
    const uint16_t* src = p.x[w] + static_cast<long long>(t) * p.st[w] + static_cast<long long>(h) * p.sh[w] + c8;
    uint4 v[NL];
#pragma unroll
    for (int k = 0; k < NL; ++k) {
        const int r = r0 + k * rows;
        v[k] = make_uint4(0, 0, 0, 0);
        if (on && r < n) v[k] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<long long>(r) * p.st[w]));
    }
    const long long ph = static_cast<long long>(page) * p.Hk + h;
    const bool fresh = place == 0;
    const float old = fresh ? 0.f : p.scale[w][ph];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < NL; ++k) {
        const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack16(u[i], BF16);
            const float a = fabsf(f.x), b = fabsf(f.y);
            if (a < INFINITY) amax = fmaxf(amax, a);   // an infinity or NaN does not count
            if (b < INFINITY) amax = fmaxf(amax, b);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const bool with_bounds = w == 0 && p.bounds != nullptr;
    if constexpr (TH > 32) {
        if ((tid & 31) == 0) red[tid >> 5] = amax;
    }
    if (with_bounds)
        for (int c = tid; c < p.d; c += TH) blo[c] = 127, bhi[c] = -128;
    sync();
    if constexpr (TH > 32) {
#pragma unroll
        for (int i = 0; i < TH / 32; ++i) amax = fmaxf(amax, red[i]);
    }
    float s = pow2(cache_scale_exp(amax));
    if (old > s) s = old;                       // never shrinks while a page is in use
    const bool grown = !fresh && s > old;
    const float inv = 1.f / s;                  // exact: s is a power of two
    if (tid == 0) p.scale[w][ph] = s;
    uint8_t* base = p.codes[w] + (ph << p.page_shift) * p.d;
    if (grown) {  // the page's older codes, rounded again to the new scale
        const float ratio = old * inv;
        const int words = (place * p.d) >> 2;
        uint32_t* o4 = reinterpret_cast<uint32_t*>(base);
        for (int i = tid; i < words; i += TH) {
            const uint32_t c = o4[i];
            const float2 a = half2_floats(e4m3x2_to_half2(c & 0xFFFFu));
            const float2 b = half2_floats(e4m3x2_to_half2(c >> 16));
            const uint32_t lo = e4m3x2(a.x * ratio, a.y * ratio), hi = e4m3x2(b.x * ratio, b.y * ratio);
            o4[i] = lo | (hi << 16);
            if (with_bounds) {
                const int ch = (i * 4) % p.d;
                const float2 x = half2_floats(e4m3x2_to_half2(lo)), y = half2_floats(e4m3x2_to_half2(hi));
                const float f[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    int l = 127, m = -128;
                    code_bounds(f[e], l, m);
                    atomicMin(&blo[ch + e], l);
                    atomicMax(&bhi[ch + e], m);
                }
            }
        }
    }
    int lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) lo[e] = 127, hi[e] = -128;
#pragma unroll
    for (int k = 0; k < NL; ++k) {
        const int r = r0 + k * rows;
        if (!on || r >= n) continue;
        const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack16(u[i], BF16);
            q[i] = e4m3x2(f.x * inv, f.y * inv);
        }
        *reinterpret_cast<uint2*>(base + (place + r) * p.d + c8) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        if (with_bounds) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = half2_floats(e4m3x2_to_half2(q[i]));
                code_bounds(f.x, lo[2 * i], hi[2 * i]);
                code_bounds(f.y, lo[2 * i + 1], hi[2 * i + 1]);
            }
        }
    }
    if (with_bounds) {
        if (on && r0 < n) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                atomicMin(&blo[c8 + e], lo[e]);
                atomicMax(&bhi[c8 + e], hi[e]);
            }
        }
        sync();
        int8_t* bd = p.bounds + ph * 2 * p.d;
        const bool keep = !fresh && !grown;     // the older codes stand: so do their bounds
        for (int c = tid; c < p.d; c += TH) {
            int l = blo[c], m = bhi[c];
            if (keep) l = min(l, static_cast<int>(bd[c])), m = max(m, static_cast<int>(bd[p.d + c]));
            bd[c] = static_cast<int8_t>(l);
            bd[p.d + c] = static_cast<int8_t>(m);
        }
    }
    sync();  // the team's shared arrays are free again
    (void)P;
}

template <int NL, bool BF16>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
    constexpr int kWarps = kAppendThreads / 32;
    __shared__ uint32_t breaks[8];              // bit i: row t0 + i does not go on from the row before it
    __shared__ int n_short, n_long;
    __shared__ int short_runs[kAppendMaxChunk], long_runs[kAppendMaxChunk];  // row in the chunk | length << 8
    __shared__ float red[kWarps];
    __shared__ int blo[kWarps][256], bhi[kWarps][256];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = 1 << p.page_shift;
    const int t0 = blockIdx.x * p.chunk;
    if (tid == 0) n_short = 0, n_long = 0;
    dependents_may_start();
    wait_for_previous();
    // rows t0 .. t0 + 255: the chunk and what runs that begin in it may reach
    const int t = t0 + tid;
    const int slot = t < p.T ? __ldg(p.slots + t) : -1;
    int before = __shfl_up_sync(0xffffffffu, slot, 1);
    if (lane == 0) before = (t > 0 && t - 1 < p.T) ? __ldg(p.slots + t - 1) : -1;
    const bool same = slot >= 0 && before >= 0 && (slot >> p.page_shift) == (before >> p.page_shift);
    bool go_on = same && slot == before + 1;
    const uint32_t bits = __ballot_sync(0xffffffffu, !go_on);
    if (lane == 0) breaks[warp] = bits;
    __syncthreads();
    if (tid < p.chunk && slot >= 0 && !go_on) {
        const int page = slot >> p.page_shift, place = slot & (P - 1);
        if (same || page >= p.num_pages) {
            // the same page again, not in order, or no page of the cache: not stored
            report(kBadData);
        } else {
            int e = tid + 1;                    // first row after this one that breaks the run
            while (e < kAppendThreads) {
                const uint32_t m = breaks[e >> 5] >> (e & 31);
                if (m) { e += __ffs(m) - 1; break; }
                e = (e | 31) + 1;
            }
            const int n = min(e - tid, P - place);
            const int rows = 32 / (p.d >> 3);
            if (n <= kAppendShortRows * rows)
                short_runs[atomicAdd(&n_short, 1)] = tid | (n << 8);
            else
                long_runs[atomicAdd(&n_long, 1)] = tid | (n << 8);
        }
    }
    __syncthreads();
    const int h = blockIdx.y >> 1, w = blockIdx.y & 1;
    for (int i = 0; i < n_long; ++i) {
        const int row = long_runs[i] & 255, n = long_runs[i] >> 8;
        const int s = __ldg(p.slots + t0 + row);
        append_item<kAppendThreads, NL, BF16>(p, t0 + row, n, s >> p.page_shift, s & (P - 1), h, w, tid, red, blo[0], bhi[0]);
    }
    for (int i = warp; i < n_short; i += kWarps) {
        const int row = short_runs[i] & 255, n = short_runs[i] >> 8;
        const int s = __ldg(p.slots + t0 + row);
        append_item<32, kAppendShortRows, BF16>(p, t0 + row, n, s >> p.page_shift, s & (P - 1), h, w, lane, red, blo[warp], bhi[warp]);
    }
}

}  // namespace paged
}  // namespace fa
