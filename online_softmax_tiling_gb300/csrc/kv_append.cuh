// kv_append.cuh - new keys and values quantised into their pages.
//
// Per page and head the scale is a power of two, s = 2^e with e the smallest
// exponent for which every finite |x| <= 448 s; code = round_e4m3(x / s).
// Dividing by a power of two is exact, so the only rounding is the one to
// e4m3, and a page whose scale grows is rounded again only where its codes
// fall below the normal range.
//
// A run is the tokens of one page that a call brings (slots ascending by one; rows
// left out may stand between them); an item is one run of one head of K or of V.  A
// CTA looks through a chunk of slots, finds the runs that begin there and takes them for
// one to four pairs of (head, K or V); a run of a few tokens (a decode step) is
// one warp's item, a longer one is the CTA's.  Either way the team holds the
// item's 16-bit values in registers between the maximum and the rounding, so HBM
// is read once and written once, and the CTA reads its next item meanwhile.
// What bounds it: HBM for prompts (4 d bytes read and 2 d written per token
// and head), launch and two dependent reads for a decode step.  45 thousand tokens of 8
// heads, d 128: 58.7 us, 5.2 TB/s; without the item read ahead and with 16 CTAs per
// chunk instead of 4 it was 109.  32 single tokens: 4.5 us.
// Rows left out between the tokens of a page must not split it into two runs, which would
// race on its scale: a CTA that meets such rows counts its tokens out first, and every row is
// looked up in shared memory.  Calls without them pay 0.2 us for it (57.4 and 4.3 us before),
// calls with them 2.3 us (32 requests padded to 16 rows: 4.7 before, 7.0); the search or all of
// the rest in a function of its own costs more (spills: 70 us).
#pragma once

#include "rotary.cuh"

namespace fa {
namespace paged {

constexpr int kAppendThreads = 256;
constexpr int kAppendMaxChunk = 64;  // slots a CTA looks through for beginnings of runs
constexpr int kAppendShortRows = 4;  // rows per thread of a one-warp item
constexpr int kAppendGap = 128;      // rows from a token to the next of its run, at most
constexpr int kAppendEntries = kAppendThreads + 128;  // stored rows of a window, and of a run that passes it

struct AppendParams {
    const uint16_t* x[2];       // k, v: [T, Hk, d] 16-bit
    long long st[2], sh[2];     // token and head strides, elements
    uint8_t* codes[2];          // [num_pages, Hk, P, d]
    float* scale[2];            // [num_pages, Hk]
    int8_t* bounds;             // [num_pages, Hk, 2, d] or null (K only)
    const int* slots;
    int T, Hk, d, num_pages, page_shift;
    int chunk;                  // slots a CTA looks through
    int pairs;                  // (head, K or V) pairs it takes
    // keys turned on their way (the ROT kernels): the table, the queries that are turned beside
    // them (T = 0: none) by the grid's rows from `pair_rows` on
    RotaryTable turn;
    RotaryWork q;
    int pair_rows;
};

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
__device__ __forceinline__ uint32_t as_bits(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
// bounds of a code: floor and ceiling of code / 4 (NaN counts as 0)
__device__ __forceinline__ void code_bounds(float c, int& lo, int& hi) {
    const float q = (c != c) ? 0.f : c * 0.25f;
    lo = min(lo, __float2int_rd(q));
    hi = max(hi, __float2int_ru(q));
}

struct AppendItem {
    int e, n, page, place;  // n tokens from the CTA's e-th into place `place` of `page`
    int h, w;               // head; K (0) or V (1)
};

// A thread's rows of an item, 16-bit values; where keys are turned also the channels that make pairs with them.  Turned
// values are fp32 (so that a key is rounded once, to e4m3), and for more rows than the registers hold of these,
// nothing is held: rows are read twice.  24.6 thousand tokens of 8 heads, d 128, half of the channels turned: 60 us for keys
// and values (39 unturned: the table's reads, and registers for two CTAs per SM; bounded to three CTAs they spill and it takes
// longer), and 95 for pages of 128 with d 256, which are read twice.
template <int NL, bool ROT>
struct AppendRows {
    uint4 v[NL];
};
template <int NL>
struct AppendRows<NL, true> {
    uint4 v[NL <= 4 ? NL : 1], other[NL <= 4 ? NL : 1];
};

// What a team of TH threads does with one item: load() its rows into registers,
// then store() them.  NL: rows of the run each thread holds.
template <int TH, int NL, bool BF16, bool BOUNDS, bool ROT>
struct AppendTeam {
    using Rows = AppendRows<NL, ROT>;
    static constexpr bool kReadTwice = ROT && NL > 4;
    const AppendParams& p;
    const int tid;
    const int* row_of;           // rows of the CTA's tokens
    const int* pos_of;           // ROT: their rows of the table, -1 where they are not turned
    const int LR, rows, r0, c8;  // threads per row (8 channels each), rows per pass, this thread's place
    const bool on;
    float* red;                  // team's shared memory: a value per warp,
    uint4* bred;                 //   least, then largest codes of a thread's rows (fp16 pairs),
    int *blo, *bhi;              //   bounds of a page's older codes

    __device__ AppendTeam(const AppendParams& p_, int tid_, const int* row_of_, const int* pos_of_, float* red_, uint4* bred_, int* blo_, int* bhi_)
        : p(p_), tid(tid_), row_of(row_of_), pos_of(pos_of_), LR(p_.d >> 3), rows(TH / LR), r0(tid / LR), c8((tid - r0 * LR) * 8), on(r0 < rows),
          red(red_), bred(bred_), blo(blo_), bhi(bhi_) {}

    __device__ static void sync() {
        if constexpr (TH == 32) __syncwarp(); else __syncthreads();
    }

    // Whether the thread's channels of this item are turned, and where their partners are (in the thread's own piece
    // where pairs are neighbours).
    __device__ bool turned(const AppendItem& m) const { return m.w == 0 && c8 < 2 * p.turn.half; }
    __device__ int partner() const { return c8 < p.turn.half ? c8 + p.turn.half : c8 - p.turn.half; }

    // 16-bit values of the thread's k-th row (of the item's first where it has none) and their partners.
    __device__ void fetch(const AppendItem& m, int k, uint4& v, uint4& other) const {
        const int r = r0 + k * rows;
        const uint16_t* x = (m.w ? p.x[1] : p.x[0]) + m.h * (m.w ? p.sh[1] : p.sh[0]) +
                            row_of[m.e + (on && r < m.n ? r : 0)] * (m.w ? p.st[1] : p.st[0]);
        v = ld(reinterpret_cast<const uint4*>(x + (on ? c8 : 0)));
        if (turned(m) && !p.turn.interleaved) other = ld(reinterpret_cast<const uint4*>(x + partner()));
    }

    // Rows k0 .. k0 + N - 1 in fp32, keys turned.  The table's loads are unconditional (its first row for a row that is not
    // turned), so that those of N rows are on their way at once.
    template <int N>
    __device__ void turn(const AppendItem& m, int k0, const uint4* v, const uint4* other, float (*f)[8]) const {
        const int half = p.turn.half;
        const bool pairs_here = p.turn.interleaved != 0, first = c8 < half, here = turned(m);
        float4 cs[N][2], sn[N][2];
        int at[N];
        if (here) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int r = r0 + (k0 + k) * rows;
                at[k] = pos_of[m.e + (on && r < m.n ? r : 0)];
                const float* row = p.turn.rows + static_cast<long long>(max(at[k], 0)) * (2 * half);
                const float4 *c = reinterpret_cast<const float4*>(row + (pairs_here ? c8 / 2 : first ? c8 : c8 - half)),
                             *s = reinterpret_cast<const float4*>(row + half + (pairs_here ? c8 / 2 : first ? c8 : c8 - half));
                cs[k][0] = ld(c), sn[k][0] = ld(s);
                if (!pairs_here) cs[k][1] = ld(c + 1), sn[k][1] = ld(s + 1);
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t a[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = unpack16(a[i], BF16);
                f[k][2 * i] = x.x, f[k][2 * i + 1] = x.y;
            }
            if (!here || at[k] < 0) continue;
            if (pairs_here) {
                const float c[4] = {cs[k][0].x, cs[k][0].y, cs[k][0].z, cs[k][0].w}, s[4] = {sn[k][0].x, sn[k][0].y, sn[k][0].z, sn[k][0].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = f[k][2 * i], y = f[k][2 * i + 1];
                    f[k][2 * i] = turn_first(x, y, c[i], s[i]), f[k][2 * i + 1] = turn_second(x, y, c[i], s[i]);
                }
            } else {
                const uint32_t b[4] = {other[k].x, other[k].y, other[k].z, other[k].w};
                const float c[8] = {cs[k][0].x, cs[k][0].y, cs[k][0].z, cs[k][0].w, cs[k][1].x, cs[k][1].y, cs[k][1].z, cs[k][1].w};
                const float s[8] = {sn[k][0].x, sn[k][0].y, sn[k][0].z, sn[k][0].w, sn[k][1].x, sn[k][1].y, sn[k][1].z, sn[k][1].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = unpack16(b[i], BF16);
                    const float x0 = f[k][2 * i], x1 = f[k][2 * i + 1];
                    f[k][2 * i] = first ? turn_first(x0, y.x, c[2 * i], s[2 * i]) : turn_second(y.x, x0, c[2 * i], s[2 * i]);
                    f[k][2 * i + 1] = first ? turn_first(x1, y.y, c[2 * i + 1], s[2 * i + 1]) : turn_second(y.y, x1, c[2 * i + 1], s[2 * i + 1]);
                }
            }
        }
    }

    // The k-th of this thread's rows in fp32 (`held`: all of them, turned).
    __device__ void values(const AppendItem& m, const Rows& v, int k, const float (*held)[8], float (&f)[8]) const {
        if constexpr (kReadTwice) {
            uint4 own, other = make_uint4(0, 0, 0, 0);
            float one[1][8];
            fetch(m, k, own, other);
            turn<1>(m, k, &own, &other, one);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = one[0][i];
        } else if constexpr (ROT) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = held[k][i];
        } else {
            const uint32_t u[4] = {v.v[k].x, v.v[k].y, v.v[k].z, v.v[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = unpack16(u[i], BF16);
                f[2 * i] = x.x, f[2 * i + 1] = x.y;
            }
        }
    }

    __device__ void load(const AppendItem& m, Rows& rows16, float& old) const {
        old = m.place == 0 ? 0.f : (m.w ? p.scale[1] : p.scale[0])[static_cast<long long>(m.page) * p.Hk + m.h];
        if constexpr (kReadTwice) {
        } else if constexpr (ROT) {
#pragma unroll
            for (int k = 0; k < NL; ++k) {
                // (a decode step's one-warp items have one row: the others are not read)
                if constexpr (TH == 32) rows16.v[k] = rows16.other[k] = make_uint4(0, 0, 0, 0);
                if (TH > 32 || k * rows < m.n) fetch(m, k, rows16.v[k], rows16.other[k]);
            }
        } else {
            load16(m, rows16.v);
        }
    }

    __device__ void load16(const AppendItem& m, uint4 (&v)[NL]) const {
        // (selected, not indexed: the parameters stay in constant memory)
        const long long st = m.w ? p.st[1] : p.st[0];
        const uint16_t* src = (m.w ? p.x[1] : p.x[0]) + m.h * (m.w ? p.sh[1] : p.sh[0]) + c8;
        // Many rows a thread: where none is left out their addresses come from one row's (45K
        // tokens, P 128, d 128: 99 us; 189 with every row looked up).
        const int first = row_of[m.e];
        if (NL > 4 && row_of[m.e + m.n - 1] - first == m.n - 1) {
            const uint16_t* at = src + first * st;
#pragma unroll
            for (int k = 0; k < NL; ++k) {
                const int r = r0 + k * rows;
                v[k] = make_uint4(0, 0, 0, 0);
                if (on && r < m.n) v[k] = ld(reinterpret_cast<const uint4*>(at + r * st));
            }
        } else {
#pragma unroll
            for (int k = 0; k < NL; ++k) {
                const int r = r0 + k * rows;
                v[k] = make_uint4(0, 0, 0, 0);
                if (on && r < m.n) v[k] = ld(reinterpret_cast<const uint4*>(src + row_of[m.e + r] * st));
            }
        }
    }

    __device__ void store(const AppendItem& m, const Rows& v, float old) const {
        float amax = 0.f;
        float held[ROT && !kReadTwice ? NL : 1][8];
        if constexpr (ROT && !kReadTwice) {
#pragma unroll
            for (int k = 0; k < NL; k += 2)
                if (TH > 32 || k * rows < m.n) turn<2>(m, k, v.v + k, v.other + k, held + k);
        }
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            if (ROT && !(on && r0 + k * rows < m.n)) continue;  // (else they are zeros)
            float f[8];
            values(m, v, k, held, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (fabsf(f[i]) < INFINITY) amax = fmaxf(amax, fabsf(f[i]));  // an infinity or NaN does not count
        }
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // (not negative)
        if constexpr (TH > 32) {
            if ((tid & 31) == 0) red[tid >> 5] = amax;
            sync();
#pragma unroll
            for (int i = 0; i < TH / 32; ++i) amax = fmaxf(amax, red[i]);
        }
        float s = pow2(cache_scale_exp(amax));
        if (old > s) s = old;                        // never shrinks while a page is in use
        const bool fresh = m.place == 0, grown = !fresh && s > old;
        const float inv = 1.f / s;                   // exact: s is a power of two
        const long long ph = static_cast<long long>(m.page) * p.Hk + m.h;
        if (tid == 0) (m.w ? p.scale[1] : p.scale[0])[ph] = s;
        uint8_t* base = (m.w ? p.codes[1] : p.codes[0]) + (ph << p.page_shift) * p.d;
        const bool with_bounds = BOUNDS && m.w == 0;
        if (grown) round_older(m, base, old * inv, with_bounds);
        __half2 lo[4], hi[4];  // of the new codes, channels 2 e and 2 e + 1 (NaN as 0)
        if constexpr (BOUNDS) {
#pragma unroll
            for (int e = 0; e < 4; ++e) lo[e] = __float2half2_rn(INFINITY), hi[e] = __float2half2_rn(-INFINITY);
        }
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            const int r = r0 + k * rows;
            if (!on || r >= m.n) continue;
            float f[8];
            values(m, v, k, held, f);
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = e4m3x2(f[2 * i] * inv, f[2 * i + 1] * inv);
            *reinterpret_cast<uint2*>(base + (m.place + r) * p.d + c8) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
            if (with_bounds) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t c = e4m3x2_to_half2(q[i]);
                    c &= __heq2_mask(as_half2(c), as_half2(c));
                    lo[i] = __hmin2(lo[i], as_half2(c));
                    hi[i] = __hmax2(hi[i], as_half2(c));
                }
            }
        }
        if (with_bounds) {
            bred[2 * tid] = make_uint4(as_bits(lo[0]), as_bits(lo[1]), as_bits(lo[2]), as_bits(lo[3]));
            bred[2 * tid + 1] = make_uint4(as_bits(hi[0]), as_bits(hi[1]), as_bits(hi[2]), as_bits(hi[3]));
            sync();
            // a thread takes the floors or the ceilings of two channels
            const int have = min(rows, m.n);
            for (int i = tid; i < p.d; i += TH) {
                const bool top = i >= p.d / 2;
                const int c2 = top ? i - p.d / 2 : i;  // channels 2 c2, 2 c2 + 1
                const uint32_t* col = reinterpret_cast<const uint32_t*>(bred + 2 * (c2 >> 2) + top) + (c2 & 3);
                __half2 x = as_half2(col[0]);
                for (int r = 1; r < have; ++r) {
                    const __half2 y = as_half2(col[r * LR * 8]);
                    x = top ? __hmax2(x, y) : __hmin2(x, y);
                }
                const float2 f = __half22float2(x);
                int a = top ? __float2int_ru(f.x * 0.25f) : __float2int_rd(f.x * 0.25f);
                int b = top ? __float2int_ru(f.y * 0.25f) : __float2int_rd(f.y * 0.25f);
                int8_t* at = p.bounds + ph * 2 * p.d + (top ? p.d : 0) + 2 * c2;
                if (!fresh) {
                    // the older codes': as they stand, or as rounded again
                    int c, d;
                    if (grown) {
                        c = (top ? bhi : blo)[2 * c2], d = (top ? bhi : blo)[2 * c2 + 1];
                    } else {
                        const char2 o = *reinterpret_cast<const char2*>(at);
                        c = o.x, d = o.y;
                    }
                    a = top ? max(a, c) : min(a, c), b = top ? max(b, d) : min(b, d);
                }
                *reinterpret_cast<char2*>(at) = make_char2(static_cast<signed char>(a), static_cast<signed char>(b));
            }
        }
        sync();  // the team's shared memory is free again
    }

    // The page's older codes (places before the first one written), rounded again.
    __device__ void round_older(const AppendItem& m, uint8_t* base, float ratio, bool with_bounds) const {
        if (with_bounds) {
            for (int c = tid; c < p.d; c += TH) blo[c] = 127, bhi[c] = -128;
            sync();
        }
        uint32_t* o4 = reinterpret_cast<uint32_t*>(base);
        for (int i = tid; i < (m.place * p.d) >> 2; i += TH) {
            const uint32_t c = o4[i];
            const float2 a = half2_floats(e4m3x2_to_half2(c & 0xFFFFu));
            const float2 b = half2_floats(e4m3x2_to_half2(c >> 16));
            const uint32_t l = e4m3x2(a.x * ratio, a.y * ratio), h = e4m3x2(b.x * ratio, b.y * ratio);
            o4[i] = l | (h << 16);
            if (with_bounds) {
                const int ch = (i * 4) % p.d;
                const float2 x = half2_floats(e4m3x2_to_half2(l)), y = half2_floats(e4m3x2_to_half2(h));
                const float f[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    int lo = 127, hi = -128;
                    code_bounds(f[e], lo, hi);
                    atomicMin(&blo[ch + e], lo);
                    atomicMax(&bhi[ch + e], hi);
                }
            }
        }
        if (with_bounds) sync();
    }
};

template <int NL, bool BF16, bool BOUNDS, bool ROT>
__global__ void __launch_bounds__(kAppendThreads, NL == 4 && !ROT ? 4 : 2) kv_append_kernel(const AppendParams p) {
    constexpr int kWarps = kAppendThreads / 32;
    __shared__ uint32_t breaks[kAppendEntries / 32];  // bit e: token e does not go on from the one before it
    __shared__ int n_short, n_long;
    __shared__ int2 short_runs[kAppendMaxChunk], long_runs[kAppendMaxChunk];  // first token | length << 8, slot
    __shared__ int row_of[kAppendEntries];      // rows of the tokens
    __shared__ int pos_of[ROT ? kAppendEntries : 1];
    __shared__ float red[kWarps];
    __shared__ uint4 bred[BOUNDS ? 2 * kAppendThreads : 1];
    __shared__ int blo[BOUNDS ? kWarps : 1][256], bhi[BOUNDS ? kWarps : 1][256];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = 1 << p.page_shift;
    const int t0 = blockIdx.x * p.chunk;
    if (tid == 0) n_short = 0, n_long = 0;
    dependents_may_start();
    wait_for_previous();
    if constexpr (ROT) {
        if (static_cast<int>(blockIdx.y) >= p.pair_rows) {  // queries
            const unsigned items = static_cast<unsigned>(p.q.T) * static_cast<unsigned>(p.q.groups * (p.q.cols + p.q.tail));
            const unsigned long long step = 1ull * gridDim.x * (gridDim.y - p.pair_rows) * kAppendThreads;
            for (unsigned long long i = (1ull * (blockIdx.y - p.pair_rows) * gridDim.x + blockIdx.x) * kAppendThreads + tid; i < items; i += step)
                rotary_item<1, BF16>(p.q, static_cast<unsigned>(i));
            return;
        }
    }
    // rows t0 .. t0 + 255: the chunk and what runs that begin in it may reach
    const int t = t0 + tid;
    int slot = t < p.T ? ld_meta(p.slots + t) : -1;
    int edge = -1, position = -1;
    if (lane == 0 && t > 0 && t - 1 < p.T) edge = ld_meta(p.slots + t - 1);
    if constexpr (ROT) position = t < p.T ? ld_meta(p.turn.positions + t) : -1;
    int before = __shfl_up_sync(0xffffffffu, slot, 1);
    if (lane == 0) before = edge;
    if constexpr (ROT) position = rotary_row(p.turn, position);
    bool same = slot >= 0 && before >= 0 && (slot >> p.page_shift) == (before >> p.page_shift);
    bool go_on = same && slot == before + 1;
    const uint32_t new_run = __ballot_sync(0xffffffffu, !go_on);
    if (lane == 0) breaks[warp] = new_run;
    row_of[tid] = t;
    if constexpr (ROT) pos_of[tid] = position;
    // Tokens are numbered from the chunk's start.  Mostly that is their row, and a token goes on
    // from the row above; where one stands behind rows left out, or a run may pass the end of
    // the window over such rows, they are counted out.
    const bool left_out = slot >= 0 ? before < 0 && t > 0 : before >= 0 && tid > kAppendGap && t0 + kAppendThreads < p.T;
    const bool sparse = __syncthreads_or(left_out);
    int row = t, limit = kAppendThreads;
    if (sparse) {
        __shared__ int slot_of[kAppendEntries];
        __shared__ uint32_t stored[kWarps], marks[kWarps];
        __shared__ int back_slot[kAppendGap / 32], back_row[kAppendGap / 32];
        const uint32_t below = (1u << lane) - 1u;
        auto rank_of_row = [&] {
            int n = __popc(stored[warp] & below);
            for (int w = 0; w < warp; ++w) n += __popc(stored[w]);
            return n;
        };
        auto count = [&] {
            int n = 0;
            for (int w = 0; w < kWarps; ++w) n += __popc(stored[w]);
            return n;
        };
        const uint32_t here = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) stored[warp] = here;
        if (warp < kAppendGap / 32) {  // the last token of the rows before the chunk
            const int at = t0 - kAppendGap + tid, s = at >= 0 ? ld_meta(p.slots + at) : -1;
            const uint32_t has = __ballot_sync(0xffffffffu, s >= 0);
            if (lane == 0) back_row[warp] = -1;  // none
            __syncwarp();
            if (has && lane == 31 - __clz(has)) back_slot[warp] = s, back_row[warp] = at;
        }
        __syncthreads();
        const int rank = rank_of_row(), tokens = count();
        if (slot >= 0) slot_of[rank] = slot, row_of[rank] = t;
        if constexpr (ROT) {
            if (slot >= 0) pos_of[rank] = position;
        }
        if (tid < kAppendEntries / 32 - kWarps) breaks[kWarps + tid] = 0;
        __syncthreads();
        slot = -1, before = -1;
        if (tid < tokens) {
            slot = slot_of[tid], row = row_of[tid];
            int row_before = 0;
            if (tid > 0) {
                before = slot_of[tid - 1], row_before = row_of[tid - 1];
            } else {
#pragma unroll
                for (int w = 0; w < kAppendGap / 32; ++w)
                    if (back_row[w] >= 0) before = back_slot[w], row_before = back_row[w];
            }
            if (row - row_before > kAppendGap) before = -1;
        }
        same = slot >= 0 && before >= 0 && (slot >> p.page_shift) == (before >> p.page_shift);
        go_on = same && slot == before + 1;
        const uint32_t bits = __ballot_sync(0xffffffffu, slot >= 0 && !go_on);
        if (lane == 0) breaks[warp] = bits;
        __syncthreads();
        // the last run's tokens behind the window, if it begins in the chunk
        limit = tokens;
        int begin = -1;
        for (int w = 0; w < kWarps; ++w)
            if (breaks[w]) begin = 32 * w + 31 - __clz(breaks[w]);
        if (begin >= 0 && row_of[begin] < t0 + p.chunk) {
            for (int u = t0 + kAppendThreads; u < p.T; u += kAppendThreads) {
                const int last = slot_of[limit - 1], left = P - 1 - (last & (P - 1));  // places of the page that are left
                if (left == 0 || u - row_of[limit - 1] > kAppendGap) break;
                const int s = u + tid < p.T ? ld_meta(p.slots + u + tid) : -1;
                const uint32_t has = __ballot_sync(0xffffffffu, s >= 0);
                __syncthreads();
                if (lane == 0) stored[warp] = has;
                __syncthreads();
                const int at = rank_of_row(), all = count();
                if (s >= 0 && at < left) {
                    slot_of[limit + at] = s, row_of[limit + at] = u + tid;
                    if constexpr (ROT) pos_of[limit + at] = rotary_position(p.turn, u + tid);
                }
                __syncthreads();
                const int i = limit + tid;
                const bool goes_on = tid < min(all, left) && slot_of[i] == last + 1 + tid && row_of[i] - row_of[i - 1] <= kAppendGap;
                const uint32_t ends = __ballot_sync(0xffffffffu, !goes_on);
                if (lane == 0) marks[warp] = ends;
                __syncthreads();
                int more = 0;  // (at most 127 < kAppendThreads go on)
                while (marks[more >> 5] == 0) more += 32;
                more += __ffs(marks[more >> 5]) - 1;
                limit += more;
                if (more < all) break;
            }
        }
    }
    if (slot >= 0 && row < t0 + p.chunk && !go_on) {
        const int page = slot >> p.page_shift, place = slot & (P - 1);
        if (same || page >= p.num_pages) {
            // the same page again, not in order, or no page of the cache: not stored
            report(kBadData);
        } else {
            int e = tid + 1;                    // first token after this one that breaks the run
            while (e < limit) {
                const uint32_t m = breaks[e >> 5] >> (e & 31);
                if (m) { e += __ffs(m) - 1; break; }
                e = (e | 31) + 1;
            }
            const int n = min(min(e, limit) - tid, P - place);
            const int rows = 32 / (p.d >> 3);
            if (n <= kAppendShortRows * rows)
                short_runs[atomicAdd(&n_short, 1)] = make_int2(tid | (n << 8), slot);
            else
                long_runs[atomicAdd(&n_long, 1)] = make_int2(tid | (n << 8), slot);
        }
    }
    __syncthreads();
    // items: (run, pair) of the lists and the CTA's pairs
    const int pair0 = blockIdx.y * p.pairs, pairs = min(p.pairs, 2 * p.Hk - pair0);
    auto item = [&](const int2* runs, int i) {
        const int run = i / pairs, pair = pair0 + i - run * pairs;
        const int2 r = runs[run];
        return AppendItem{r.x & 255, r.x >> 8, r.y >> p.page_shift, r.y & (P - 1), pair >> 1, pair & 1};
    };
    if (n_long > 0) {
        const AppendTeam<kAppendThreads, NL, BF16, BOUNDS, ROT> team(p, tid, row_of, pos_of, red, bred, blo[0], bhi[0]);
        const int items = n_long * pairs;
        if constexpr (NL <= 4) {  // the next item is read while this one is stored
            AppendRows<NL, ROT> v, next;
            float old, next_old = 0.f;
            AppendItem m = item(long_runs, 0);
            team.load(m, v, old);
            for (int i = 0; i < items; ++i) {
                AppendItem nm = m;
                if (i + 1 < items) {
                    nm = item(long_runs, i + 1);
                    team.load(nm, next, next_old);
                }
                team.store(m, v, old);
                m = nm, old = next_old;
                v = next;
            }
        } else {
            for (int i = 0; i < items; ++i) {
                const AppendItem m = item(long_runs, i);
                AppendRows<NL, ROT> v;
                float old;
                team.load(m, v, old);
                team.store(m, v, old);
            }
        }
    }
    if (n_short > 0) {
        const int w = BOUNDS ? warp : 0;
        const AppendTeam<32, kAppendShortRows, BF16, BOUNDS, ROT> team(p, lane, row_of, pos_of, red, bred + (BOUNDS ? 64 * warp : 0), blo[w], bhi[w]);
        for (int i = warp; i < n_short * pairs; i += kWarps) {
            const AppendItem m = item(short_runs, i);
            AppendRows<kAppendShortRows, ROT> v;
            float old;
            team.load(m, v, old);
            team.store(m, v, old);
        }
    }
}

}  // namespace paged
}  // namespace fa
