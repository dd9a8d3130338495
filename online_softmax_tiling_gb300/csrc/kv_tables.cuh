// kv_tables.cuh - one serving step's bookkeeping: pages released and taken,
// and the slot of every new token.
//
// With have_b = ceil(len_b / P) pages held, need_b more to take and back_b to
// give back, three prefix sums over the requests place everything: tokens
// (cu), pages taken (pop) and pages released (push).  The i-th page taken is
// entry count + R - 1 - i of the stack after the R pushes; an entry at or
// above `count` is one of this step's pushes and is read from the row it
// comes from.  So no step waits for another's writes: every CTA computes the
// prefix sums for itself (B values, from L2), then takes its share of the
// three flat ranges (tokens, pages taken, pages released), and the whole step
// is one launch without a barrier between CTAs.  Inputs are never written:
// lens_out and free_count_out are other buffers, rows that are read (ended
// requests) are not rows that are written (growing requests), and pushes go
// to entries >= count while pops read entries < count.
//
// What bounds it: latency.  3.4 us on the GPU for 8 requests, 7.3 us for 1000 that
// bring 50 thousand tokens with ends and prompts among them, 5.6 us for 128 prompts of
// 340 thousand tokens (the write of the slots alone would be 0.2 us): two dependent
// reads, the prefix sums, the search for a token's request, its page, the write.  A
// token per thread (1024 a CTA) beat four (9.3 us for the second).
#pragma once

#include "paged_common.cuh"

namespace fa {
namespace paged {

constexpr int kTablesThreads = 1024;
constexpr int kTablesMaxB = 16384;
constexpr int kTablesKeptLens = 8192;  // requests whose lengths stay in shared memory

struct TablesParams {
    const int* new_tokens;
    const int* lens;
    int* table;
    int* free_pages;
    const int* free_count;
    int B, max_pages, free_capacity, page_shift, max_tokens;
    int* slots;
    int* cu;
    int* lens_out;
    int* free_count_out;
    int* status;
};

__global__ void __launch_bounds__(kTablesThreads) kv_tables_kernel(const TablesParams p) {
    extern __shared__ int tab_smem[];
    int* cu = tab_smem;                 // [B + 1] tokens before request b
    int* pop = cu + p.B + 1;            // [B + 1] pages taken before request b
    int* push = pop + p.B + 1;          // [B + 1] pages released before request b
    int* len_of = push + p.B + 1;       // [B] tokens held, where they fit
    const bool keep_lens = p.B <= kTablesKeptLens;
    __shared__ long long warp_sums[3][kTablesThreads / 32];
    __shared__ long long totals[3];
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P1 = (1 << p.page_shift) - 1;
    if (tid == 0) bad = 0;
    dependents_may_start();
    wait_for_previous();
    __syncthreads();

    auto request = [&](int b, int& add, int& need, int& back) {
        const int n = ld_meta(p.new_tokens + b), len = ld_meta(p.lens + b);
        if (keep_lens) len_of[b] = len;
        const long long after = static_cast<long long>(max(len, 0)) + max(n, 0);
        const long long have = (static_cast<long long>(max(len, 0)) + P1) >> p.page_shift;
        const long long want = (after + P1) >> p.page_shift;
        if (len < 0 || have > p.max_pages || (n >= 0 && want > p.max_pages)) {
            bad = 1;
            add = need = back = 0;
            return;
        }
        add = max(n, 0);
        need = n < 0 ? 0 : static_cast<int>(want - have);
        back = n < 0 ? static_cast<int>(have) : 0;
    };

    const int count = ld_meta(p.free_count);
    // each thread sums a run of consecutive requests, then the block scans the sums
    const int per = (p.B + kTablesThreads - 1) / kTablesThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long s[3] = {0, 0, 0};
    int add0 = 0, need0 = 0, back0 = 0;  // of the thread's first request, its only one up to 1024
    for (int b = b0; b < b1; ++b) {
        int add, need, back;
        request(b, add, need, back);
        if (b == b0) add0 = add, need0 = need, back0 = back;
        s[0] += add, s[1] += need, s[2] += back;
    }
    long long incl[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        long long x = s[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        incl[k] = x;
        if (lane == 31) warp_sums[k][warp] = x;
    }
    __syncthreads();
    if (warp < 3) {
        constexpr int W = kTablesThreads / 32;
        long long x = lane < W ? warp_sums[warp][lane] : 0;
        const long long own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane < W) warp_sums[warp][lane] = x - own;
        if (lane == 31) totals[warp] = x;
    }
    __syncthreads();
    const long long T = totals[0], A = totals[1], R = totals[2];
    int status = 0;
    if (bad || count < 0 || count + R > p.free_capacity || T > p.max_tokens)
        status = 1;  // FA_ERR_INVALID_ARG
    else if (A > count + R)
        status = 6;  // FA_ERR_NO_PAGES
    if (status == 0) {
        int run[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) run[k] = static_cast<int>(warp_sums[k][warp] + incl[k] - s[k]);
        for (int b = b0; b < b1; ++b) {
            int add = add0, need = need0, back = back0;
            if (b != b0) request(b, add, need, back);
            cu[b] = run[0], pop[b] = run[1], push[b] = run[2];
            run[0] += add, run[1] += need, run[2] += back;
        }
        if (tid == 0) cu[p.B] = static_cast<int>(T), pop[p.B] = static_cast<int>(A), push[p.B] = static_cast<int>(R);
    }
    __syncthreads();

    auto length = [&](int b) { return keep_lens ? len_of[b] : ld_meta(p.lens + b); };
    const long long stride = static_cast<long long>(gridDim.x) * kTablesThreads;
    const long long first = static_cast<long long>(blockIdx.x) * kTablesThreads + tid;
    if (status != 0) {
        for (long long i = first; i < p.max_tokens; i += stride) p.slots[i] = -1;
        for (long long b = first; b <= p.B; b += stride) p.cu[b] = 0;
        for (long long b = first; b < p.B; b += stride) p.lens_out[b] = length(b);
        if (first == 0) *p.free_count_out = count, *p.status = status;
        return;
    }
    // the page an entry of the stack holds after the pushes
    auto stack = [&](int i) {
        if (i < count) return ld_meta(p.free_pages + i);
        const int r = i - count, b = owner_of(push, p.B, r);
        return ld_meta(p.table + static_cast<long long>(b) * p.max_pages + (r - push[b]));
    };
    const int top = count + static_cast<int>(R) - 1;
    for (long long t = first; t < p.max_tokens; t += stride) {
        int slot = -1;
        if (t < T) {
            const int b = owner_of(cu, p.B, static_cast<int>(t));
            const int len = length(b);
            const int pos = len + static_cast<int>(t) - cu[b];
            const int j = pos >> p.page_shift, have = (len + P1) >> p.page_shift;
            const int page = j < have ? ld_meta(p.table + static_cast<long long>(b) * p.max_pages + j)
                                      : stack(top - (pop[b] + j - have));
            // (a larger number's slot would wrap to another page's)
            if (page < 0 || page > (0x7FFFFFFF >> p.page_shift))
                report(kBadData);
            else
                slot = (page << p.page_shift) | (pos & P1);
        }
        p.slots[t] = slot;
    }
    for (long long i = first; i < A; i += stride) {
        const int b = owner_of(pop, p.B, static_cast<int>(i));
        const int have = (length(b) + P1) >> p.page_shift;
        p.table[static_cast<long long>(b) * p.max_pages + have + (static_cast<int>(i) - pop[b])] =
            stack(top - static_cast<int>(i));
    }
    for (long long i = first; i < R; i += stride) p.free_pages[count + i] = stack(count + static_cast<int>(i));
    for (long long b = first; b < p.B; b += stride) {
        const int n = ld_meta(p.new_tokens + b);
        p.cu[b] = cu[b];
        p.lens_out[b] = n < 0 ? 0 : length(b) + n;
    }
    if (first == 0) {
        p.cu[p.B] = static_cast<int>(T);
        *p.free_count_out = count + static_cast<int>(R - A);
        *p.status = 0;
    }
}

}  // namespace paged
}  // namespace fa
