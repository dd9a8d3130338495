// latent_append.cuh - a token's latent vector and its turned key part into a row of the paged
// latent cache [pages, P, C + R], and the queries' R channels turned beside it.
//
// What bounds it: HBM for prompts (4 (C + R) bytes per token, 4 H R for the queries), one launch and two
// dependent reads (position, then the table's row) for a decode step.  The first CTAs take 8-channel
// pieces of the cache's rows, a piece a thread, the others the queries.  18 thousand tokens with 16 heads' queries: 26 us, 4.7 TB/s,
// of which some 4 us are start and end; 16384 with 128 heads 91.5, 6.3 TB/s; 64 tokens with 128 heads 2.3 us in a graph.
#pragma once

#include "rotary.cuh"

namespace fa {
namespace paged {

struct LatentAppendParams {
    const uint16_t* latent;
    const uint16_t* rope;
    long long latent_st, rope_st;  // token strides, elements
    uint16_t* cache;
    const int* slots;
    RotaryTable r;                 // rows null: the key part is stored as it is
    RotaryWork q;                  // T = 0: none
    int T, C, R, num_slots;
    int latent_ctas;
};

template <int U, bool BF16>
__global__ void __launch_bounds__(kRotaryThreads) latent_append_kernel(const LatentAppendParams p) {
    dependents_may_start();
    wait_for_previous();
    if (static_cast<int>(blockIdx.x) >= p.latent_ctas) {
        const unsigned item = (blockIdx.x - p.latent_ctas) * static_cast<unsigned>(kRotaryThreads) + threadIdx.x;
        if (item < static_cast<unsigned>(p.q.T) * static_cast<unsigned>(p.q.groups * (p.q.cols + p.q.tail))) rotary_item<U, BF16>(p.q, item);
        return;
    }
    // pieces of a row: C / 8 copied, then R / 16 turned (two of 8 channels each) or R / 8 copied
    const unsigned copied = p.C >> 3, width = copied + (p.r.rows ? p.R >> 4 : p.R >> 3);
    const unsigned item = blockIdx.x * static_cast<unsigned>(kRotaryThreads) + threadIdx.x, token = item / width, col = item - token * width;
    if (token >= static_cast<unsigned>(p.T)) return;
    // (the slot is needed for the store alone: it is read beside the row's piece, not before it)
    const int slot = ld_meta(p.slots + token), at = static_cast<int>(col - copied);
    const bool turned = at >= 0 && p.r.rows;
    const uint16_t* src = at < 0 ? p.latent + token * p.latent_st : p.rope + token * p.rope_st;
    const int c0 = at < 0 ? col * 8 : !turned ? at * 8 : p.r.interleaved ? at * 16 : at * 8;
    const int c1 = turned ? p.r.interleaved ? c0 + 8 : c0 + p.r.half : c0;
    uint4 u = ld(reinterpret_cast<const uint4*>(src + c0)), v = u;
    if (turned) {
        v = ld(reinterpret_cast<const uint4*>(src + c1));
        if (const int row_at = slot < 0 ? -1 : rotary_position(p.r, token); row_at >= 0) {
            const float* row = p.r.rows + static_cast<long long>(row_at) * p.R;
            float c[8], s[8];
            load_floats8(row + at * 8, c);
            load_floats8(row + p.r.half + at * 8, s);
            turn16(u, v, c, s, p.r.interleaved != 0, BF16);
        }
    }
    if (slot >= p.num_slots) report(kBadData);
    if (slot < 0 || slot >= p.num_slots) return;
    uint16_t* dst = p.cache + static_cast<long long>(slot) * (p.C + p.R) + (at < 0 ? 0 : p.C);
    *reinterpret_cast<uint4*>(dst + c0) = u;
    if (turned) *reinterpret_cast<uint4*>(dst + c1) = v;
}

}  // namespace paged
}  // namespace fa
