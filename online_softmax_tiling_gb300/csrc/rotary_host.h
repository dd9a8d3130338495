// rotary_host.h - checks and kernel parameters of the structures of include/fa_rotary.h.
#pragma once

#include "../../include/fa.h"
#include "../../include/fa_rotary.h"
#include "host_common.h"
#include "rotary.cuh"

namespace {

namespace pg = fa::paged;

// d: head width that the turned channels are of; T: tokens.
int check_rotary(const fa_rotary* r, int d, int T) {
    if (!r || r->num_positions < 1 || (T > 0 && (!r->table || !r->positions))) return FA_ERR_INVALID_ARG;
    if (r->dim < 16 || r->dim > 512 || r->dim % 16 != 0 || r->dim > d) return FA_ERR_UNSUPPORTED;
    return misaligned(r->table, 16) || misaligned(r->positions, 4) ? FA_ERR_MISALIGNED : FA_OK;
}
int check_part(const fa_rotary_part* p, int T) {
    if ((T > 0 && (!p->x || !p->y)) || p->heads < 1) return FA_ERR_INVALID_ARG;
    if (bad_strides(p->x_stride) || bad_strides(p->y_stride) || misaligned(p->x, 16) || misaligned(p->y, 16)) return FA_ERR_MISALIGNED;
    // in place with other strides, one token or head would be written where another is read
    if (T > 0 && p->x == p->y && ((T > 1 && p->x_stride[0] != p->y_stride[0]) || (p->heads > 1 && p->x_stride[1] != p->y_stride[1])))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}
pg::RotaryTable rotary_table(const fa_rotary& r) {
    return {r.table, r.positions, r.num_positions, r.dim / 2, r.interleaved != 0, r.inverse != 0};
}
// Work of one part or two (groups is left to the caller).
pg::RotaryWork rotary_work(const fa_rotary& r, const fa_rotary_part* q, const fa_rotary_part* k, int T, int d) {
    pg::RotaryWork w = {};
    w.r = rotary_table(r);
    bool in_place = true;
    const fa_rotary_part* parts[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        const fa_rotary_part* p = parts[i];
        if (!p) continue;
        w.part[i] = {static_cast<const uint16_t*>(p->x), static_cast<uint16_t*>(p->y), p->x_stride[0], p->x_stride[1],
                     p->y_stride[0], p->y_stride[1], p->heads};
        in_place = in_place && p->x == p->y;
    }
    w.T = T;
    w.cols = r.dim / 16;
    w.tail = in_place ? 0 : (d - r.dim + 15) / 16;
    w.d = d;
    return w;
}

// Heads per item: two have twice the bytes on their way and read the table half as often (16000 tokens of 40 heads of 128: 50.5 us,
// with one 59.2, with four 52.9; 16384 latents with 128 heads' queries 91.5, with one 101.7); one, where there are too few
// items to fill the SMs.
[[maybe_unused]] int set_groups(pg::RotaryWork& w) {
    const int heads = w.part[0].heads + w.part[1].heads;
    const bool single = static_cast<int64_t>(w.T) * heads * (w.cols + w.tail) < 4ll * 2048 * sm_count();
    w.groups = single ? heads : (heads + pg::kRotaryHeads - 1) / pg::kRotaryHeads;
    return single ? 1 : pg::kRotaryHeads;
}
// The launch that turns them.
[[maybe_unused]] int launch_rotary(pg::RotaryWork w, bool bf16, void* stream) {
    const bool single = set_groups(w) == 1;
    const int64_t items = static_cast<int64_t>(w.T) * w.groups * (w.cols + w.tail);
    if (items > INT32_MAX) return FA_ERR_INVALID_ARG;
    const void* fn = single ? (bf16 ? reinterpret_cast<const void*>(&pg::rotary_kernel<1, true>) : reinterpret_cast<const void*>(&pg::rotary_kernel<1, false>))
                            : (bf16 ? reinterpret_cast<const void*>(&pg::rotary_kernel<pg::kRotaryHeads, true>)
                                    : reinterpret_cast<const void*>(&pg::rotary_kernel<pg::kRotaryHeads, false>));
    void* args[] = {&w};
    return launch(fn, (items + pg::kRotaryThreads - 1) / pg::kRotaryThreads, 1, pg::kRotaryThreads, 0, 1, stream, args) ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
