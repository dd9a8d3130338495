// rotary.cuh - rotary positions: the first 2 h channels of a head turned in h pairs,
//   (a, b) -> (a cos - b sin, b cos + a sin),
// pairs (i, i + h), or (2 i, 2 i + 1) interleaved, with the token's row of a table of
// cosines and sines.  Products and sums are rounded to fp32 one by one, then the result
// once to 16 bits: the same bits wherever a value is turned (alone, or on its way into a cache).
//
// What bounds it: HBM (4 bytes per channel, a table row of 8 h bytes per token).  An item is 8 pairs of
// one or two heads of one token: two 16-byte reads and writes per head, 64 bytes of table that
// stay in registers over the heads.  16000 tokens of 40 heads, d 128: 50.5 us, 6.6 TB/s, 99% of what a copy reaches; a decode
// step of 8 tokens 1.9 us in a graph, a launch and two dependent reads.
#pragma once

#include "paged_common.cuh"

namespace fa {
namespace paged {

struct RotaryTable {
    const float* rows;       // [num_positions][2 h]: cosines, then sines
    const int* positions;    // per token; negative: not turned
    int num_positions, half; // half = h, a multiple of 8
    int interleaved, inverse;
};
// The table's row for a position (-1: not turned), a token's row.
__device__ __forceinline__ int rotary_row(const RotaryTable& r, int position) {
    if (position >= r.num_positions) report(kBadData);
    return position < r.num_positions ? max(position, -1) : -1;
}
__device__ __forceinline__ int rotary_position(const RotaryTable& r, int token) { return rotary_row(r, ld_meta(r.positions + token)); }
// Some heads of every token; y may be x.
struct RotaryPart {
    const uint16_t* x;
    uint16_t* y;
    long long xt, xh, yt, yh;  // token and head strides, elements
    int heads;
};
struct RotaryWork {
    RotaryTable r;
    RotaryPart part[2];
    int T;
    int cols, tail;  // items of 8 pairs per head; of 16 channels behind them that are copied (0 in place)
    int d;
    int groups;      // of heads
};

__device__ __forceinline__ float turn_first(float a, float b, float c, float s) { return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)); }
__device__ __forceinline__ float turn_second(float a, float b, float c, float s) { return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)); }

__device__ __forceinline__ void load_floats8(const float* p, float (&f)[8]) {
    const float4 u = ld(reinterpret_cast<const float4*>(p)), v = ld(reinterpret_cast<const float4*>(p) + 1);
    f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
}

// Two pieces of 8 channels turned: pairs (u[i], v[i]), or neighbours within u, then within v.
__device__ __forceinline__ void turn16(uint4& u, uint4& v, const float (&c)[8], const float (&s)[8], bool interleaved, bool bf16) {
    uint32_t* a = reinterpret_cast<uint32_t*>(&u);
    uint32_t* b = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = unpack16(a[i], bf16), y = unpack16(b[i], bf16);
        if (interleaved) {
            a[i] = pack16(turn_first(x.x, x.y, c[i], s[i]), turn_second(x.x, x.y, c[i], s[i]), bf16);
            b[i] = pack16(turn_first(y.x, y.y, c[4 + i], s[4 + i]), turn_second(y.x, y.y, c[4 + i], s[4 + i]), bf16);
        } else {
            a[i] = pack16(turn_first(x.x, y.x, c[2 * i], s[2 * i]), turn_first(x.y, y.y, c[2 * i + 1], s[2 * i + 1]), bf16);
            b[i] = pack16(turn_second(x.x, y.x, c[2 * i], s[2 * i]), turn_second(x.y, y.y, c[2 * i + 1], s[2 * i + 1]), bf16);
        }
    }
}

// Item `item` of T x groups x (cols + tail): U heads of one token, `groups` apart, so that a warp reads neighbouring heads at a time.
template <int U, bool BF16>
__device__ __forceinline__ void rotary_item(const RotaryWork& w, unsigned item) {
    const unsigned width = w.cols + w.tail;
    const unsigned rest = item / width, token = rest / w.groups;
    const int col = item - rest * width, h0 = static_cast<int>(rest - token * w.groups);
    const int all = w.part[0].heads + w.part[1].heads;
    const bool turned = col < w.cols;
    // channels of the item's first and second piece
    const int c0 = !turned ? 2 * w.r.half + (col - w.cols) * 16 : w.r.interleaved ? col * 16 : col * 8;
    const int c1 = !turned || w.r.interleaved ? c0 + 8 : c0 + w.r.half;
    const bool second_piece = turned || c1 < w.d;
    uint4 u[U], v[U];
    uint16_t* dst[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int head = h0 + i * w.groups;
        dst[i] = nullptr;
        if (head < all) {
            const bool second = head >= w.part[0].heads;
            const int h = second ? head - w.part[0].heads : head;
            // (selected, not indexed: the parameters stay in constant memory)
            const uint16_t* src = (second ? w.part[1].x : w.part[0].x) + token * (second ? w.part[1].xt : w.part[0].xt) +
                                  h * (second ? w.part[1].xh : w.part[0].xh);
            dst[i] = (second ? w.part[1].y : w.part[0].y) + token * (second ? w.part[1].yt : w.part[0].yt) +
                     h * (second ? w.part[1].yh : w.part[0].yh);
            u[i] = ld(reinterpret_cast<const uint4*>(src + c0));
            if (second_piece) v[i] = ld(reinterpret_cast<const uint4*>(src + c1));
        }
    }
    const int at = turned ? rotary_position(w.r, token) : -1;
    float c[8], s[8];
    if (at >= 0) {
        const float* row = w.r.rows + static_cast<long long>(at) * (2 * w.r.half);
        load_floats8(row + col * 8, c);
        load_floats8(row + w.r.half + col * 8, s);
        if (w.r.inverse) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = -s[i];
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (!dst[i]) continue;
        if (at >= 0) turn16(u[i], v[i], c, s, w.r.interleaved != 0, BF16);
        *reinterpret_cast<uint4*>(dst[i] + c0) = u[i];
        if (second_piece) *reinterpret_cast<uint4*>(dst[i] + c1) = v[i];
    }
}

constexpr int kRotaryThreads = 256;
constexpr int kRotaryHeads = 2;  // heads of an item where there are items enough

template <int U, bool BF16>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryWork w) {
    dependents_may_start();
    wait_for_previous();
    const unsigned item = blockIdx.x * static_cast<unsigned>(kRotaryThreads) + threadIdx.x;
    if (item < static_cast<unsigned>(w.T) * static_cast<unsigned>(w.groups * (w.cols + w.tail))) rotary_item<U, BF16>(w, item);
}

}  // namespace paged
}  // namespace fa
