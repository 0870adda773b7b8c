// What the decode kernels and the differential prompts share.
//
// Even split of ragged sequences over the warps of a grid.  A stream is one (sequence, KV head, group of query rows); its work
// is the sequence's 16-token tiles.  The streams' tiles are laid end to end
// (prefix[b] = tiles of all streams of the sequences before b) and warp w of W
// takes the w-th of W equal contiguous ranges of them.
#pragma once

#include <cstdint>

namespace gbattn {

// Where exponentials are rounded to FP16 they are p = 2^(x - m) with the reference m kShift below a
// maximum of the row: the largest lie at 2^kShift, and m moves when a score passes it by kTop, so
// that none exceeds 2^15 (FP16 ends at 65504).  FP16's last step is 2^-24 whatever the value: a token
// whose p is rounded to hi + lo is off by 2^-22 of p or by 2^-25, that is 2^-(25 + kShift) of the
// row's largest, whichever is more.  With m at the maximum itself everything below 2^-25 of an
// attention sink was lost, and 2^-14 kept ten bits.  O, the sum and their records are all relative to m.
constexpr float kShift = 11.0f, kTop = 15.0f;

// First tile of warp w when W warps share U tiles.
__device__ __forceinline__ uint32_t warp_start(uint32_t w, uint32_t W, uint32_t U) {
    return static_cast<uint32_t>(static_cast<unsigned long long>(w) * U / W);
}

// The warp whose range holds tile u (the last w with warp_start(w) <= u).
__device__ __forceinline__ uint32_t warp_of(uint32_t u, uint32_t W, uint32_t U) {
    return static_cast<uint32_t>(((static_cast<unsigned long long>(u) + 1) * W - 1) / U);
}

// Where tile u lives: sequence b, stream within the sequence (hk * row_groups +
// rg), tile t within the stream, and the stream's tile range.
struct TileLoc {
    int b, sis, t;
    uint32_t s_end;
};

__device__ __forceinline__ TileLoc locate(uint32_t u, const uint32_t* prefix, int B, int per_seq) {
    int lo = 0, hi = B - 1;   // largest b with prefix[b] <= u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= u) lo = mid; else hi = mid - 1;
    }
    TileLoc L;
    L.b = lo;
    const uint32_t T = (prefix[lo + 1] - prefix[lo]) / per_seq;
    const uint32_t off = u - prefix[lo];
    L.sis = static_cast<int>(off / T);
    L.t = static_cast<int>(off - L.sis * T);
    L.s_end = prefix[lo] + (L.sis + 1) * T;
    return L;
}

}  // namespace gbattn
