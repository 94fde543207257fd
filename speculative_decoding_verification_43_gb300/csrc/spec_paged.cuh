// What the kernels over ragged rows and the paged cache share: which rows a request holds, and finding a row's
// request.
#pragma once

#include <climits>
#include <cstdint>

#include "spec_device.cuh"

namespace spec {

// Division of 0 <= n < 2^31 by a divisor known on the host: with 2^k >= d, m = floor(2^(31+k) / d) + 1
// exceeds 2^(31+k) / d by at most 1 = d / d <= 2^k / d, so n m / 2^(31+k) is off by less than 1 / d and its
// floor is right.
struct FastDiv {
    uint32_t mul = 0, shift = 0;
    FastDiv() = default;
    explicit FastDiv(int32_t d) {
        uint32_t k = 0;
        while ((1ull << k) < static_cast<uint64_t>(d)) ++k;
        shift = 31 + k;
        mul = static_cast<uint32_t>((1ull << shift) / static_cast<uint64_t>(d) + 1);
    }
    __device__ __forceinline__ int operator()(int n) const {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
    }
};

// Elements from a cache's first one to its last (for the debug build's checks).
template <typename Params>
__device__ __forceinline__ int64_t cache_extent(const Params &P) {
    return (P.n_pages - 1) * P.page_stride + (P.page_size - 1) * P.slot_stride + (P.Hkv - 1) * P.head_stride + P.D;
}

// Which rows are a request's. Request i holds rows row_off[i] .. row_off[i+1]-1 when 0 <= row_off[i] <=
// row_off[i+1] <= T and none of the offsets within [0, T] contradicts it: no earlier one is above row_off[i],
// no later one below row_off[i+1]. So no row is held twice, the rows held are T at most, and of every row that
// is held the search below finds the holder. An offset outside [0, T] costs the two requests beside it; offsets
// out of order cost those whose rows they leave in doubt.

// A request's own two offsets; where all requests' are right, all offsets are in order.
__device__ __forceinline__ bool offsets_right(int r0, int r1, int T) { return r0 >= 0 && r1 >= r0 && r1 <= T; }

// True when one of the offsets `first`, first + step, .. contradicts that request i has rows [r0, r1). Needed
// only where some request's own offsets are wrong, and read only then.
static __device__ __noinline__ bool offsets_contradict(const int32_t *row_off, int B, int T, int i, int r0, int r1,
                                                       int first, int step) {
    bool bad = false;
#pragma unroll 4
    for (int j = first; j <= B; j += step) {
        const int v = row_off[j];
        if (v >= 0 && v <= T) bad |= j <= i ? v > r0 : v < r1;
    }
    return bad;
}

// The first of the offsets from row_off[j] on that lies in [0, T]; above every row when there is none.
__device__ __forceinline__ int offset_from(const int32_t *row_off, int B, int T, int j) {
    int v = row_off[j];
#pragma unroll 1
    while (v < 0 || v > T) {
        if (++j > B) return INT_MAX;
        v = row_off[j];
    }
    return v;
}

// The request holding row r: the largest i < B with row_off[i] <= r. Called by a whole warp with the
// same r; every step of the search narrows the range 32-fold (two dependent loads up to 1024
// requests). For a row that nobody holds the result is still in [0, B).
__device__ __forceinline__ int find_request(const int32_t *row_off, int B, int T, int r, int lane) {
    int lo = 0, n = B;
#pragma unroll 1
    while (n > 1) {
        const int step = (n + kWarp - 1) / kWarp;
        const int x = lane * step;
        const bool le = x < n && offset_from(row_off, B, T, lo + x) <= r;
        const int k = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}
// The same by one thread.
__device__ __forceinline__ int find_request(const int32_t *row_off, int B, int T, int r) {
    int lo = 0, n = B;
#pragma unroll 1
    while (n > 1) {
        const int half = n / 2;
        if (offset_from(row_off, B, T, lo + half) <= r) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

}  // namespace spec
