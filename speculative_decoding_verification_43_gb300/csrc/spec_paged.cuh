// What the kernels over ragged rows and the paged cache share: finding a row's request.
#pragma once

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

// The request owning row r: the largest i < B with row_off[i] <= r. Called by a whole warp with the
// same r; every step of the search narrows the range 32-fold (two dependent loads up to 1024
// requests). With inconsistent offsets the result is still in [0, B).
__device__ __forceinline__ int find_request(const int32_t *row_off, int B, int r, int lane) {
    int lo = 0, n = B;
#pragma unroll 1
    while (n > 1) {
        const int step = (n + kWarp - 1) / kWarp;
        const int x = lane * step;
        const bool le = x < n && row_off[lo + x] <= r;
        const int k = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

}  // namespace spec
