// What the kernels over ragged rows and the paged cache share: finding a row's request.
#pragma once

#include <cstdint>

#include "spec_device.cuh"

namespace spec {

// The request owning row r: the largest i < B with row_off[i] <= r. Called by a whole warp with the
// same r; every step of the search narrows the range 32-fold (two dependent loads up to 1024
// requests). With inconsistent offsets the result is still in [0, B).
__device__ __forceinline__ int find_request(const int32_t *row_off, int B, int r, int lane) {
    int lo = 0, n = B;
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
