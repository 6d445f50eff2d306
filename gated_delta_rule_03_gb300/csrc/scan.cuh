// scan.cuh -- sums along a warp.
#pragma once

#include <stdint.h>

namespace gdr {

// Inclusive sum over the lanes of a warp.
__device__ __forceinline__ int64_t warp_scan(int64_t x) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t y = __shfl_up_sync(~0u, x, d);
        if ((int)(threadIdx.x & 31) >= d) x += y;
    }
    return x;
}

}  // namespace gdr
