// What the kernels of the 4-bit cache share: the row's layout and the search for a token's sequence.
#pragma once

#include "kda_device.cuh"
#include "kda_ops.h"

namespace kda {

constexpr int QC_ROW = KDA_QCACHE_ROW, QC_NUMBERS = 128;   // codes of k, codes of v, scales and zeros

// The whole warp: the last n in [0, nseq) with cu[n] <= t (0 if there is none), 32 candidates at a time.
__device__ __forceinline__ int sequence_of(const int64_t* cu, int nseq, int64_t t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, width = nseq;
    while (width > 1) {
        const int step = (width + 31) / 32, c = lo + lane * step;
        const uint32_t at = __ballot_sync(0xffffffffu, c < lo + width && cu[c] <= t);
        const int b = at ? 31 - __clz(at) : 0;
        width = min(step, width - b * step);
        lo += b * step;
    }
    return lo;
}

}  // namespace kda
