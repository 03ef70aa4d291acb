// The experts' row ranges, read from the caller's offsets.
#pragma once

#include <cstdint>

#include "gs_device.cuh"

namespace gs {

// By one whole warp: begin[e] (e <= experts) = the first row of expert e,
// begin[experts] = the first row of no expert, all within [0, rows] and never
// falling whatever the offsets hold; prefix[e] = pieces of `height` rows of
// the experts before e, prefix[experts] = all of them.  height 0: every
// expert is one piece, with rows or without.  Returns prefix[experts].
// rows + height stays below 2^31 (GS_MAX_EXPERT_ROWS).
__device__ __forceinline__ int expert_pieces(const int32_t* offsets, int experts, int64_t rows,
                                             int height, int32_t* begin, int32_t* prefix,
                                             int32_t* d_status) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int e0 = 0; e0 <= experts; e0 += 32) {
        const int e = e0 + lane;
        int v = 0;
        if (e <= experts) {
            v = offsets[e];
            if (v < 0 || v > rows) GS_BOUNDS_REPORT(d_status);
            v = (int)min(max((int64_t)v, (int64_t)0), rows);
        }
        int top = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, top, o);
            if (lane >= o) top = max(top, u);
        }
        top = max(top, carry);
        if (e <= experts) {
            if (top != v) GS_BOUNDS_REPORT(d_status);
            begin[e] = top;
        }
        carry = __shfl_sync(0xffffffffu, top, 31);
    }
    __syncwarp();
    int run = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
        const int e = e0 + lane;
        int n = 0;
        if (e < experts) n = height ? (begin[e + 1] - begin[e] + height - 1) / height : 1;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        if (e < experts) prefix[e] = run + sum - n;
        run += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) prefix[experts] = run;
    __syncwarp();
    return run;
}

// The expert that piece `piece` (below prefix[experts]) belongs to.
__device__ __forceinline__ int expert_of(const int32_t* prefix, int experts, int piece) {
    int lo = 0, hi = experts;  // prefix[lo] <= piece < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (prefix[mid] <= piece)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

}  // namespace gs
