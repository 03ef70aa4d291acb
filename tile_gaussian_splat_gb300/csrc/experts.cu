// Pairs sorted by expert (a stable counting sort), rows copied into that
// order, and rows summed back with their weights.
#include <cstdint>

#include "gs_device.cuh"
#include "gs_head_internal.h"
#include "gs_types.cuh"

namespace gs {

namespace {

constexpr int kSortUnitThreads = 128;
constexpr int kSortUnitWarps = kSortUnitThreads / 32;
constexpr int kMaxUnits = 152 * 16;
constexpr int kScanThreads = 256;
constexpr int kRowThreads = 128;
constexpr int kRowWarps = kRowThreads / 32;

// Range of pairs of one unit (a warp): whole groups of 32.
__device__ __forceinline__ void unit_range(int64_t n, int units, int unit, int64_t* i0,
                                           int64_t* i1) {
    const int64_t groups = (n + 31) / 32;
    const int64_t per = (groups + units - 1) / units;
    *i0 = min(n, unit * per * 32);
    *i1 = min(n, (unit + 1) * per * 32);
}

// counts[unit][e] = pairs of expert e in the unit's range.
__global__ void __launch_bounds__(kSortUnitThreads)
    k_expert_count(const int32_t* __restrict__ ids, int64_t n, int experts, int units,
                   int32_t* __restrict__ counts) {
    extern __shared__ int32_t sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int unit = blockIdx.x * kSortUnitWarps + warp;
    int32_t* own = sm + warp * experts;
    for (int e = lane; e < experts; e += 32) own[e] = 0;
    __syncwarp();
    if (unit >= units) return;
    int64_t i0, i1;
    unit_range(n, units, unit, &i0, &i1);
    for (int64_t i = i0 + lane; i < i1; i += 32) {
        const int e = ids[i];
        if (e >= 0 && e < experts) atomicAdd(&own[e], 1);
    }
    __syncwarp();
    for (int e = lane; e < experts; e += 32) counts[(int64_t)unit * experts + e] = own[e];
}

// Exclusive prefix over the units of one expert's counts (block e), in place,
// and its total.
__global__ void __launch_bounds__(kScanThreads)
    k_expert_scan(int32_t* __restrict__ counts, int units, int experts,
                  int32_t* __restrict__ totals) {
    __shared__ int32_t part[kScanThreads];
    const int e = blockIdx.x, t = threadIdx.x;
    const int per = (units + kScanThreads - 1) / kScanThreads;
    const int u0 = min(units, t * per), u1 = min(units, u0 + per);
    int32_t sum = 0;
    for (int u = u0; u < u1; ++u) sum += counts[(int64_t)u * experts + e];
    part[t] = sum;
    __syncthreads();
    for (int o = 1; o < kScanThreads; o <<= 1) {
        const int32_t v = t >= o ? part[t - o] : 0;
        __syncthreads();
        part[t] += v;
        __syncthreads();
    }
    int32_t run = part[t] - sum;
    for (int u = u0; u < u1; ++u) {
        const int32_t c = counts[(int64_t)u * experts + e];
        counts[(int64_t)u * experts + e] = run;
        run += c;
    }
    if (t == kScanThreads - 1) totals[e] = part[t];
}

// offsets from the totals.
__global__ void k_expert_offsets(const int32_t* __restrict__ totals, int experts,
                                 int32_t* __restrict__ offsets) {
    if (threadIdx.x == 0) {
        int32_t run = 0;
        for (int e = 0; e < experts; ++e) {
            offsets[e] = run;
            run += totals[e];
        }
        offsets[experts] = run;
    }
}

// Each unit walks its range in order, 32 pairs at a time; a pair's row is its
// expert's start plus the pairs of that expert before it.
__global__ void __launch_bounds__(kSortUnitThreads)
    k_expert_place(const int32_t* __restrict__ ids, int64_t n, int experts, int units,
                   const int32_t* __restrict__ counts, const int32_t* __restrict__ offsets,
                   int32_t* __restrict__ order, int32_t* __restrict__ slots) {
    extern __shared__ int32_t sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int unit = blockIdx.x * kSortUnitWarps + warp;
    const int64_t kept = offsets[experts];
    for (int64_t i = kept + (int64_t)blockIdx.x * kSortUnitThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * kSortUnitThreads)
        order[i] = -1;
    if (unit >= units) return;
    int32_t* own = sm + warp * experts;
    for (int e = lane; e < experts; e += 32)
        own[e] = offsets[e] + counts[(int64_t)unit * experts + e];
    __syncwarp();
    int64_t i0, i1;
    unit_range(n, units, unit, &i0, &i1);
    for (int64_t g = i0; g < i1; g += 32) {
        const int64_t i = g + lane;
        int e = i < i1 ? ids[i] : -1;
        if (e < 0 || e >= experts) e = -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int before = __popc(same & ((1u << lane) - 1u));
        int32_t at = -1;
        if (e >= 0) at = own[e] + before;
        __syncwarp();
        if (e >= 0 && before == 0) own[e] += __popc(same);
        __syncwarp();
        if (i < i1) {
            slots[i] = at;
            if (at >= 0) order[at] = (int32_t)i;
        }
    }
}

// A slot read from the caller's array: -1 unless it names one of n rows.
__device__ __forceinline__ int64_t checked_slot(int32_t slot, int64_t n, int32_t* d_status) {
    if (slot >= n) GS_BOUNDS_REPORT(d_status);
    return slot >= 0 && slot < n ? slot : -1;
}

__device__ __forceinline__ int64_t checked_kept(const int32_t* offsets, int experts, int64_t n,
                                                int32_t* d_status) {
    const int64_t k = offsets[experts];
    if (k < 0 || k > n) GS_BOUNDS_REPORT(d_status);
    return min(max(k, (int64_t)0), n);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    k_dispatch(RowArgs a, const T* __restrict__ x, int64_t ldx, const int32_t* __restrict__ slots,
               const int32_t* __restrict__ offsets, T* __restrict__ xs) {
    const int lane = threadIdx.x & 31;
    const int64_t first = blockIdx.x * (int64_t)kRowWarps + threadIdx.x / 32;
    const int64_t step = (int64_t)gridDim.x * kRowWarps;
    const int64_t n = a.tokens * a.topk;
    for (int64_t t = first; t < a.tokens; t += step)
        for (int j = 0; j < a.topk; ++j) {
            const int64_t s = checked_slot(slots[t * a.topk + j], n, a.d_status);
            if (s < 0) continue;
            for (int c = lane; c < a.channels; c += 32)
                xs[s * a.channels + c] = x[t * ldx + c];
        }
    for (int64_t r = checked_kept(offsets, a.experts, n, a.d_status) + first; r < n; r += step)
        for (int c = lane; c < a.channels; c += 32) xs[r * a.channels + c] = from_f<T>(0.f);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    k_combine(RowArgs a, const T* __restrict__ ys, const int32_t* __restrict__ slots,
              const float* __restrict__ weights, T* __restrict__ y, int64_t ldy) {
    const int lane = threadIdx.x & 31;
    const int64_t n = a.tokens * a.topk;
    for (int64_t t = blockIdx.x * (int64_t)kRowWarps + threadIdx.x / 32; t < a.tokens;
         t += (int64_t)gridDim.x * kRowWarps)
        for (int c = lane; c < a.channels; c += 32) {
            float sum = 0.f;
            for (int j = 0; j < a.topk; ++j) {
                const int64_t s = checked_slot(slots[t * a.topk + j], n, a.d_status);
                if (s < 0) continue;
                const float v = to_f(ys[s * a.channels + c]);
                sum += weights ? weights[t * a.topk + j] * v : v;
            }
            y[t * ldy + c] = from_f<T>(sum);
        }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    k_combine_bwd(RowArgs a, const T* __restrict__ gy, int64_t ldgy, const T* __restrict__ ys,
                  const int32_t* __restrict__ slots, const float* __restrict__ weights,
                  const int32_t* __restrict__ offsets, T* __restrict__ gys,
                  float* __restrict__ gw) {
    const int lane = threadIdx.x & 31;
    const int64_t first = blockIdx.x * (int64_t)kRowWarps + threadIdx.x / 32;
    const int64_t step = (int64_t)gridDim.x * kRowWarps;
    const int64_t n = a.tokens * a.topk;
    for (int64_t t = first; t < a.tokens; t += step)
        for (int j = 0; j < a.topk; ++j) {
            const int64_t p = t * a.topk + j;
            const int64_t s = checked_slot(slots[p], n, a.d_status);
            float sum = 0.f;
            if (s >= 0) {
                const float w = weights ? weights[p] : 1.0f;
                for (int c = lane; c < a.channels; c += 32) {
                    const float g = to_f(gy[t * ldgy + c]);
                    gys[s * a.channels + c] = from_f<T>(w * g);
                    if (gw) sum += g * to_f(ys[s * a.channels + c]);
                }
            }
            if (gw) {
                sum = warp_sum(sum);
                if (lane == 0) gw[p] = sum;
            }
        }
    for (int64_t r = checked_kept(offsets, a.experts, n, a.d_status) + first; r < n; r += step)
        for (int c = lane; c < a.channels; c += 32) gys[r * a.channels + c] = from_f<T>(0.f);
}

int row_blocks(int64_t rows) {
    const int64_t b = (rows + kRowWarps - 1) / kRowWarps;
    return (int)(b < 152 * 64 ? b : 152 * 64);
}

}  // namespace

int sort_units(int64_t n) {
    const int64_t u = (n + 255) / 256;
    return (int)(u < 1 ? 1 : u > kMaxUnits ? kMaxUnits : u);
}

void launch_expert_sort(const int32_t* ids, int64_t n, int experts, int32_t* offsets,
                        int32_t* order, int32_t* slots, int32_t* counts, int32_t* totals,
                        cudaStream_t s) {
    const int units = sort_units(n);
    const int blocks = (units + kSortUnitWarps - 1) / kSortUnitWarps;
    const size_t smem = (size_t)kSortUnitWarps * experts * sizeof(int32_t);
    k_expert_count<<<blocks, kSortUnitThreads, smem, s>>>(ids, n, experts, units, counts);
    k_expert_scan<<<experts, kScanThreads, 0, s>>>(counts, units, experts, totals);
    k_expert_offsets<<<1, 32, 0, s>>>(totals, experts, offsets);
    k_expert_place<<<blocks, kSortUnitThreads, smem, s>>>(ids, n, experts, units, counts, offsets,
                                                          order, slots);
}

void launch_dispatch(const RowArgs& a, const void* x, int64_t ldx, const int32_t* slots,
                     const int32_t* offsets, void* xs, cudaStream_t s) {
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        k_dispatch<T><<<row_blocks(a.tokens), kRowThreads, 0, s>>>(a, (const T*)x, ldx, slots,
                                                                   offsets, (T*)xs);
    });
}

void launch_combine(const RowArgs& a, const void* ys, const int32_t* slots, const float* weights,
                    void* y, int64_t ldy, cudaStream_t s) {
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        k_combine<T><<<row_blocks(a.tokens), kRowThreads, 0, s>>>(a, (const T*)ys, slots, weights,
                                                                  (T*)y, ldy);
    });
}

void launch_combine_bwd(const RowArgs& a, const void* grad_y, int64_t ldgy, const void* ys,
                        const int32_t* slots, const float* weights, const int32_t* offsets,
                        void* grad_ys, float* grad_weights, cudaStream_t s) {
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        k_combine_bwd<T><<<row_blocks(a.tokens), kRowThreads, 0, s>>>(
            a, (const T*)grad_y, ldgy, (const T*)ys, slots, weights, offsets, (T*)grad_ys,
            grad_weights);
    });
}

}  // namespace gs
