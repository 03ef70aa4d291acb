// Pairs sorted by expert (a stable counting sort), rows copied into that
// order, and rows summed back with their weights.
//
// The sort counts and places 32 pairs at a time per warp, each warp a
// contiguous range, so equal experts keep their order without a digit pass:
// 1843200 pairs of 16 experts take 23 us in three launches, bound by the
// latency of each range's chain.  The row calls read and write every row once
// and are bound by memory: dispatch of 921600 x 64 float32 to two experts
// 111 us (6.3 TB/s), the combine's backward of 131072 x 512 bfloat16 98 us
// (6.9 TB/s, part of its writes still in the L2).
#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "gs_device.cuh"
#include "gs_head_internal.h"
#include "gs_types.cuh"

namespace gs {

namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxUnits = 152 * 32;
constexpr int kScanThreads = 256;
// Most pairs of the one-block sort: 8192 of 16 experts take it 7.8 us and three
// launches 8.6; 16384 take it 13.0.
constexpr int kSmallSort = 8192;
constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kAhead = 8;  // groups of 32 ids a warp has in flight

// Range of pairs of one unit (a warp): whole groups of 32.
__device__ __forceinline__ void unit_range(int64_t n, int units, int unit, int64_t* i0,
                                           int64_t* i1) {
    const int64_t groups = (n + 31) / 32;
    const int64_t per = (groups + units - 1) / units;
    *i0 = min(n, unit * per * 32);
    *i1 = min(n, (unit + 1) * per * 32);
}

// Calls f(i, e) for the unit's pairs, 32 at a time in order; e = -1 for a
// dropped pair and beyond the range.
template <typename F>
__device__ __forceinline__ void walk_pairs(const int32_t* __restrict__ ids, int64_t i0,
                                           int64_t i1, int experts, F&& f) {
    const int lane = threadIdx.x & 31;
    for (int64_t g = i0; g < i1; g += 32 * kAhead) {
        int e[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int64_t i = g + q * 32 + lane;
            e[q] = i < i1 ? ids[i] : -1;
            if (e[q] >= experts) e[q] = -1;
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (g + q * 32 < i1) f(g + q * 32 + lane, e[q] < 0 ? -1 : e[q]);
    }
}

// own[e] = the unit's pairs of expert e.
__device__ __forceinline__ void count_unit(const int32_t* __restrict__ ids, int64_t i0,
                                           int64_t i1, int experts, int32_t* own) {
    for (int e = threadIdx.x & 31; e < experts; e += 32) own[e] = 0;
    __syncwarp();
    walk_pairs(ids, i0, i1, experts, [&](int64_t, int e) {
        if (e >= 0) atomicAdd(&own[e], 1);
    });
    __syncwarp();
}

// Places the unit's pairs; own[e]: the row of its first pair of expert e.  A
// pair's row is that plus the pairs of its expert before it in the unit.
__device__ __forceinline__ void place_unit(const int32_t* __restrict__ ids, int64_t i0,
                                           int64_t i1, int experts, int32_t* own,
                                           int32_t* __restrict__ order,
                                           int32_t* __restrict__ slots) {
    __syncwarp();
    walk_pairs(ids, i0, i1, experts, [&](int64_t i, int e) {
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int before = __popc(same & lanemask_lt());
        const int32_t at = e >= 0 ? own[e] + before : -1;
        __syncwarp();
        if (e >= 0 && before == 0) own[e] += __popc(same);
        __syncwarp();
        if (i < i1) {
            slots[i] = at;
            if (at >= 0) order[at] = (int32_t)i;
        }
    });
}

// Exclusive prefix of v[0 .. experts) into out[0 .. experts], by one warp.
__device__ __forceinline__ void warp_prefix(const int32_t* v, int experts, int32_t* out) {
    const int lane = threadIdx.x & 31;
    int run = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
        const int n = e0 + lane < experts ? v[e0 + lane] : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        if (e0 + lane < experts) out[e0 + lane] = run + sum - n;
        run += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) out[experts] = run;
}

// The whole sort in one block, for few pairs: one launch in place of three.
__global__ void __launch_bounds__(kSmallThreads)
    k_expert_sort_small(const int32_t* __restrict__ ids, int64_t n, int experts,
                        int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                        int32_t* __restrict__ slots) {
    extern __shared__ int32_t sm[];  // counts [warps][experts], totals, first [experts + 1]
    int32_t* totals = sm + kSmallWarps * experts;
    int32_t* first = totals + experts;
    const int warp = threadIdx.x / 32;
    int32_t* own = sm + warp * experts;
    int64_t i0, i1;
    unit_range(n, kSmallWarps, warp, &i0, &i1);
    count_unit(ids, i0, i1, experts, own);
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kSmallThreads) {
        int32_t run = 0;
#pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) {
            const int32_t c = sm[w * experts + e];
            sm[w * experts + e] = run;
            run += c;
        }
        totals[e] = run;
    }
    __syncthreads();
    if (warp == 0) warp_prefix(totals, experts, first);
    __syncthreads();
    for (int e = threadIdx.x; e <= experts; e += kSmallThreads) offsets[e] = first[e];
    for (int64_t i = first[experts] + threadIdx.x; i < n; i += kSmallThreads) order[i] = -1;
    for (int e = threadIdx.x & 31; e < experts; e += 32) own[e] += first[e];
    place_unit(ids, i0, i1, experts, own, order, slots);
}

// counts[e][unit] = pairs of expert e in the unit's range.
__global__ void __launch_bounds__(kSortThreads)
    k_expert_count(const int32_t* __restrict__ ids, int64_t n, int experts, int units,
                   int32_t* __restrict__ counts) {
    extern __shared__ int32_t sm[];
    const int unit = blockIdx.x * kSortWarps + threadIdx.x / 32;
    int32_t* own = sm + threadIdx.x / 32 * experts;
    if (unit >= units) return;
    int64_t i0, i1;
    unit_range(n, units, unit, &i0, &i1);
    count_unit(ids, i0, i1, experts, own);
    for (int e = threadIdx.x & 31; e < experts; e += 32)
        counts[(int64_t)e * units + unit] = own[e];
}

// Exclusive prefix over the units of one expert's counts (block e), in place,
// and its total.
__global__ void __launch_bounds__(kScanThreads)
    k_expert_scan(int32_t* __restrict__ counts, int units, int experts,
                  int32_t* __restrict__ totals) {
    __shared__ int64_t scratch[32];
    constexpr int kEach = (kMaxUnits + kScanThreads - 1) / kScanThreads;
    const int e = blockIdx.x, t = threadIdx.x;
    int32_t c[kEach];
    int64_t sum = 0, total;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int u = t * kEach + i;
        c[i] = u < units ? counts[(int64_t)e * units + u] : 0;
        sum += c[i];
    }
    int32_t run = (int32_t)block_exclusive_scan<kScanThreads>(sum, scratch, &total);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int u = t * kEach + i;
        if (u < units) counts[(int64_t)e * units + u] = run;
        run += c[i];
    }
    if (t == 0) totals[e] = (int32_t)total;
}

__global__ void __launch_bounds__(kSortThreads)
    k_expert_place(const int32_t* __restrict__ ids, int64_t n, int experts, int units,
                   const int32_t* __restrict__ counts, const int32_t* __restrict__ totals,
                   int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                   int32_t* __restrict__ slots) {
    extern __shared__ int32_t sm[];  // first row of the pairs [warps][experts], first [experts + 1]
    int32_t* first = sm + kSortWarps * experts;
    const int unit = blockIdx.x * kSortWarps + threadIdx.x / 32;
    if (threadIdx.x < 32) warp_prefix(totals, experts, first);
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= experts; e += kSortThreads) offsets[e] = first[e];
    for (int64_t i = first[experts] + (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * kSortThreads)
        order[i] = -1;
    if (unit >= units) return;
    int32_t* own = sm + threadIdx.x / 32 * experts;
    for (int e = threadIdx.x & 31; e < experts; e += 32)
        own[e] = first[e] + counts[(int64_t)e * units + unit];
    int64_t i0, i1;
    unit_range(n, units, unit, &i0, &i1);
    place_unit(ids, i0, i1, experts, own, order, slots);
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

// Rows [kept, n) of out are 0, shared among all the grid's row groups.
template <typename Word, int kLanes>
__device__ __forceinline__ void zero_rows(Word* out, int words, int64_t kept, int64_t n) {
    constexpr int kGroups = kRowThreads / kLanes;
    for (int64_t r = kept + (int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes; r < n;
         r += (int64_t)gridDim.x * kGroups)
        for (int c = threadIdx.x % kLanes; c < words; c += kLanes) out[r * words + c] = Word{};
}

// A row is moved in words of 16, 8, 4 or 2 bytes, whatever its type: read once,
// written topk times.  kRows tokens of a lane in flight.
template <typename Word, int kLanes, int kItems, int kRows>
__global__ void __launch_bounds__(kRowThreads)
    k_dispatch(RowArgs a, const Word* __restrict__ x, int64_t ldx, int words,
               const int32_t* __restrict__ slots, const int32_t* __restrict__ offsets,
               Word* __restrict__ xs) {
    constexpr int kGroups = kRowThreads / kLanes;
    const int64_t n = a.tokens * a.topk, step = (int64_t)gridDim.x * kGroups;
    const int at = threadIdx.x % kLanes;
    for (int64_t t0 = (int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes; t0 < a.tokens;
         t0 += step * kRows)
        for (int c0 = at; c0 < words; c0 += kLanes * kItems) {
            Word v[kRows][kItems];
#pragma unroll
            for (int u = 0; u < kRows; ++u)
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    const int64_t t = t0 + u * step;
                    const int c = c0 + i * kLanes;
                    v[u][i] = t < a.tokens && c < words ? x[t * ldx + c] : Word{};
                }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int64_t t = t0 + u * step;
                if (t >= a.tokens) break;
                for (int j = 0; j < a.topk; ++j) {
                    const int64_t s = checked_slot(slots[t * a.topk + j], n, a.d_status);
                    if (s < 0) continue;
#pragma unroll
                    for (int i = 0; i < kItems; ++i) {
                        const int c = c0 + i * kLanes;
                        if (c < words) xs[s * words + c] = v[u][i];
                    }
                }
            }
        }
    zero_rows<Word, kLanes>(xs, words, checked_kept(offsets, a.experts, n, a.d_status), n);
}

// The slots and weights of kChoices choices of kTokens tokens, loaded one round
// ahead of the rows they name: a row's load waits for its slot's, and with
// both in one round that wait was most of the time (100003 tokens, 3 of 7
// experts, 131 float16 channels: 42 us against 15 us for the bytes).
template <int kChoices, int kTokens>
struct PairRound {
    int32_t slot[kTokens][kChoices];
    float weight[kTokens][kChoices];

    // Token t0 + u * step, choices from j0 on; -1 beyond the ends.
    __device__ __forceinline__ void load(const RowArgs& a, const int32_t* __restrict__ slots,
                                         const float* __restrict__ weights, int64_t t0,
                                         int64_t step, int j0) {
#pragma unroll
        for (int u = 0; u < kTokens; ++u)
#pragma unroll
            for (int q = 0; q < kChoices; ++q) {
                const int64_t t = t0 + u * step, p = t * a.topk + j0 + q;
                const bool is = t < a.tokens && j0 + q < a.topk;
                slot[u][q] = is ? slots[p] : -1;
                weight[u][q] = is && weights ? weights[p] : 1.f;
            }
    }
};

// y[t] = sum over j of w[t, j] * ys[slots[t, j]], j ascending.  kChoices of a
// token's rows and kTokens tokens are in flight.
template <typename T, int kVec, int kLanes, int kItems, int kChoices, int kTokens>
__global__ void __launch_bounds__(kRowThreads)
    k_combine(RowArgs a, const T* __restrict__ ys, const int32_t* __restrict__ slots,
              const float* __restrict__ weights, T* __restrict__ y, int64_t ldy) {
    constexpr int kGroups = kRowThreads / kLanes;
    const int64_t n = a.tokens * a.topk, step = (int64_t)gridDim.x * kGroups;
    const int64_t first = (int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes;
    for (int c0 = threadIdx.x % kLanes * kVec; c0 < a.channels; c0 += kLanes * kVec * kItems) {
        bool in[kItems];  // this lane's accesses
#pragma unroll
        for (int i = 0; i < kItems; ++i) in[i] = c0 + i * kLanes * kVec < a.channels;
        PairRound<kChoices, kTokens> next;
        next.load(a, slots, weights, first, step, 0);
        for (int64_t t0 = first; t0 < a.tokens; t0 += step * kTokens) {
            float sum[kTokens][kItems][kVec] = {};
            for (int j0 = 0; j0 < a.topk; j0 += kChoices) {
                const PairRound<kChoices, kTokens> now = next;
                RawVec<T, kVec> raw[kTokens][kChoices][kItems];
                int64_t s[kTokens][kChoices];
#pragma unroll
                for (int u = 0; u < kTokens; ++u)
#pragma unroll
                    for (int q = 0; q < kChoices; ++q) {
                        s[u][q] = checked_slot(now.slot[u][q], n, a.d_status);
                        if (s[u][q] < 0) continue;
                        const T* row = ys + s[u][q] * a.channels + c0;
#pragma unroll
                        for (int i = 0; i < kItems; ++i)
                            if (in[i])
                                raw[u][q][i] = load_raw<T, kVec>(row + i * kLanes * kVec);
                    }
                if (j0 + kChoices < a.topk)
                    next.load(a, slots, weights, t0, step, j0 + kChoices);
                else
                    next.load(a, slots, weights, t0 + step * kTokens, step, 0);
#pragma unroll
                for (int u = 0; u < kTokens; ++u)
#pragma unroll
                    for (int q = 0; q < kChoices; ++q) {
                        if (s[u][q] < 0) continue;
#pragma unroll
                        for (int i = 0; i < kItems; ++i) {
                            float v[kVec];
                            unpack<T, kVec>(raw[u][q][i], v);
#pragma unroll
                            for (int k = 0; k < kVec; ++k)
                                sum[u][i][k] += now.weight[u][q] * v[k];
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < kTokens; ++u) {
                const int64_t t = t0 + u * step;
                if (t >= a.tokens) continue;
                T* row = y + t * ldy + c0;
#pragma unroll
                for (int i = 0; i < kItems; ++i)
                    if (in[i]) store_vec<T, kVec>(row + i * kLanes * kVec, sum[u][i]);
            }
        }
    }
}

// Per pair: grad_ys[s] = w grad_y[t] and grad_weights = <grad_y[t], ys[s]>.
// grad_y[t] is read once for the pairs in flight.
template <typename T, int kVec, int kLanes, int kItems, int kChoices, int kTokens>
__global__ void __launch_bounds__(kRowThreads)
    k_combine_bwd(RowArgs a, const T* __restrict__ gy, int64_t ldgy, const T* __restrict__ ys,
                  const int32_t* __restrict__ slots, const float* __restrict__ weights,
                  const int32_t* __restrict__ offsets, T* __restrict__ gys,
                  float* __restrict__ gw) {
    constexpr int kGroups = kRowThreads / kLanes, kPairs = kTokens * kChoices;
    __shared__ RowScratch scratch;
    int half = 0;
    const int64_t n = a.tokens * a.topk, step = (int64_t)gridDim.x * kGroups;
    const int at = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    PairRound<kChoices, kTokens> next;
    next.load(a, slots, weights, (int64_t)blockIdx.x * kGroups + group, step, 0);
    // whole rounds: the lanes of a row stay together for its sums
    for (int64_t b0 = (int64_t)blockIdx.x * kGroups; b0 < a.tokens; b0 += step * kTokens) {
        const int64_t t0 = b0 + group;
        for (int j0 = 0; j0 < a.topk; j0 += kChoices) {
            const PairRound<kChoices, kTokens> now = next;
            int64_t s[kPairs];
            float dot[kPairs];
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                s[q] = checked_slot(now.slot[q / kChoices][q % kChoices], n, a.d_status);
                dot[q] = 0.f;
            }
            for (int c0 = at * kVec; c0 < a.channels; c0 += kLanes * kVec * kItems) {
                RawVec<T, kVec> rg[kTokens][kItems], ry[kPairs][kItems];
                bool in[kItems];
#pragma unroll
                for (int i = 0; i < kItems; ++i) in[i] = c0 + i * kLanes * kVec < a.channels;
#pragma unroll
                for (int u = 0; u < kTokens; ++u) {
                    const int64_t t = t0 + u * step;
                    const T* row = gy + t * ldgy + c0;
#pragma unroll
                    for (int i = 0; i < kItems; ++i)
                        rg[u][i] = t < a.tokens && in[i]
                                           ? load_raw<T, kVec>(row + i * kLanes * kVec)
                                           : RawVec<T, kVec>{};
                }
#pragma unroll
                for (int q = 0; q < kPairs; ++q) {
                    const T* row = ys + s[q] * a.channels + c0;
#pragma unroll
                    for (int i = 0; i < kItems; ++i)
                        ry[q][i] = gw && s[q] >= 0 && in[i]
                                           ? load_raw<T, kVec>(row + i * kLanes * kVec)
                                           : RawVec<T, kVec>{};
                }
                if (c0 == at * kVec) {
                    if (j0 + kChoices < a.topk)
                        next.load(a, slots, weights, t0, step, j0 + kChoices);
                    else
                        next.load(a, slots, weights, t0 + step * kTokens, step, 0);
                }
#pragma unroll
                for (int q = 0; q < kPairs; ++q) {
                    if (s[q] < 0) continue;
                    T* row = gys + s[q] * a.channels + c0;
#pragma unroll
                    for (int i = 0; i < kItems; ++i) {
                        float g[kVec], v[kVec], o[kVec];
                        unpack<T, kVec>(rg[q / kChoices][i], g);
                        unpack<T, kVec>(ry[q][i], v);
#pragma unroll
                        for (int k = 0; k < kVec; ++k) {
                            dot[q] += g[k] * v[k];
                            o[k] = now.weight[q / kChoices][q % kChoices] * g[k];
                        }
                        if (in[i]) store_vec<T, kVec>(row + i * kLanes * kVec, o);
                    }
                }
            }
            // lanes without a channel still need the next round
            if (at * kVec >= a.channels) {
                if (j0 + kChoices < a.topk)
                    next.load(a, slots, weights, t0, step, j0 + kChoices);
                else
                    next.load(a, slots, weights, t0 + step * kTokens, step, 0);
            }
            if (!gw) continue;
            row_sums<kLanes, kPairs>(dot, scratch, half);
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                const int64_t t = t0 + q / kChoices * step;
                const int j = j0 + q % kChoices;
                if (at == q && t < a.tokens && j < a.topk) gw[t * a.topk + j] = dot[q];
            }
        }
    }
    constexpr int kBytes = kVec * (int)sizeof(T);
    zero_rows<typename Raw<kBytes>::type, kLanes>(
        reinterpret_cast<typename Raw<kBytes>::type*>(gys), a.channels / kVec,
        checked_kept(offsets, a.experts, n, a.d_status), n);
}

// Calls f with the form for rows of n accesses of kVec elements: as few lanes
// as hold a row with two accesses each (eight of one or two elements).
template <int kVec, typename F>
void with_row_form(int n, F&& f) {
    if constexpr (kVec <= 2) {
        if (n <= 32) return f(Form<kVec, 8, 4, 2>{});
        if (n <= 64) return f(Form<kVec, 8, 8, 1>{});
        if (n <= 96) return f(Form<kVec, 32, 3, 2>{});
        if (n <= 160) return f(Form<kVec, 32, 5, 1>{});
        if (n <= 256) return f(Form<kVec, 32, 8, 1>{});
        return f(Form<kVec, 128, 4, 2>{});
    } else {
        if (n <= 8) return f(Form<kVec, 8, 1, 4>{});
        if (n <= 16) return f(Form<kVec, 8, 2, 2>{});
        if (n <= 128) return f(Form<kVec, 32, 2, 2>{});
        return f(Form<kVec, 128, 2, 2>{});
    }
}

// Blocks for `tokens` rows, `groups` a block: never more than are resident.
int row_blocks(int64_t tokens, int groups, int resident) {
    return (int)std::min<int64_t>((tokens + groups - 1) / groups, resident);
}

}  // namespace

int sort_units(int64_t n) {
    if (n <= kSmallSort) return 0;
    const int64_t u = (n + 255) / 256;
    return (int)std::min<int64_t>(u, kMaxUnits);
}

void launch_expert_sort(const int32_t* ids, int64_t n, int experts, int32_t* offsets,
                        int32_t* order, int32_t* slots, int32_t* counts, int32_t* totals,
                        cudaStream_t s) {
    const int units = sort_units(n);
    const size_t word = sizeof(int32_t), own = (size_t)kSortWarps * experts * word;
    if (units == 0) {
        const auto bytes = [&](int e) { return ((size_t)(kSmallWarps + 2) * e + 1) * word; };
        static PerDevice raised;
        raised.get(0, [&] {  // a launch that needs it fails without
            return cudaFuncSetAttribute(k_expert_sort_small,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)bytes(GS_MAX_EXPERTS)) == cudaSuccess;
        });
        k_expert_sort_small<<<1, kSmallThreads, bytes(experts), s>>>(ids, n, experts, offsets,
                                                                     order, slots);
        return;
    }
    const int blocks = (units + kSortWarps - 1) / kSortWarps;
    k_expert_count<<<blocks, kSortThreads, own, s>>>(ids, n, experts, units, counts);
    k_expert_scan<<<experts, kScanThreads, 0, s>>>(counts, units, experts, totals);
    k_expert_place<<<blocks, kSortThreads, own + (experts + 1) * word, s>>>(
        ids, n, experts, units, counts, totals, offsets, order, slots);
}

void launch_dispatch(const RowArgs& a, const void* x, int64_t ldx, const int32_t* slots,
                     const int32_t* offsets, void* xs, cudaStream_t s) {
    const int size = (int)dtype_size(a.dtype);
    const auto run = [&](auto word) {
        using Word = decltype(word);
        const int per = (int)sizeof(Word) / size;
        const int words = a.channels / per;
        with_row_form<sizeof(Word) >= 8 ? 8 : 1>(words, [&](auto form) {
            using F = decltype(form);
            const auto kernel = k_dispatch<Word, F::kLanes, F::kItems, F::kRows>;
            static PerDevice resident;
            const int blocks = row_blocks(a.tokens, kRowThreads / F::kLanes,
                                          resident_blocks(resident, kernel, 0));
            kernel<<<blocks, kRowThreads, 0, s>>>(a, static_cast<const Word*>(x), ldx / per,
                                                  words, slots, offsets,
                                                  static_cast<Word*>(xs));
        });
    };
    const auto whole = [&](int bytes) {
        return ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(xs)) & (bytes - 1)) ==
                   0 &&
               ldx * size % bytes == 0 && a.channels * size % bytes == 0;
    };
    if (whole(16))
        run(uint4{});
    else if (whole(8))
        run(uint2{});
    else if (whole(4))
        run(uint32_t{});
    else
        run(uint16_t{});
}

namespace {

// Four pairs in flight: kChoices of a token's and kTokens tokens.
template <int kChoices_>
struct Flight {
    static constexpr int kChoices = kChoices_, kTokens = 4 / kChoices_;
};

// f(element, form, flight) for the widest accesses (16, 8 or 4 bytes, or one
// element) at which every row of the arrays begins and ends.
template <typename F>
void with_rows(const RowArgs& a, std::initializer_list<const void*> arrays, int64_t ld, F&& f) {
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        const auto go = [&](auto form) {
            if (a.topk == 1)
                f(t, form, Flight<1>{});
            else if (a.topk == 2)
                f(t, form, Flight<2>{});
            else
                f(t, form, Flight<4>{});
        };
        uintptr_t all = (uintptr_t)(ld * sizeof(T)) | (uintptr_t)(a.channels * sizeof(T));
        for (const void* p : arrays) all |= reinterpret_cast<uintptr_t>(p);
        with_width<T>(all, [&](auto width) {
            constexpr int kVec = decltype(width)::value;
            with_row_form<kVec>(a.channels / kVec, go);
        });
    });
}

}  // namespace

void launch_combine(const RowArgs& a, const void* ys, const int32_t* slots, const float* weights,
                    void* y, int64_t ldy, cudaStream_t s) {
    with_rows(a, {ys, y}, ldy, [&](auto t, auto form, auto flight) {
        using T = decltype(t);
        using F = decltype(form);
        using P = decltype(flight);
        const auto kernel = k_combine<T, F::kVec, F::kLanes, F::kItems, P::kChoices, P::kTokens>;
        static PerDevice resident;
        const int blocks = row_blocks(a.tokens, kRowThreads / F::kLanes,
                                      resident_blocks(resident, kernel, 0));
        kernel<<<blocks, kRowThreads, 0, s>>>(
            a, static_cast<const T*>(ys), slots, weights, static_cast<T*>(y), ldy);
    });
}

void launch_combine_bwd(const RowArgs& a, const void* grad_y, int64_t ldgy, const void* ys,
                        const int32_t* slots, const float* weights, const int32_t* offsets,
                        void* grad_ys, float* grad_weights, cudaStream_t s) {
    with_rows(a, {grad_y, ys, grad_ys}, ldgy, [&](auto t, auto form, auto flight) {
        using T = decltype(t);
        using F = decltype(form);
        using P = decltype(flight);
        const auto kernel = k_combine_bwd<T, F::kVec, F::kLanes, F::kItems, P::kChoices,
                                          P::kTokens>;
        static PerDevice resident;
        const int blocks = row_blocks(a.tokens, kRowThreads / F::kLanes,
                                      resident_blocks(resident, kernel, 0));
        kernel<<<blocks, kRowThreads, 0, s>>>(
            a, static_cast<const T*>(grad_y), ldgy, static_cast<const T*>(ys), slots, weights,
            offsets, static_cast<T*>(grad_ys), grad_weights);
    });
}

}  // namespace gs
