// The router of the expert head: every token's choice of experts from its
// logits, the choices' weights, the experts' counts and the balance loss, and
// their gradient in the logits.
//
// Both directions read each row of logits once, so memory bandwidth is their
// floor; what bounds them is the instructions a row takes, in the few warps that
// 70 to 120 registers a thread leave on an SM (forward, 16 float32: issue 65 %,
// warps 21 %, DRAM 33 %; gradient 69, 35 and 44 %).  kLanes lanes share a
// row (up to 16 experts a thread has it alone and exchanges nothing); a lane owns
// the same experts of every row it meets, so the sums of probabilities behind the
// balance loss stay in registers until the end and are then added up in a fixed
// order.  The choice is topk rounds of a maximum, then the lowest index that has
// it: each lane keeps its logits as unsigned words in the order of the values, 0
// where there is nothing to choose.
//
// 921600 rows of 16 float32, two choices: 27 us (floor 11; without the next row on
// its way 33, before that with IEEE divisions and expf 49, with four lanes a row
// 66).  Gradient, the same rows: 30 us (floor 19); 230400 of 64 bfloat16, four
// choices 24 us (floor 9.7), forward 36 (floor 5.4).
#include <algorithm>
#include <cstdint>

#include "gs_device.cuh"
#include "gs_head_internal.h"
#include "gs_types.cuh"

namespace gs {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// How many lanes share a row, accesses of kVec elements and accesses a lane; a
// lane holds up to kSlots choices (32 lanes all that there can be).
template <int kVec_, int kLanes_, int kItems_>
struct Spread {
    static constexpr int kVec = kVec_, kLanes = kLanes_, kItems = kItems_;
    static constexpr int kSlots = kLanes == 1 ? 4 : 2;
    static constexpr int kChoices = kLanes * kSlots;
};

// Logits as words in the order of the values: an addition of 0 makes both zeros
// the same and every NaN the positive one, which is above everything.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ (uint32_t)((int32_t)u >> 31 | (int32_t)0x80000000);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// exp(v) by the hardware's power of two: off by about (2 + |v|) 2^-23 of it, 0
// below 2^-126.  The small probabilities are off the most: weights of logits three
// apart by 1e-6 at most, 4e-8 of their norm, where expf and IEEE divisions for the
// choices alone leave 6e-7 and 4e-8, and take 32 us for the forward's 27 and 33 for
// the gradient's 30.
__device__ __forceinline__ float exp_approx(float v) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * 1.44269504f));
    return e;
}
constexpr uint32_t kLowest = 0x007fffffu;  // minus infinity: not chosen, nor what is below

template <int kLanes>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

template <int kLanes>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    if constexpr (kLanes == 32) return __reduce_max_sync(kAll, v);
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
template <int kLanes>
__device__ __forceinline__ int group_min(int v) {
    if constexpr (kLanes == 32) return __reduce_min_sync(kAll, v);
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) v = min(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

struct RouteFwd {
    const void* logits;
    const uint8_t* keep;
    int32_t *ids, *counts;      // counts: or null
    float *weights, *loss;      // loss: or null
    float* partial;             // (blocks, experts + 1): sums of probabilities
    int32_t* part_counts;       // (blocks, experts + 1)
    float* totals;              // experts + 1
    uint32_t* ticket;
    int64_t ld, tokens;
    int topk, experts, renormalise;
    int pairs;                  // two choices a token, to be written together
};

// loss = experts * sum over e of share_e * mean probability_e, by one warp in
// a fixed order.  volatile: other blocks' sums, from where they wrote them.
__device__ __forceinline__ float balance(const volatile float* sums,
                                         const volatile int32_t* counts, int experts) {
    const int lane = threadIdx.x & 31;
    float dot = 0.f;
    int pairs = 0;
    for (int e = lane; e < experts; e += 32) {
        const int c = counts[e];
        dot += sums[e] * (float)c;
        pairs += c;
    }
    dot = warp_sum(dot);
    pairs = __reduce_add_sync(kAll, pairs);
    const int taking = counts[experts];
    return pairs > 0 ? (float)experts * (dot / ((float)taking * (float)pairs)) : 0.f;
}

template <typename T, typename F>
__global__ void __launch_bounds__(kThreads) k_route_fwd(RouteFwd a) {
    constexpr int kVec = F::kVec, kLanes = F::kLanes, kItems = F::kItems, kSlots = F::kSlots;
    constexpr int kGroups = kThreads / kLanes;
    extern __shared__ int32_t shared[];
    int32_t* count = shared;                                          // experts + 1
    float* sums = reinterpret_cast<float*>(shared + a.experts + 1);   // kWarps x experts
    const bool tally = a.counts;
    const int at = threadIdx.x % kLanes;
    cudaTriggerProgrammaticLaunchCompletion();  // k_route_sum may come up, and wait
    if (tally) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && gridDim.x > 1) *a.ticket = 0;
        for (int e = threadIdx.x; e <= a.experts; e += kThreads) count[e] = 0;
        __syncthreads();
    }
    float sum[kItems][kVec] = {};
    int taking = 0;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    // the next row comes in while this one is worked on
    RawVec<T, kVec> ahead[kItems];
    bool keep_ahead;
    const auto load = [&](int64_t r) {
        keep_ahead = r < a.tokens && (!a.keep || a.keep[r]);
        const T* x = static_cast<const T*>(a.logits) + r * a.ld + at * kVec;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            ahead[i] = keep_ahead && (i * kLanes + at) * kVec < a.experts
                           ? load_raw<T, kVec>(x + i * kLanes * kVec)
                           : RawVec<T, kVec>{};
    };
    load((int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes);
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < a.tokens; r0 += step) {
        const int64_t r = r0 + threadIdx.x / kLanes;
        const bool keep = keep_ahead;
        RawVec<T, kVec> raw[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) raw[i] = ahead[i];
        load(r + step);
        uint32_t key[kItems][kVec];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            float v[kVec];
            unpack<T, kVec>(raw[i], v);
            const bool in = keep && (i * kLanes + at) * kVec < a.experts;
#pragma unroll
            for (int j = 0; j < kVec; ++j) key[i][j] = in ? order_key(v[j]) : 0;
        }
        int id[kSlots];
        float e[kSlots];
        float top = 0.f;
        bool any = false;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            id[s] = -1;
            e[s] = 0.f;
            for (int l = 0; l < kLanes; ++l) {
                const int round = s * kLanes + l;
                if (round >= a.topk) break;
                uint32_t best = kLowest;
#pragma unroll
                for (int i = 0; i < kItems; ++i)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) best = max(best, key[i][j]);
                best = group_max<kLanes>(best);
                int index = 0x7fffffff;  // the lowest that has it
#pragma unroll
                for (int i = kItems - 1; i >= 0; --i)
#pragma unroll
                    for (int j = kVec - 1; j >= 0; --j)
                        if (key[i][j] == best) index = (i * kLanes + at) * kVec + j;
                index = group_min<kLanes>(index);
#pragma unroll
                for (int i = 0; i < kItems; ++i)
#pragma unroll
                    for (int j = 0; j < kVec; ++j)
                        if (index == (i * kLanes + at) * kVec + j) key[i][j] = 0;
                if (round == 0) {
                    any = best > kLowest;
                    top = key_value(best);
                }
                if (at == l && best > kLowest) {
                    id[s] = index;
                    e[s] = exp_approx(key_value(best) - top);
                }
            }
        }
        float all = 0.f, chosen = 0.f;
        float p[kItems][kVec];
        if (tally || !a.renormalise) {
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                float v[kVec];
                unpack<T, kVec>(raw[i], v);
                const bool in = any && (i * kLanes + at) * kVec < a.experts;
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    p[i][j] = in ? exp_approx(v[j] - top) : 0.f;
                    all += p[i][j];
                }
            }
            all = group_sum<kLanes>(all);
        }
        if (tally && any) {
            const float each = __fdividef(1.0f, all);
#pragma unroll
            for (int i = 0; i < kItems; ++i)
#pragma unroll
                for (int j = 0; j < kVec; ++j) sum[i][j] += p[i][j] * each;
            taking += at == 0;
        }
        if (a.renormalise) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s) chosen += e[s];
            chosen = group_sum<kLanes>(chosen);
        } else {
            chosen = all;
        }
        if (r >= a.tokens) continue;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            e[s] = id[s] >= 0 ? __fdividef(e[s], chosen) : 0.f;
            if (tally && id[s] >= 0) atomicAdd(count + id[s], 1);
        }
        const int64_t to = r * a.topk;
        if constexpr (kLanes == 1)
            if (a.pairs) {
                *reinterpret_cast<int2*>(a.ids + to) = int2{id[0], id[1]};
                *reinterpret_cast<float2*>(a.weights + to) = float2{e[0], e[1]};
                continue;
            }
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            const int round = s * kLanes + at;
            if (round < a.topk) {
                a.ids[to + round] = id[s];
                a.weights[to + round] = e[s];
            }
        }
    }
    if (!tally) return;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
#pragma unroll
            for (int o = kLanes; o < 32; o <<= 1)
                sum[i][j] += __shfl_xor_sync(kAll, sum[i][j], o);
            const int c = (i * kLanes + at) * kVec + j;
            if ((threadIdx.x & 31) < kLanes && c < a.experts)
                sums[threadIdx.x / 32 * a.experts + c] = sum[i][j];
        }
    taking = __reduce_add_sync(kAll, taking);
    if ((threadIdx.x & 31) == 0) atomicAdd(count + a.experts, taking);
    __syncthreads();
    const bool alone = gridDim.x == 1;
    int32_t* counts = alone ? a.counts : a.part_counts + (int64_t)blockIdx.x * (a.experts + 1);
    for (int e = threadIdx.x; e <= a.experts; e += kThreads) {
        float v = 0.f;
        if (e < a.experts)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += sums[w * a.experts + e];
        if (!alone)
            a.partial[(int64_t)blockIdx.x * (a.experts + 1) + e] = v;
        else if (e < a.experts)
            sums[e] = v;
        counts[e] = count[e];
    }
    if (!alone || !a.loss) return;
    __syncthreads();
    if (threadIdx.x < 32) {
        const float loss = balance(sums, count, a.experts);
        if (threadIdx.x == 0) *a.loss = loss;
    }
}

// The blocks' sums and counts added up, eight columns a block and 128 threads
// a column; the last block to finish then has the loss.  Launched while the
// blocks are still at work, so that it is there when they end (2 us).
constexpr int kSumThreads = 1024, kSumColumns = 8;

__global__ void __launch_bounds__(kSumThreads) k_route_sum(RouteFwd a, int blocks) {
    constexpr int kParts = kSumThreads / kSumColumns;
    __shared__ float part[kSumColumns][kParts + 1];
    __shared__ int32_t parts[kSumColumns][kParts + 1];
    __shared__ bool last;
    const int c = threadIdx.x % kSumColumns, g = threadIdx.x / kSumColumns;
    const int column = blockIdx.x * kSumColumns + c, columns = a.experts + 1;
    cudaGridDependencySynchronize();
    float sum = 0.f;
    int32_t count = 0;
    if (column < columns) {
#pragma unroll 4
        for (int i = g; i < blocks; i += kParts) {
            sum += a.partial[(int64_t)i * columns + column];
            count += a.part_counts[(int64_t)i * columns + column];
        }
    }
    part[c][g] = sum;
    parts[c][g] = count;
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int mine = blockIdx.x * kSumColumns + warp;
    if (warp < kSumColumns && mine < columns) {
        sum = 0.f;
        count = 0;
#pragma unroll
        for (int i = 0; i < kParts / 32; ++i) {
            sum += part[warp][i * 32 + lane];
            count += parts[warp][i * 32 + lane];
        }
        sum = warp_sum(sum);
        count = __reduce_add_sync(kAll, count);
        if (lane == 0) {
            a.totals[mine] = sum;
            a.counts[mine] = count;
        }
    }
    if (!a.loss) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.ticket, 1u) + 1 == gridDim.x;
    __syncthreads();
    if (!last || threadIdx.x >= 32) return;
    __threadfence();
    const float loss = balance(a.totals, a.counts, a.experts);
    if (threadIdx.x == 0) *a.loss = loss;
}

struct RouteBwd {
    const void* logits;
    const int32_t *ids, *counts;     // counts: or null
    const float *grad_weights, *grad_loss;  // each or null
    void* grad;
    int32_t* d_status;
    int64_t ld, ldg, tokens;
    int topk, experts, renormalise;
};

// With p the softmax of a row, h_e = grad_loss * experts * share_e / tokens
// that take part, and g_j the gradient of the weight of choice j:
//   renormalised:  d_j = w_j (g_j - sum w g), w the softmax over the chosen
//   otherwise:     d_j = p_j g_j, and D = sum of d_j
//   grad_e = p_e (h_e - sum p h - D) + the d_j of the choices that are e
template <typename T, typename F>
__global__ void __launch_bounds__(kThreads) k_route_bwd(RouteBwd a) {
    constexpr int kVec = F::kVec, kLanes = F::kLanes, kItems = F::kItems, kSlots = F::kSlots;
    constexpr int kGroups = kThreads / kLanes;
    const int at = threadIdx.x % kLanes;
    float h[kItems][kVec] = {};
    if (a.grad_loss) {
        int pairs = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const int c = (i * kLanes + at) * kVec + j;
                const int n = c < a.experts ? a.counts[c] : 0;
                pairs += n;
                h[i][j] = (float)n;
            }
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) pairs += __shfl_xor_sync(kAll, pairs, o);
        const float scale = pairs > 0 ? *a.grad_loss * (float)a.experts /
                                            ((float)pairs * (float)a.counts[a.experts])
                                      : 0.f;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j) h[i][j] *= scale;
    }
    const int64_t step = (int64_t)gridDim.x * kGroups;
    // the next row and its choices come in while this one is worked on
    RawVec<T, kVec> ahead[kItems];
    int id_ahead[kSlots];
    float g_ahead[kSlots];
    const auto load = [&](int64_t r) {
        const T* x = static_cast<const T*>(a.logits) + r * a.ld + at * kVec;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            ahead[i] = r < a.tokens && (i * kLanes + at) * kVec < a.experts
                           ? load_raw<T, kVec>(x + i * kLanes * kVec)
                           : RawVec<T, kVec>{};
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            const int round = s * kLanes + at;
            const bool in = r < a.tokens && round < a.topk;
            id_ahead[s] = in ? a.ids[r * a.topk + round] : -1;
            g_ahead[s] = in && a.grad_weights ? a.grad_weights[r * a.topk + round] : 0.f;
        }
    };
    load((int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes);
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < a.tokens; r0 += step) {
        const int64_t r = r0 + threadIdx.x / kLanes;
        const T* row = static_cast<const T*>(a.logits) + r * a.ld;
        RawVec<T, kVec> raw[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) raw[i] = ahead[i];
        int id[kSlots];
        float g[kSlots], e[kSlots];
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            id[s] = id_ahead[s];
            if (id[s] < -1 || id[s] >= a.experts) {
                GS_BOUNDS_REPORT(a.d_status);
                id[s] = -1;
            }
            g[s] = id[s] >= 0 ? g_ahead[s] : 0.f;
            e[s] = 0.f;
        }
        load(r + step);
        // the first choice tells whether the row takes part
        const bool take = __shfl_sync(kAll, id[0], 0, kLanes) >= 0;
        // renormalised weights sum to one: what all gradients have in common
        // drops out, and before it is multiplied loses nothing of the rest
        if (a.renormalise) {
            const float common = __shfl_sync(kAll, g[0], 0, kLanes);
#pragma unroll
            for (int s = 0; s < kSlots; ++s) g[s] = id[s] >= 0 ? g[s] - common : 0.f;
        }
        float p[kItems][kVec];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            unpack<T, kVec>(raw[i], p[i]);
            const bool in = (i * kLanes + at) * kVec < a.experts;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (!in) p[i][j] = -INFINITY;
                top = fmaxf(top, p[i][j]);
            }
        }
        top = group_max<kLanes>(top);
        // the choices' exponentials, from their own logits
        float chosen = 0.f, mean = 0.f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            if (take && id[s] >= 0) e[s] = exp_approx(to_f(row[id[s]]) - top);
            chosen += e[s];
            mean += e[s] * g[s];
        }
        float all = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                p[i][j] = exp_approx(p[i][j] - top);
                all += p[i][j];
                dot += p[i][j] * h[i][j];
            }
        all = group_sum<kLanes>(all);
        const float each = __fdividef(1.0f, all);
        dot = a.grad_loss ? group_sum<kLanes>(dot) * each : 0.f;
        mean = group_sum<kLanes>(mean);
        chosen = a.renormalise ? group_sum<kLanes>(chosen) : all;
        mean = __fdividef(mean, chosen);  // renormalised: sum w g; otherwise D
        const float down = dot + (a.renormalise ? 0.f : mean);
        if (a.renormalise) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s) g[s] -= mean;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j) p[i][j] *= each * (h[i][j] - down);
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            const float d = __fdividef(e[s], chosen) * g[s];
            for (int l = 0; l < kLanes; ++l) {
                if (s * kLanes + l >= a.topk) break;
                const int index = __shfl_sync(kAll, id[s], l, kLanes);
                const float add = __shfl_sync(kAll, d, l, kLanes);
#pragma unroll
                for (int i = 0; i < kItems; ++i)
#pragma unroll
                    for (int j = 0; j < kVec; ++j)
                        if (index == (i * kLanes + at) * kVec + j) p[i][j] += add;
            }
        }
        if (r >= a.tokens) continue;
        T* out = static_cast<T*>(a.grad) + r * a.ldg + at * kVec;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (!take)
#pragma unroll
                for (int j = 0; j < kVec; ++j) p[i][j] = 0.f;
            if ((i * kLanes + at) * kVec < a.experts)
                store_vec<T, kVec>(out + i * kLanes * kVec, p[i]);
        }
    }
}

// Calls f with how rows of `experts` elements are spread: sixteen elements a lane
// keep what is done once a row, and exchanged between lanes, small beside what is
// done for each element, and many rows in flight.  Measured before the next row
// came in ahead (since then 27, 36 and 27 us): forward, 460800 rows of 32 float32
// and 230400 of 64 bfloat16, 31 and 38 us, 49 and 47 with eight lanes; 921600 of 16
// float32 in a thread each 33, in two lanes 33, in four 43.  The gradient's
// rows are written too, which wants neighbours: two lanes at least (921600 of 16
// float32: 31 us, a thread each 43; 900000 of 7 float16 18.5 and 22.6), single
// elements eight a lane up to 64 (460800 of 31: 35.5 us, sixteen a lane 47).
template <typename T, int kVec, bool kBackward, typename F>
void with_spread(int experts, int topk, F&& f) {
    const auto fits = [&](auto spread, int most) {
        return experts <= most && topk <= decltype(spread)::kChoices;
    };
    constexpr int k8 = 8 / kVec, k16 = 16 / kVec, k32 = 32 / kVec;
    if constexpr (!kBackward) {
        if (fits(Spread<kVec, 1, k8>{}, 8)) return f(Spread<kVec, 1, k8>{});
        if (fits(Spread<kVec, 1, k16>{}, 16)) return f(Spread<kVec, 1, k16>{});
    } else {
        if constexpr (kVec < 8)
            if (fits(Spread<kVec, 2, 4 / kVec>{}, 8)) return f(Spread<kVec, 2, 4 / kVec>{});
        if (fits(Spread<kVec, 2, k8>{}, 16)) return f(Spread<kVec, 2, k8>{});
    }
    if constexpr (kBackward && kVec == 1) {
        if (fits(Spread<1, 4, 8>{}, 32)) return f(Spread<1, 4, 8>{});
        if (fits(Spread<1, 8, 8>{}, 64)) return f(Spread<1, 8, 8>{});
    } else {
        if (fits(Spread<kVec, 2, k16>{}, 32)) return f(Spread<kVec, 2, k16>{});
        if (fits(Spread<kVec, 4, k16>{}, 64)) return f(Spread<kVec, 4, k16>{});
    }
    if (fits(Spread<kVec, 8, k16>{}, 128)) return f(Spread<kVec, 8, k16>{});
    if (fits(Spread<kVec, 16, k16>{}, 256)) return f(Spread<kVec, 16, k16>{});
    if (fits(Spread<kVec, 32, k8>{}, 256)) return f(Spread<kVec, 32, k8>{});
    if (fits(Spread<kVec, 32, k16>{}, 512)) return f(Spread<kVec, 32, k16>{});
    return f(Spread<kVec, 32, k32>{});
}

// Whole 16-byte vectors, or single elements.
template <typename T, typename F>
void with_route_width(uintptr_t all, F&& f) {
    if (all % 16 == 0) return f(std::integral_constant<int, 16 / (int)sizeof(T)>{});
    return f(std::integral_constant<int, 1>{});
}

int route_blocks(int64_t tokens, int groups, int cap) {
    return (int)std::min<int64_t>((tokens + groups - 1) / groups, cap);
}

size_t align_words(size_t words) { return (words + 63) / 64 * 64; }

}  // namespace

size_t route_workspace(int64_t tokens, int experts) {
    if (tokens <= kThreads / 32) return 0;  // one block, whatever the spread
    const size_t columns = experts + 1;
    // a block takes a row or more
    const size_t blocks = (size_t)std::min<int64_t>(std::max<int64_t>(tokens, 1), kMaxRouteBlocks);
    return 4 * (64 + align_words(columns) + 2 * align_words(blocks * columns));
}

void launch_route_fwd(const RouteArgs& n, const uint8_t* keep, int32_t* ids, float* weights,
                      int32_t* counts, float* loss, void* workspace, cudaStream_t s) {
    RouteFwd a{};
    a.logits = n.logits;
    a.keep = keep;
    a.ids = ids;
    a.counts = counts;
    a.weights = weights;
    a.loss = loss;
    a.ld = n.ld;
    a.tokens = n.tokens;
    a.topk = n.topk;
    a.experts = n.experts;
    a.renormalise = n.renormalise;
    a.pairs = n.topk == 2 &&
              ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(weights)) & 7u) == 0;
    const size_t columns = n.experts + 1;
    with_dtype(n.dtype, [&](auto t) {
        using T = decltype(t);
        const auto go = [&](auto form) {
            using F = decltype(form);
            const int groups = kThreads / F::kLanes;
            const auto kernel = k_route_fwd<T, F>;
            const auto smem = [&](int experts) {
                return counts ? ((size_t)experts + 1) * 4 + (size_t)kWarps * experts * 4 : 0;
            };
            static PerDevice resident;
            const int most = F::kVec * F::kLanes * F::kItems;
            const int blocks = route_blocks(
                n.tokens, groups,
                std::min(kMaxRouteBlocks,
                         resident_blocks(resident, kernel,
                                         ((size_t)most + 1) * 4 + (size_t)kWarps * most * 4,
                                         kThreads)));
            if (counts) {
                uint32_t* w = static_cast<uint32_t*>(workspace);
                a.ticket = w;
                a.totals = reinterpret_cast<float*>(w + 64);
                a.partial = a.totals + align_words(columns);
                a.part_counts = reinterpret_cast<int32_t*>(a.partial + align_words(blocks * columns));
            }
            kernel<<<blocks, kThreads, smem(n.experts), s>>>(a);
            if (counts && blocks > 1) {
                cudaLaunchConfig_t config = {};
                config.gridDim = dim3((unsigned)((columns + kSumColumns - 1) / kSumColumns));
                config.blockDim = dim3(kSumThreads);
                config.stream = s;
                cudaLaunchAttribute early = {};
                early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
                early.val.programmaticStreamSerializationAllowed = 1;
                config.attrs = &early;
                config.numAttrs = 1;
                (void)cudaLaunchKernelEx(&config, k_route_sum, a, blocks);
            }
        };
        with_route_width<T>(row_bits<T>(n.logits, n.ld) | (uintptr_t)(n.experts * sizeof(T)),
                            [&](auto width) {
                                with_spread<T, decltype(width)::value, false>(n.experts, n.topk, go);
                            });
    });
}

void launch_route_bwd(const RouteArgs& n, const int32_t* ids, const int32_t* counts,
                      const float* grad_weights, const float* grad_loss, void* grad, int64_t ldg,
                      int32_t* d_status, cudaStream_t s) {
    const RouteBwd a{n.logits, ids,  counts, grad_weights, grad_loss, grad,         d_status,
                     n.ld,     ldg, n.tokens, n.topk,      n.experts, n.renormalise};
    with_dtype(n.dtype, [&](auto t) {
        using T = decltype(t);
        const auto go = [&](auto form) {
            using F = decltype(form);
            const auto kernel = k_route_bwd<T, F>;
            static PerDevice resident;
            const int blocks = route_blocks(n.tokens, kThreads / F::kLanes,
                                            resident_blocks(resident, kernel, 0, kThreads));
            kernel<<<blocks, kThreads, 0, s>>>(a);
        };
        with_route_width<T>(row_bits<T>(n.logits, n.ld) | row_bits<T>(grad, ldg) |
                                (uintptr_t)(n.experts * sizeof(T)),
                            [&](auto width) {
                                with_spread<T, decltype(width)::value, true>(n.experts, n.topk, go);
                            });
    });
}

}  // namespace gs
