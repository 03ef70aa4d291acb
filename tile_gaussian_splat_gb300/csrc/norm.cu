// Layer norm over the channels of each row, forward and backward.
//
// Both directions read each input once and write each output once, so they
// are bound by memory bandwidth.  Up to 4096 channels a row lives in the
// registers of kLanes lanes (the mean, the variance about it and the output
// come from one read), a lane owns the same channels of every row it meets --
// weight and bias are loaded once, the sums of their gradients stay in
// registers -- and several rows are loaded before the first is used.  Longer
// rows take one block each and are read again from the cache.
// Forward, 2073600 rows of 64 of 67 float32 channels: 171 us, 6.3 TB/s (94 % of
// a copy's rate).  Backward, 921600 x 128 bfloat16: 130 us, 5.5 TB/s, bound by
// the loads that 12 warps of 161 registers keep in flight.
#include <algorithm>
#include <cstdint>

#include "gs_head_internal.h"
#include "gs_types.cuh"

namespace gs {

namespace {

constexpr int kNormThreads = kRowThreads;
constexpr int kLongThreads = 256;
// Longest row kept in registers.  Through the cache instead, 200000 x 1024
// float32 took 564 us forward and 1596 backward, in registers 259 and 393.
constexpr int kRegisterChannels = 4096;
constexpr int kMaxSlices = 152 * 16;  // blocks that leave partial parameter gradients

struct NormFwd {
    const void *x, *weight, *bias;
    void* y;
    float *mean, *rstd;
    int64_t ldx, ldy, rows;
    int channels, param_dtype;
    float eps;
};

struct NormBwd {
    const void *gy, *x, *weight;
    const float *mean, *rstd;
    void* gx;
    float* partial;  // or null
    int64_t ldgy, ldx, ldgx, rows;
    int channels, param_dtype;
};

// kVec elements per access, kLanes lanes a row, kItems accesses a lane and
// row, kRows rows of a lane in flight.
template <typename T, int kVec, int kLanes, int kItems, int kRows>
__global__ void __launch_bounds__(kNormThreads) k_norm_fwd(NormFwd a) {
    constexpr int kGroups = kNormThreads / kLanes;
    __shared__ RowScratch scratch;
    int half = 0;
    const int at = threadIdx.x % kLanes;
    float w[kItems][kVec], b[kItems][kVec];
    bool in[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int c = (i * kLanes + at) * kVec;
        in[i] = c < a.channels;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            w[i][j] = in[i] && a.weight ? load_any(a.weight, a.param_dtype, c + j) : 1.f;
            b[i][j] = in[i] && a.bias ? load_any(a.bias, a.param_dtype, c + j) : 0.f;
        }
    }
    const float n = (float)a.channels;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < a.rows; r0 += step * kRows) {
        RawVec<T, kVec> raw[kRows][kItems];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t r = r0 + u * step + threadIdx.x / kLanes;
            const T* x = static_cast<const T*>(a.x) + r * a.ldx + at * kVec;
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                raw[u][i] = r < a.rows && in[i] ? load_raw<T, kVec>(x + i * kLanes * kVec)
                                                : RawVec<T, kVec>{};
        }
        float mu[kRows], rs[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            mu[u] = 0.f;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                float v[kVec];
                unpack<T, kVec>(raw[u][i], v);
#pragma unroll
                for (int j = 0; j < kVec; ++j) mu[u] += v[j];
            }
        }
        row_sums<kLanes, kRows>(mu, scratch, half);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            mu[u] /= n;
            rs[u] = 0.f;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                float v[kVec];
                unpack<T, kVec>(raw[u][i], v);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const float d = in[i] ? v[j] - mu[u] : 0.f;
                    rs[u] += d * d;
                }
            }
        }
        row_sums<kLanes, kRows>(rs, scratch, half);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t r = r0 + u * step + threadIdx.x / kLanes;
            if (r >= a.rows) continue;
            rs[u] = 1.0f / sqrtf(rs[u] / n + a.eps);
            T* y = static_cast<T*>(a.y) + r * a.ldy + at * kVec;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                float v[kVec];
                unpack<T, kVec>(raw[u][i], v);
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[j] = (v[j] - mu[u]) * rs[u] * w[i][j] + b[i][j];
                if (in[i]) store_vec<T, kVec>(y + i * kLanes * kVec, v);
            }
            if (a.mean && at == 0) {
                a.mean[r] = mu[u];
                a.rstd[r] = rs[u];
            }
        }
    }
}

// grad_x, and per block the sums over its rows of grad_y * xh and grad_y.
template <typename T, int kVec, int kLanes, int kItems, int kRows>
__global__ void __launch_bounds__(kNormThreads) k_norm_bwd(NormBwd a) {
    constexpr int kGroups = kNormThreads / kLanes;
    extern __shared__ float sums[];  // [kGroups - 1][2][channels]
    __shared__ RowScratch scratch;
    int half = 0;
    const int at = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    float w[kItems][kVec], gw[kItems][kVec], gb[kItems][kVec];
    bool in[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int c = (i * kLanes + at) * kVec;
        in[i] = c < a.channels;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            w[i][j] = in[i] && a.weight ? load_any(a.weight, a.param_dtype, c + j) : 1.f;
            gw[i][j] = gb[i][j] = 0.f;
        }
    }
    const float n = (float)a.channels;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups; r0 < a.rows; r0 += step * kRows) {
        RawVec<T, kVec> rx[kRows][kItems], rg[kRows][kItems];
        float mu[kRows], rs[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t r = r0 + u * step + group;
            const bool here = r < a.rows;
            const T* x = static_cast<const T*>(a.x) + r * a.ldx + at * kVec;
            const T* g = static_cast<const T*>(a.gy) + r * a.ldgy + at * kVec;
            mu[u] = here ? a.mean[r] : 0.f;
            rs[u] = here ? a.rstd[r] : 0.f;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const bool take = here && in[i];
                rx[u][i] = take ? load_raw<T, kVec>(x + i * kLanes * kVec) : RawVec<T, kVec>{};
                rg[u][i] = take ? load_raw<T, kVec>(g + i * kLanes * kVec) : RawVec<T, kVec>{};
            }
        }
        float s01[2 * kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                float x[kVec], g[kVec];
                unpack<T, kVec>(rx[u][i], x);
                unpack<T, kVec>(rg[u][i], g);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const float xh = in[i] ? (x[j] - mu[u]) * rs[u] : 0.f;
                    gw[i][j] += g[j] * xh;
                    gb[i][j] += g[j];
                    const float gn = g[j] * w[i][j];
                    s0 += gn;
                    s1 += gn * xh;
                }
            }
            s01[2 * u] = s0;
            s01[2 * u + 1] = s1;
        }
        if (!a.gx) continue;
        row_sums<kLanes, 2 * kRows>(s01, scratch, half);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t r = r0 + u * step + group;
            const float s0 = s01[2 * u] / n, s1 = s01[2 * u + 1] / n;
            if (r >= a.rows) continue;
            T* out = static_cast<T*>(a.gx) + r * a.ldgx + at * kVec;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                float x[kVec], g[kVec];
                unpack<T, kVec>(rx[u][i], x);
                unpack<T, kVec>(rg[u][i], g);
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    x[j] = rs[u] * (g[j] * w[i][j] - s0 - (x[j] - mu[u]) * rs[u] * s1);
                if (in[i]) store_vec<T, kVec>(out + i * kLanes * kVec, x);
            }
        }
    }
    if (!a.partial) return;
    if (group > 0) {
        float* mine = sums + (int64_t)(group - 1) * 2 * a.channels;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (in[i]) {
                    const int c = (i * kLanes + at) * kVec + j;
                    mine[c] = gw[i][j];
                    mine[a.channels + c] = gb[i][j];
                }
    }
    __syncthreads();
    if (group > 0) return;
    float* out = a.partial + (int64_t)blockIdx.x * 2 * a.channels;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (in[i]) {
                const int c = (i * kLanes + at) * kVec + j;
                for (int q = 0; q < kGroups - 1; ++q) {
                    gw[i][j] += sums[q * 2 * a.channels + c];
                    gb[i][j] += sums[q * 2 * a.channels + a.channels + c];
                }
                out[c] = gw[i][j];
                out[a.channels + c] = gb[i][j];
            }
}

// The block's sum of v, in every thread.  `scratch`: one float a warp.
__device__ __forceinline__ float block_sum(float v, float* scratch) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kLongThreads / 32; ++i) v += scratch[i];
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads) k_norm_fwd_long(NormFwd a) {
    __shared__ float scratch[kLongThreads / 32];
    const float n = (float)a.channels;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.ldx;
        float s = 0.f;
        for (int c = threadIdx.x; c < a.channels; c += kLongThreads) s += to_f(x[c]);
        const float mu = block_sum(s, scratch) / n;
        s = 0.f;
        for (int c = threadIdx.x; c < a.channels; c += kLongThreads) {
            const float d = to_f(x[c]) - mu;
            s += d * d;
        }
        const float rs = 1.0f / sqrtf(block_sum(s, scratch) / n + a.eps);
        T* y = static_cast<T*>(a.y) + r * a.ldy;
        for (int c = threadIdx.x; c < a.channels; c += kLongThreads) {
            float v = (to_f(x[c]) - mu) * rs;
            if (a.weight) v *= load_any(a.weight, a.param_dtype, c);
            if (a.bias) v += load_any(a.bias, a.param_dtype, c);
            y[c] = from_f<T>(v);
        }
        if (a.mean && threadIdx.x == 0) {
            a.mean[r] = mu;
            a.rstd[r] = rs;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads) k_norm_bwd_long(NormBwd a) {
    __shared__ float scratch[kLongThreads / 32];
    const float n = (float)a.channels;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.ldx;
        const T* gy = static_cast<const T*>(a.gy) + r * a.ldgy;
        const float mu = a.mean[r], rs = a.rstd[r];
        float s0 = 0.f, s1 = 0.f;
        for (int c = threadIdx.x; c < a.channels; c += kLongThreads) {
            const float g =
                to_f(gy[c]) * (a.weight ? load_any(a.weight, a.param_dtype, c) : 1.f);
            s0 += g;
            s1 += g * ((to_f(x[c]) - mu) * rs);
        }
        s0 = block_sum(s0, scratch) / n;
        s1 = block_sum(s1, scratch) / n;
        T* gx = static_cast<T*>(a.gx) + r * a.ldgx;
        for (int c = threadIdx.x; c < a.channels; c += kLongThreads) {
            const float g =
                to_f(gy[c]) * (a.weight ? load_any(a.weight, a.param_dtype, c) : 1.f);
            gx[c] = from_f<T>(rs * (g - s0 - (to_f(x[c]) - mu) * rs * s1));
        }
    }
}

// Long rows' parameter sums: a thread a channel, a block a slice of the rows.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_norm_params_long(NormBwd a) {
    const int c = blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= a.channels) return;
    const int64_t per = (a.rows + gridDim.y - 1) / gridDim.y;
    const int64_t r0 = blockIdx.y * per, r1 = min(a.rows, r0 + per);
    float sw = 0.f, sb = 0.f;
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) {
        const float g = to_f(static_cast<const T*>(a.gy)[r * a.ldgy + c]);
        const float x = to_f(static_cast<const T*>(a.x)[r * a.ldx + c]);
        sw += g * ((x - a.mean[r]) * a.rstd[r]);
        sb += g;
    }
    float* out = a.partial + (int64_t)blockIdx.y * 2 * a.channels;
    out[c] = sw;
    out[a.channels + c] = sb;
}

// The slices' partial sums added up: eight channels of one of the two sums a
// block, 128 threads a channel, so that a thread meets few slices one after
// the other (32 threads a channel took 7.5 us for 760 slices of 1021 channels,
// eight 18 us, these 6.5).
constexpr int kSumThreads = 1024, kSumChannels = 8;

__global__ void __launch_bounds__(kSumThreads)
    k_norm_params_sum(const float* __restrict__ partial, int slices, int channels,
                      int param_dtype, void* gw, void* gb) {
    constexpr int kParts = kSumThreads / kSumChannels;
    __shared__ float part[kSumChannels][kParts + 1];
    void* out = blockIdx.y == 0 ? gw : gb;
    if (!out) return;
    const int c = threadIdx.x % kSumChannels, g = threadIdx.x / kSumChannels;
    const int channel = blockIdx.x * kSumChannels + c;
    float sum = 0.f;
    if (channel < channels) {
        const float* p = partial + blockIdx.y * channels + channel;
#pragma unroll 8
        for (int i = g; i < slices; i += kParts) sum += p[(int64_t)i * 2 * channels];
    }
    part[c][g] = sum;
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (warp >= kSumChannels) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kParts / 32; ++i) sum += part[warp][i * 32 + lane];
    sum = warp_sum(sum);
    const int mine = blockIdx.x * kSumChannels + warp;
    if (lane == 0 && mine < channels) store_any(out, param_dtype, mine, sum);
}

// Calls f with the form for rows of `channels` elements.  Few lanes a row
// with several accesses each keep the instructions spent on sums across lanes
// and on addresses small beside those on elements (with 32 lanes and two
// elements a lane the forward over 64 channels was bound by instruction issue:
// 279 us for 2 M rows, against 162 us for its bytes); a lane still holds at
// most 16 elements of up to 1024 channels (32 beyond), so that many rows are in
// flight.
template <typename T, int kVec, typename F>
void with_form(int channels, F&& f) {
    const int n = (channels + kVec - 1) / kVec;
    if constexpr (kVec <= 2) {
        if (n <= 32) return f(Form<kVec, 8, 4, 4>{});
        if (n <= 64) return f(Form<kVec, 8, 8, 2>{});
        if (n <= 96) return f(Form<kVec, 16, 6, 2>{});
        if (n <= 128) return f(Form<kVec, 16, 8, 2>{});
        if (n <= 192) return f(Form<kVec, 32, 6, 2>{});
        if (n <= 256) return f(Form<kVec, 32, 8, 2>{});
        if (n <= 512) return f(Form<kVec, 128, 4, 4>{});
        if (n <= 1024) return f(Form<kVec, 128, 8, 2>{});
        if (n <= 2048) return f(Form<kVec, 128, 16, 1>{});
        if constexpr (kVec == 1) return f(Form<1, 128, 32, 1>{});
    } else {
        if (n <= 8) return f(Form<kVec, 8, 1, 4>{});
        if (n <= 16) return f(Form<kVec, 8, 2, 2>{});
        if (n <= 32) return f(Form<kVec, 32, 1, 4>{});
        if (n <= 64) return f(Form<kVec, 32, 2, 2>{});
        if constexpr (kVec == 8) {
            if (n <= 128) return f(Form<8, 128, 1, 4>{});
        } else {
            if (n <= 128) return f(Form<kVec, 32, 4, 1>{});
        }
        if (n <= 256) return f(Form<kVec, 128, 2, 2>{});
        if (n <= 512) return f(Form<kVec, 128, 4, 1>{});
        if constexpr (kVec == 4) return f(Form<4, 128, 8, 1>{});
    }
}

int blocks_for(int64_t rows, int groups, int cap) {
    return (int)std::min<int64_t>((rows + groups - 1) / groups, cap);
}

}  // namespace

int norm_bwd_slices(int64_t rows, int channels) {
    return (int)std::min<int64_t>(std::max<int64_t>((rows + 3) / 4, 1), kMaxSlices);
}

void launch_norm_fwd(const NormArgs& n, const void* bias, float eps, void* y, int64_t ldy,
                     float* mean, float* rstd, cudaStream_t s) {
    const NormFwd a{n.x, n.weight, bias, y, mean, rstd, n.ldx, ldy, n.rows, n.channels,
                    n.param_dtype, eps};
    with_dtype(n.dtype, [&](auto t) {
        using T = decltype(t);
        if (n.channels > kRegisterChannels) {
            k_norm_fwd_long<T><<<blocks_for(n.rows, 1, 152 * 8), kLongThreads, 0, s>>>(a);
            return;
        }
        const auto go = [&](auto form) {
            using F = decltype(form);
            const int groups = kNormThreads / F::kLanes;
            const auto kernel = k_norm_fwd<T, F::kVec, F::kLanes, F::kItems, F::kRows>;
            static PerDevice resident;
            const int blocks = blocks_for(n.rows, groups, resident_blocks(resident, kernel, 0));
            kernel<<<blocks, kNormThreads, 0, s>>>(a);
        };
        with_width<T>(row_bits<T>(n.x, n.ldx) | row_bits<T>(y, ldy) |
                          (uintptr_t)(n.channels * sizeof(T)),
                      [&](auto width) { with_form<T, decltype(width)::value>(n.channels, go); });
    });
}

void launch_norm_bwd(const NormArgs& n, const void* grad_y, int64_t ldgy, const float* mean,
                     const float* rstd, void* grad_x, int64_t ldgx, void* grad_weight,
                     void* grad_bias, float* partial, cudaStream_t s) {
    const bool params = grad_weight || grad_bias;
    const NormBwd a{grad_y, n.x, n.weight, mean, rstd, grad_x, params ? partial : nullptr, ldgy,
                    n.ldx, ldgx, n.rows, n.channels, n.param_dtype};
    int slices = 0;
    if (n.rows > 0) with_dtype(n.dtype, [&](auto t) {
        using T = decltype(t);
        if (n.channels > kRegisterChannels) {
            if (grad_x)
                k_norm_bwd_long<T><<<blocks_for(n.rows, 1, 152 * 8), kLongThreads, 0, s>>>(a);
            if (params) {
                slices = blocks_for(n.rows, 64, norm_bwd_slices(n.rows, n.channels));
                k_norm_params_long<T>
                    <<<dim3((n.channels + kNormThreads - 1) / kNormThreads, slices),
                       kNormThreads, 0, s>>>(a);
            }
            return;
        }
        const auto go = [&](auto form) {
            using F = decltype(form);
            const int groups = kNormThreads / F::kLanes;
            const size_t smem = params ? (groups - 1) * 2 * n.channels * sizeof(float) : 0;
            const auto kernel = k_norm_bwd<T, F::kVec, F::kLanes, F::kItems, F::kRows>;
            static PerDevice resident;
            const size_t most = (groups - 1) * 2 * F::kVec * F::kLanes * F::kItems * sizeof(float);
            slices = blocks_for(n.rows, groups,
                                std::min(norm_bwd_slices(n.rows, n.channels),
                                         resident_blocks(resident, kernel, most)));
            kernel<<<slices, kNormThreads, smem, s>>>(a);
        };
        with_width<T>(row_bits<T>(n.x, n.ldx) | row_bits<T>(grad_y, ldgy) |
                          (grad_x ? row_bits<T>(grad_x, ldgx) : 0) |
                          (uintptr_t)(n.channels * sizeof(T)),
                      [&](auto width) { with_form<T, decltype(width)::value>(n.channels, go); });
    });
    if (params)
        k_norm_params_sum<<<dim3((n.channels + kSumChannels - 1) / kSumChannels, 2), kSumThreads, 0,
                            s>>>(
            partial, slices, n.channels, n.param_dtype, grad_weight, grad_bias);
}

}  // namespace gs
