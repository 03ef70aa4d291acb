// Layer norm over the channels of each row, forward and backward.
#include <cstdint>

#include "gs_head_internal.h"
#include "gs_types.cuh"

namespace gs {

namespace {

constexpr int kNormThreads = 128;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kMaxSlices = 1216;

// One warp a row, three passes over the row.
template <typename T, typename P>
__global__ void __launch_bounds__(kNormThreads)
    k_norm_fwd(const T* __restrict__ x, int64_t ldx, const P* __restrict__ w,
               const P* __restrict__ b, int64_t rows, int channels, float eps, T* __restrict__ y,
               int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd) {
    const int lane = threadIdx.x & 31;
    for (int64_t r = blockIdx.x * (int64_t)kNormWarps + threadIdx.x / 32; r < rows;
         r += (int64_t)gridDim.x * kNormWarps) {
        const T* xr = x + r * ldx;
        float s = 0.f;
        for (int c = lane; c < channels; c += 32) s += to_f(xr[c]);
        const float mu = warp_sum(s) / (float)channels;
        s = 0.f;
        for (int c = lane; c < channels; c += 32) {
            const float d = to_f(xr[c]) - mu;
            s += d * d;
        }
        const float rs = 1.0f / sqrtf(warp_sum(s) / (float)channels + eps);
        for (int c = lane; c < channels; c += 32) {
            float v = (to_f(xr[c]) - mu) * rs;
            if (w) v *= to_f(w[c]);
            if (b) v += to_f(b[c]);
            y[r * ldy + c] = from_f<T>(v);
        }
        if (mean && lane == 0) {
            mean[r] = mu;
            rstd[r] = rs;
        }
    }
}

template <typename T, typename P>
__global__ void __launch_bounds__(kNormThreads)
    k_norm_bwd_x(const T* __restrict__ gy, int64_t ldgy, const T* __restrict__ x, int64_t ldx,
                 const P* __restrict__ w, const float* __restrict__ mean,
                 const float* __restrict__ rstd, int64_t rows, int channels, T* __restrict__ gx,
                 int64_t ldgx) {
    const int lane = threadIdx.x & 31;
    for (int64_t r = blockIdx.x * (int64_t)kNormWarps + threadIdx.x / 32; r < rows;
         r += (int64_t)gridDim.x * kNormWarps) {
        const float mu = mean[r], rs = rstd[r];
        float s0 = 0.f, s1 = 0.f;
        for (int c = lane; c < channels; c += 32) {
            const float g = to_f(gy[r * ldgy + c]) * (w ? to_f(w[c]) : 1.0f);
            s0 += g;
            s1 += g * ((to_f(x[r * ldx + c]) - mu) * rs);
        }
        s0 = warp_sum(s0) / (float)channels;
        s1 = warp_sum(s1) / (float)channels;
        for (int c = lane; c < channels; c += 32) {
            const float g = to_f(gy[r * ldgy + c]) * (w ? to_f(w[c]) : 1.0f);
            const float xh = (to_f(x[r * ldx + c]) - mu) * rs;
            gx[r * ldgx + c] = from_f<T>(rs * (g - s0 - xh * s1));
        }
    }
}

// Partial column sums of grad_y * xh and grad_y over one slice of rows.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    k_norm_bwd_params(const T* __restrict__ gy, int64_t ldgy, const T* __restrict__ x,
                      int64_t ldx, const float* __restrict__ mean,
                      const float* __restrict__ rstd, int64_t rows, int channels,
                      float* __restrict__ partial) {
    const int c = blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= channels) return;
    const int64_t per = (rows + gridDim.y - 1) / gridDim.y;
    const int64_t r0 = blockIdx.y * per, r1 = min(rows, r0 + per);
    float sw = 0.f, sb = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float g = to_f(gy[r * ldgy + c]);
        sw += g * ((to_f(x[r * ldx + c]) - mean[r]) * rstd[r]);
        sb += g;
    }
    float* out = partial + (int64_t)blockIdx.y * 2 * channels;
    out[c] = sw;
    out[channels + c] = sb;
}

template <typename P>
__global__ void __launch_bounds__(kNormThreads)
    k_norm_bwd_reduce(const float* __restrict__ partial, int slices, int channels,
                      P* __restrict__ gw, P* __restrict__ gb) {
    const int c = blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= channels) return;
    float sw = 0.f, sb = 0.f;
    for (int i = 0; i < slices; ++i) {
        sw += partial[(int64_t)i * 2 * channels + c];
        sb += partial[(int64_t)i * 2 * channels + channels + c];
    }
    if (gw) gw[c] = from_f<P>(sw);
    if (gb) gb[c] = from_f<P>(sb);
}

int norm_blocks(int64_t rows) {
    const int64_t b = (rows + kNormWarps - 1) / kNormWarps;
    return (int)(b < 152 * 64 ? b : 152 * 64);
}

template <typename F>
void with_types(int dtype, int param_dtype, F&& f) {
    with_dtype(dtype, [&](auto t) {
        if (param_dtype == dtype)
            f(t, t);
        else
            f(t, float{});
    });
}

}  // namespace

int norm_bwd_slices(int64_t rows, int channels) {
    int64_t s = (rows + 63) / 64;
    if (s > kMaxSlices) s = kMaxSlices;
    return (int)(s < 1 ? 1 : s);
}

void launch_norm_fwd(const NormArgs& a, const void* bias, float eps, void* y, int64_t ldy,
                     float* mean, float* rstd, cudaStream_t s) {
    with_types(a.dtype, a.param_dtype, [&](auto t, auto p) {
        using T = decltype(t);
        using P = decltype(p);
        k_norm_fwd<T, P><<<norm_blocks(a.rows), kNormThreads, 0, s>>>(
            (const T*)a.x, a.ldx, (const P*)a.weight, (const P*)bias, a.rows, a.channels, eps,
            (T*)y, ldy, mean, rstd);
    });
}

void launch_norm_bwd(const NormArgs& a, const void* grad_y, int64_t ldgy, const float* mean,
                     const float* rstd, void* grad_x, int64_t ldgx, void* grad_weight,
                     void* grad_bias, float* partial, cudaStream_t s) {
    with_types(a.dtype, a.param_dtype, [&](auto t, auto p) {
        using T = decltype(t);
        using P = decltype(p);
        if (grad_x && a.rows > 0)
            k_norm_bwd_x<T, P><<<norm_blocks(a.rows), kNormThreads, 0, s>>>(
                (const T*)grad_y, ldgy, (const T*)a.x, a.ldx, (const P*)a.weight, mean, rstd,
                a.rows, a.channels, (T*)grad_x, ldgx);
        if (grad_weight || grad_bias) {
            const int cb = (a.channels + kNormThreads - 1) / kNormThreads;
            const int slices = norm_bwd_slices(a.rows, a.channels);
            k_norm_bwd_params<T><<<dim3(cb, slices), kNormThreads, 0, s>>>(
                (const T*)grad_y, ldgy, (const T*)a.x, a.ldx, mean, rstd, a.rows, a.channels,
                partial);
            k_norm_bwd_reduce<P><<<cb, kNormThreads, 0, s>>>(partial, slices, a.channels,
                                                             (P*)grad_weight, (P*)grad_bias);
        }
    });
}

}  // namespace gs
