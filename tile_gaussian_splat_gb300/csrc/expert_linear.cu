// Every expert's matrix product over its sorted rows, and its gradients.
#include <cstdint>

#include "gs_device.cuh"
#include "gs_head_internal.h"
#include "gs_types.cuh"

namespace gs {

namespace {

constexpr int kTile = 64;        // rows and columns of a block's output tile
constexpr int kDepth = 16;       // terms of the sum staged at a time
constexpr int kTileThreads = 256;  // 16 x 16, each 4 x 4 outputs

// Rows [begin, end) of expert e; e == experts names the rows of no expert.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int experts, int64_t rows,
                                            int e, int64_t* begin, int64_t* end,
                                            int32_t* d_status) {
    const int64_t b = offsets[e], n = e == experts ? rows : offsets[e + 1];
    if (b < 0 || b > n || n > rows) GS_BOUNDS_REPORT(d_status);
    *begin = min(max(b, (int64_t)0), rows);
    *end = max(*begin, min(n, rows));
}

// The expert and first row of row tile `tile` (tiles of `height` rows, each
// expert's rows starting a new tile).  False if there is no such tile.
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int experts, int64_t rows,
                                          int64_t tile, int height, int* expert, int64_t* row0,
                                          int64_t* row1, int32_t* d_status) {
    for (int e = 0; e <= experts; ++e) {
        int64_t b, n;
        expert_rows(offsets, experts, rows, e, &b, &n, d_status);
        const int64_t tiles = (n - b + height - 1) / height;
        if (tile < tiles) {
            *expert = e;
            *row0 = b + tile * height;
            *row1 = min(n, *row0 + height);
            return true;
        }
        tile -= tiles;
    }
    return false;
}

// acc += A^T B over kDepth staged terms.
__device__ __forceinline__ void tile_step(const float (*sa)[kTile + 4], const float (*sb)[kTile + 4],
                                          int ty, int tx, float (*acc)[4]) {
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = sa[k][ty * 4 + i];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = sb[k][tx * 4 + i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
}

// out[r, n] = sum_k a[r, k] * w[e][n * sn + k * sk] + bias[e][n]
template <typename T>
__global__ void __launch_bounds__(kTileThreads)
    k_rows_product(LinearArgs g, const T* __restrict__ a, int depth, const T* __restrict__ w,
                   int64_t sn, int64_t sk, const T* __restrict__ bias, int width,
                   T* __restrict__ out) {
    __shared__ float sa[kDepth][kTile + 4], sb[kDepth][kTile + 4];
    int e;
    int64_t r0, r1;
    if (!find_tile(g.offsets, g.experts, g.rows, blockIdx.x, kTile, &e, &r0, &r1, g.d_status))
        return;
    const int n0 = blockIdx.y * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    if (e < g.experts) {
        const T* we = w + (int64_t)e * g.in * g.out;
        for (int k0 = 0; k0 < depth; k0 += kDepth) {
            for (int i = threadIdx.x; i < kTile * kDepth; i += kTileThreads) {
                const int k = i % kDepth, r = i / kDepth;
                sa[k][r] = r0 + r < r1 && k0 + k < depth
                               ? to_f(a[(r0 + r) * depth + k0 + k]) : 0.f;
            }
            for (int i = threadIdx.x; i < kTile * kDepth; i += kTileThreads) {
                const int k = sk == 1 ? i % kDepth : i / kTile;
                const int n = sk == 1 ? i / kDepth : i % kTile;
                sb[k][n] = n0 + n < width && k0 + k < depth
                               ? to_f(we[(n0 + n) * sn + (k0 + k) * sk]) : 0.f;
            }
            __syncthreads();
            tile_step(sa, sb, ty, tx, acc);
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + ty * 4 + i;
            const int n = n0 + tx * 4 + j;
            if (r >= r1 || n >= width) continue;
            float v = acc[i][j];
            if (bias && e < g.experts) v += to_f(bias[(int64_t)e * width + n]);
            out[r * width + n] = from_f<T>(v);
        }
}

// grad_weight[e][m, n] = sum over the expert's rows of gys[r, m] * xs[r, n]
template <typename T>
__global__ void __launch_bounds__(kTileThreads)
    k_weight_grad(LinearArgs g, const T* __restrict__ gys, const T* __restrict__ xs,
                  T* __restrict__ gw) {
    __shared__ float sa[kDepth][kTile + 4], sb[kDepth][kTile + 4];
    const int e = blockIdx.z, m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    int64_t r0, r1;
    expert_rows(g.offsets, g.experts, g.rows, e, &r0, &r1, g.d_status);
    float acc[4][4] = {};
    for (int64_t r = r0; r < r1; r += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += kTileThreads) {
            const int k = i / kTile, c = i % kTile;
            const bool in = r + k < r1;
            sa[k][c] = in && m0 + c < g.out ? to_f(gys[(r + k) * g.out + m0 + c]) : 0.f;
            sb[k][c] = in && n0 + c < g.in ? to_f(xs[(r + k) * g.in + n0 + c]) : 0.f;
        }
        __syncthreads();
        tile_step(sa, sb, ty, tx, acc);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m < g.out && n < g.in)
                gw[((int64_t)e * g.out + m) * g.in + n] = from_f<T>(acc[i][j]);
        }
}

template <typename T>
__global__ void __launch_bounds__(kTileThreads)
    k_bias_grad(LinearArgs g, const T* __restrict__ gys, T* __restrict__ gb) {
    const int e = blockIdx.y, m = blockIdx.x * kTileThreads + threadIdx.x;
    int64_t r0, r1;
    expert_rows(g.offsets, g.experts, g.rows, e, &r0, &r1, g.d_status);
    if (m >= g.out) return;
    float sum = 0.f;
    for (int64_t r = r0; r < r1; ++r) sum += to_f(gys[r * g.out + m]);
    gb[(int64_t)e * g.out + m] = from_f<T>(sum);
}

dim3 rows_grid(const LinearArgs& a, int width) {
    // each expert (and the rows of none) can leave one tile part-filled
    return dim3((unsigned)((a.rows + kTile - 1) / kTile + a.experts + 1),
                (unsigned)((width + kTile - 1) / kTile));
}

}  // namespace

void launch_linear_fwd(const LinearArgs& a, const void* xs, const void* weight, const void* bias,
                       void* ys, cudaStream_t s) {
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        k_rows_product<T><<<rows_grid(a, a.out), kTileThreads, 0, s>>>(
            a, (const T*)xs, a.in, (const T*)weight, a.in, 1, (const T*)bias, a.out, (T*)ys);
    });
}

void launch_linear_dx(const LinearArgs& a, const void* grad_ys, const void* weight, void* grad_xs,
                      cudaStream_t s) {
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        k_rows_product<T><<<rows_grid(a, a.in), kTileThreads, 0, s>>>(
            a, (const T*)grad_ys, a.out, (const T*)weight, 1, a.in, nullptr, a.in, (T*)grad_xs);
    });
}

void launch_linear_dw(const LinearArgs& a, const void* grad_ys, const void* xs,
                      void* grad_weight, cudaStream_t s) {
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        const dim3 grid((a.in + kTile - 1) / kTile, (a.out + kTile - 1) / kTile, a.experts);
        k_weight_grad<T><<<grid, kTileThreads, 0, s>>>(a, (const T*)grad_ys, (const T*)xs,
                                                       (T*)grad_weight);
    });
}

void launch_linear_db(const LinearArgs& a, const void* grad_ys, void* grad_bias, cudaStream_t s) {
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        k_bias_grad<T><<<dim3((a.out + kTileThreads - 1) / kTileThreads, a.experts),
                         kTileThreads, 0, s>>>(a, (const T*)grad_ys, (T*)grad_bias);
    });
}

}  // namespace gs
