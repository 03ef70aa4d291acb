// Every expert's matrix product over its sorted rows, and its gradients.
#include <cstdint>

#include "expert_rows.cuh"
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

// Column sums of the rows of one piece (an expert's next kBiasRows rows):
// 32 lanes take kVec * kItems columns each, eight warps every eighth row.
constexpr int kBiasRows = 512;

template <typename T, int kVec, int kItems>
__global__ void __launch_bounds__(256)
    k_bias_pieces(LinearArgs g, const T* __restrict__ gys, float* __restrict__ partial) {
    extern __shared__ int32_t begin[];  // [experts + 1], then prefix [experts + 1]
    __shared__ float part[8][32 * kVec * kItems];
    int32_t* prefix = begin + g.experts + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (warp == 0)
        expert_pieces(g.offsets, g.experts, g.rows, kBiasRows, begin, prefix, g.d_status);
    __syncthreads();
    const int piece = blockIdx.y;
    if (piece >= prefix[g.experts]) return;
    const int e = expert_of(prefix, g.experts, piece);
    const int r0 = begin[e] + (piece - prefix[e]) * kBiasRows;
    const int r1 = min(begin[e + 1], r0 + kBiasRows);
    const int m0 = blockIdx.x * 32 * kVec * kItems + lane * kVec;
    float sum[kItems][kVec] = {};
#pragma unroll 4
    for (int r = r0 + warp; r < r1; r += 8) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int m = m0 + i * 32 * kVec;
            if (m >= g.out) continue;
            float v[kVec];
            unpack<T, kVec>(load_raw<T, kVec>(gys + (int64_t)r * g.out + m), v);
#pragma unroll
            for (int k = 0; k < kVec; ++k) sum[i][k] += v[k];
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int k = 0; k < kVec; ++k) part[warp][(i * 32 + lane) * kVec + k] = sum[i][k];
    __syncthreads();
    for (int c = threadIdx.x; c < 32 * kVec * kItems; c += 256) {
        const int m = blockIdx.x * 32 * kVec * kItems + c;
        if (m >= g.out) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += part[w][c];
        partial[(int64_t)piece * g.out + m] = v;
    }
}

// grad_bias[e] = the sum of the expert's pieces.
template <typename T>
__global__ void __launch_bounds__(256)
    k_bias_sum(LinearArgs g, const float* __restrict__ partial, T* __restrict__ gb) {
    extern __shared__ int32_t begin[];
    int32_t* prefix = begin + g.experts + 1;
    if (threadIdx.x < 32)
        expert_pieces(g.offsets, g.experts, g.rows, kBiasRows, begin, prefix, nullptr);
    __syncthreads();
    const int e = blockIdx.y, m = blockIdx.x * 256 + threadIdx.x;
    if (m >= g.out) return;
    float sum = 0.f;
#pragma unroll 4
    for (int q = prefix[e]; q < prefix[e + 1]; ++q) sum += partial[(int64_t)q * g.out + m];
    gb[(int64_t)e * g.out + m] = from_f<T>(sum);
}

int64_t bias_pieces(const LinearArgs& a) { return a.rows / kBiasRows + a.experts; }

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

size_t linear_db_workspace(const LinearArgs& a) {
    return (size_t)bias_pieces(a) * a.out * sizeof(float);
}

void launch_linear_db(const LinearArgs& a, const void* grad_ys, void* grad_bias, void* workspace,
                      cudaStream_t s) {
    float* partial = static_cast<float*>(workspace);
    const size_t smem = 2 * sizeof(int32_t) * (a.experts + 1);
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int kWhole = 16 / (int)sizeof(T);
        const T* gys = static_cast<const T*>(grad_ys);
        const auto grid = [&](int columns) {
            return dim3((a.out + columns - 1) / columns, (unsigned)bias_pieces(a));
        };
        if (a.rows > 0) {
            if (a.out % kWhole == 0 && rows_aligned<T>(grad_ys, a.out))
                k_bias_pieces<T, kWhole, 1><<<grid(32 * kWhole), 256, smem, s>>>(a, gys, partial);
            else
                k_bias_pieces<T, 1, 4><<<grid(128), 256, smem, s>>>(a, gys, partial);
        }
        k_bias_sum<T><<<dim3((a.out + 255) / 256, a.experts), 256, smem, s>>>(
            a, partial, static_cast<T*>(grad_bias));
    });
}

}  // namespace gs
