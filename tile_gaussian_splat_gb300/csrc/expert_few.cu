// The experts' products for few rows (a token served, a handful of points):
// each expert's weights are read once for up to eight of its rows, which is
// what bounds them; a 128-row tile of the tensor cores would be empty, and
// float32 weights would first be rewritten.
#include <cstdint>

#include "expert_rows.cuh"
#include "gs_device.cuh"
#include "gs_head_internal.h"
#include "gs_rows8.cuh"
#include "gs_types.cuh"

namespace gs {

namespace {

constexpr int kFewRows = 8;       // rows that share one reading of the weights
constexpr int kFewThreads = 128;  // four warps
constexpr int kFewColumns = 4;    // forward: columns of a warp
constexpr int kFewDepth = 1024;   // forward: terms staged at a time
constexpr int kDxThreads = 512;   // input gradient: sixteen warps share the sum over out
constexpr int kDxDepth = 512;

// The rows of piece `piece` (at most kFewRows of one expert); false beyond the
// last piece.  Every thread of the block calls it.
__device__ __forceinline__ bool few_piece(const LinearArgs& g, int32_t* begin, int piece,
                                          int* expert, int* row0, int* rows, int* kept) {
    int32_t* prefix = begin + g.experts + 1;
    if (threadIdx.x < 32)
        expert_pieces(g.offsets, g.experts, g.rows, kFewRows, begin, prefix,
                      blockIdx.x == 0 && blockIdx.y == 0 ? g.d_status : nullptr);
    __syncthreads();
    *kept = begin[g.experts];
    if (piece >= prefix[g.experts]) return false;
    *expert = expert_of(prefix, g.experts, piece);
    *row0 = begin[*expert] + (piece - prefix[*expert]) * kFewRows;
    *rows = min(kFewRows, begin[*expert + 1] - *row0);
    return true;
}

// Rows of no expert are 0.
template <typename T>
__device__ __forceinline__ void zero_tail(T* out, int64_t kept, int64_t rows, int width) {
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t stride = (int64_t)gridDim.x * gridDim.y * blockDim.x;
    for (int64_t i = kept * width + block * blockDim.x + threadIdx.x; i < rows * width;
         i += stride)
        out[i] = from_f<T>(0.f);
}

// kRows x kFewColumns sums over this lane's terms of the staged rows.
template <typename T, int kVec, int kRows>
__device__ __forceinline__ void few_terms(const float (*x)[kFewDepth], const T* const* w,
                                          int depth, float (*sum)[kFewRows]) {
#pragma unroll 2
    for (int k = (threadIdx.x & 31) * kVec; k < depth; k += 32 * kVec) {
        float v[kFewColumns][kVec];
#pragma unroll
        for (int n = 0; n < kFewColumns; ++n) unpack<T, kVec>(load_raw<T, kVec>(w[n] + k), v[n]);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float a = x[r][k + i];
#pragma unroll
                for (int n = 0; n < kFewColumns; ++n) sum[n][r] = fmaf(a, v[n][i], sum[n][r]);
            }
        }
    }
}

template <typename T, int kVec>
__global__ void __launch_bounds__(kFewThreads)
    k_few_fwd(LinearArgs g, const T* __restrict__ xs, const T* __restrict__ weight,
              const T* __restrict__ bias, T* __restrict__ ys) {
    extern __shared__ int32_t begin[];
    __shared__ __align__(16) float x[kFewRows][kFewDepth];
    int e, row0, rows, kept;
    const bool any = few_piece(g, begin, blockIdx.y, &e, &row0, &rows, &kept);
    zero_tail(ys, kept, g.rows, g.out);
    if (!any) return;
    const int lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * (kFewThreads / 32) + threadIdx.x / 32) * kFewColumns;
    const T* w[kFewColumns];
#pragma unroll
    for (int n = 0; n < kFewColumns; ++n)
        w[n] = weight + ((int64_t)e * g.out + min(n0 + n, g.out - 1)) * g.in;
    float sum[kFewColumns][kFewRows] = {};
    for (int k0 = 0; k0 < g.in; k0 += kFewDepth) {
        const int depth = min(kFewDepth, g.in - k0);
        if (k0 > 0) __syncthreads();
        for (int r = 0; r < rows; ++r)
            for (int k = threadIdx.x; k < depth; k += kFewThreads)
                x[r][k] = to_f(xs[(int64_t)(row0 + r) * g.in + k0 + k]);
        __syncthreads();
        if (rows == 1)
            few_terms<T, kVec, 1>(x, w, depth, sum);
        else if (rows == 2)
            few_terms<T, kVec, 2>(x, w, depth, sum);
        else if (rows <= 4)
            few_terms<T, kVec, 4>(x, w, depth, sum);
        else
            few_terms<T, kVec, 8>(x, w, depth, sum);
#pragma unroll
        for (int n = 0; n < kFewColumns; ++n) w[n] += depth;
    }
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
        if (r >= rows) break;
#pragma unroll
        for (int n = 0; n < kFewColumns; ++n) {
            float v = warp_sum(sum[n][r]);
            if (lane != n || n0 + n >= g.out) continue;
            if (bias) v += to_f(bias[(int64_t)e * g.out + n0 + n]);
            ys[(int64_t)(row0 + r) * g.out + n0 + n] = from_f<T>(v);
        }
    }
}

// The same of 8-bit rows: sixteen elements of a weight row an access, of one
// block of 128, times its power of two (exact).  2 rows, 256 -> 1024: 5.6 us.  The
// rule of few_rows holds here too (calls back to back, 8 experts: 8 rows 1024 ->
// 1024 7.6 us and 9.6 on the tensor cores, 16 rows 256 -> 1024 7.7 and 8.1, 32 rows
// 10.3 and 8.1).
template <int kRows>
__device__ __forceinline__ void few8_terms(const float (*x)[kFewDepth], const uint8_t* const* w,
                                           const uint8_t* const* powers, int depth,
                                           float (*sum)[kFewRows]) {
    for (int k = (threadIdx.x & 31) * 16; k < depth; k += 32 * 16) {
        float v[kFewColumns][16];
#pragma unroll
        for (int n = 0; n < kFewColumns; ++n) {
            const uint4 q = *reinterpret_cast<const uint4*>(w[n] + k);
            const float size = scale_of(powers[n][k / GS_SCALE_BLOCK]);
            unpack8_e4m3(uint2{q.x, q.y}, v[n]);
            unpack8_e4m3(uint2{q.z, q.w}, v[n] + 8);
            // whatever lies behind the last channel
#pragma unroll
            for (int i = 0; i < 16; ++i) v[n][i] = k + i < depth ? v[n][i] * size : 0.f;
            if (powers[n][k / GS_SCALE_BLOCK] > kSafeByte<float>)
#pragma unroll
                for (int i = 0; i < 16; ++i) v[n][i] = cut_to<float>(v[n][i]);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 a = *reinterpret_cast<const float4*>(&x[r][k + i]);
#pragma unroll
                for (int n = 0; n < kFewColumns; ++n) {
                    sum[n][r] = fmaf(a.x, v[n][i], sum[n][r]);
                    sum[n][r] = fmaf(a.y, v[n][i + 1], sum[n][r]);
                    sum[n][r] = fmaf(a.z, v[n][i + 2], sum[n][r]);
                    sum[n][r] = fmaf(a.w, v[n][i + 3], sum[n][r]);
                }
            }
    }
}

template <typename T>
__global__ void __launch_bounds__(kFewThreads)
    k_few8_fwd(LinearArgs g, Rows8 xs, Rows8 weight, const T* __restrict__ bias,
               T* __restrict__ ys) {
    extern __shared__ int32_t begin[];
    __shared__ __align__(16) float x[kFewRows][kFewDepth];
    int e, row0, rows, kept;
    const bool any = few_piece(g, begin, blockIdx.y, &e, &row0, &rows, &kept);
    zero_tail(ys, kept, g.rows, g.out);
    if (!any) return;
    const int lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * (kFewThreads / 32) + threadIdx.x / 32) * kFewColumns;
    const int pitch = GS_ROW8_BYTES(g.in), scale_pitch = GS_ROW8_SCALES(g.in);
    const uint8_t *w[kFewColumns], *powers[kFewColumns];
#pragma unroll
    for (int n = 0; n < kFewColumns; ++n) {
        const int64_t row = (int64_t)e * g.out + min(n0 + n, g.out - 1);
        w[n] = weight.q + row * pitch;
        powers[n] = weight.scales + row * scale_pitch;
    }
    float sum[kFewColumns][kFewRows] = {};
    for (int k0 = 0; k0 < g.in; k0 += kFewDepth) {
        const int depth = min(kFewDepth, g.in - k0), whole = min(kFewDepth, pitch - k0);
        if (k0 > 0) __syncthreads();
        for (int r = 0; r < rows; ++r) {
            const int64_t row = row0 + r;
            for (int k = threadIdx.x * 8; k < whole; k += kFewThreads * 8) {
                float v[8];
                unpack8_e4m3(*reinterpret_cast<const uint2*>(xs.q + row * pitch + k0 + k), v);
                const float size =
                    scale_of(xs.scales[row * scale_pitch + (k0 + k) / GS_SCALE_BLOCK]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[r][k + i] = k + i < depth ? cut_to<float>(v[i] * size) : 0.f;
            }
        }
        __syncthreads();
        if (rows == 1)
            few8_terms<1>(x, w, powers, depth, sum);
        else if (rows == 2)
            few8_terms<2>(x, w, powers, depth, sum);
        else if (rows <= 4)
            few8_terms<4>(x, w, powers, depth, sum);
        else
            few8_terms<8>(x, w, powers, depth, sum);
#pragma unroll
        for (int n = 0; n < kFewColumns; ++n) {
            w[n] += kFewDepth;
            powers[n] += kFewDepth / GS_SCALE_BLOCK;
        }
    }
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
        if (r >= rows) break;
#pragma unroll
        for (int n = 0; n < kFewColumns; ++n) {
            float v = warp_sum(sum[n][r]);
            if (lane != n || n0 + n >= g.out) continue;
            if (bias) v += to_f(bias[(int64_t)e * g.out + n0 + n]);
            ys[(int64_t)(row0 + r) * g.out + n0 + n] = from_f<T>(v);
        }
    }
}

// grad_xs[r, k] = sum over n of grad_ys[r, n] weight[n, k]: a lane takes kVec
// columns, the block's warps every sixteenth n; their sums meet in shared
// memory.
template <typename T, int kVec>
__global__ void __launch_bounds__(kDxThreads)
    k_few_dx(LinearArgs g, const T* __restrict__ gys, const T* __restrict__ weight,
             T* __restrict__ gxs) {
    extern __shared__ int32_t begin[];
    constexpr int kWarps = kDxThreads / 32;
    __shared__ __align__(16) float a[kDxDepth][kFewRows];
    __shared__ float part[kWarps][32 * kVec];
    int e, row0, rows, kept;
    const bool any = few_piece(g, begin, blockIdx.y, &e, &row0, &rows, &kept);
    zero_tail(gxs, kept, g.rows, g.in);
    if (!any) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int k0 = (blockIdx.x * 32 + lane) * kVec;
    const bool in = k0 < g.in;
    float sum[kFewRows][kVec] = {};
    for (int n0 = 0; n0 < g.out; n0 += kDxDepth) {
        const int depth = min(kDxDepth, g.out - n0);
        if (n0 > 0) __syncthreads();
        for (int r = 0; r < kFewRows; ++r)
            for (int n = threadIdx.x; n < depth; n += kDxThreads)
                a[n][r] = r < rows ? to_f(gys[(int64_t)(row0 + r) * g.out + n0 + n]) : 0.f;
        __syncthreads();
        const T* w = weight + ((int64_t)e * g.out + n0) * g.in + k0;
        if (in) {
#pragma unroll 8
            for (int n = warp; n < depth; n += kWarps) {
                float v[kVec];
                unpack<T, kVec>(load_raw<T, kVec>(w + (int64_t)n * g.in), v);
#pragma unroll
                for (int r = 0; r < kFewRows; ++r) {
                    const float f = a[n][r];
#pragma unroll
                    for (int i = 0; i < kVec; ++i) sum[r][i] = fmaf(f, v[i], sum[r][i]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
        if (r >= rows) break;
#pragma unroll
        for (int i = 0; i < kVec; ++i) part[warp][i * 32 + lane] = sum[r][i];
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * kVec; i += kDxThreads) {
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) v += part[q][i];
            const int k = (blockIdx.x * 32 + i % 32) * kVec + i / 32;
            if (k < g.in) gxs[(int64_t)(row0 + r) * g.in + k] = from_f<T>(v);
        }
        __syncthreads();
    }
}

// Pieces of at most kFewRows rows there can be.
unsigned few_pieces(const LinearArgs& a) {
    const int64_t used = a.rows < a.experts ? a.rows : a.experts;
    return (unsigned)(a.rows / kFewRows + used);
}

}  // namespace

// Where the tensor cores take the weights as they lie, up to sixteen rows in
// all (8 experts of 512 x 512 bf16: 3.9 us against 7.2 for 16 rows, both 7.2
// for 64).  Where they would first be rewritten, sixteen an expert on average
// (32 experts of 512 x 512 f32, 512 rows: 29 us and 33; 64 of 1024 x 1024: 119
// and 246 for 512 rows, 212 and 247 for 1024, whose sixteen rows an expert read
// its weights twice).
bool few_rows(const LinearArgs& a, bool as_they_lie) {
    return as_they_lie ? a.rows <= 16 : a.rows <= 16 * (int64_t)a.experts && a.rows <= 1024;
}

void launch_few_fwd(const LinearArgs& a, const void* xs, const void* weight, const void* bias,
                    void* ys, cudaStream_t s) {
    const int columns = kFewColumns * kFewThreads / 32;
    const dim3 grid((a.out + columns - 1) / columns, few_pieces(a));
    const size_t smem = 2 * sizeof(int32_t) * (a.experts + 1);
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int kWhole = 16 / (int)sizeof(T);
        const T *x = static_cast<const T*>(xs), *w = static_cast<const T*>(weight),
                *b = static_cast<const T*>(bias);
        T* y = static_cast<T*>(ys);
        if (a.in % kWhole == 0 && rows_aligned<T>(weight, a.in))
            k_few_fwd<T, kWhole><<<grid, kFewThreads, smem, s>>>(a, x, w, b, y);
        else
            k_few_fwd<T, 1><<<grid, kFewThreads, smem, s>>>(a, x, w, b, y);
    });
}

void launch_few8_fwd(const LinearArgs& a, Rows8 xs, Rows8 weight, const void* bias, void* ys,
                     cudaStream_t s) {
    const int columns = kFewColumns * kFewThreads / 32;
    const dim3 grid((a.out + columns - 1) / columns, few_pieces(a));
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        k_few8_fwd<T><<<grid, kFewThreads, 2 * sizeof(int32_t) * (a.experts + 1), s>>>(
            a, xs, weight, static_cast<const T*>(bias), static_cast<T*>(ys));
    });
}

void launch_few_dx(const LinearArgs& a, const void* grad_ys, const void* weight, void* grad_xs,
                   cudaStream_t s) {
    const size_t smem = 2 * sizeof(int32_t) * (a.experts + 1);
    with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int kWhole = 16 / (int)sizeof(T);
        const T *gy = static_cast<const T*>(grad_ys), *w = static_cast<const T*>(weight);
        T* gx = static_cast<T*>(grad_xs);
        const auto grid = [&](int vec) {
            return dim3((a.in + 32 * vec - 1) / (32 * vec), few_pieces(a));
        };
        if (a.in % kWhole == 0 && rows_aligned<T>(weight, a.in))
            k_few_dx<T, kWhole><<<grid(kWhole), kDxThreads, smem, s>>>(a, gy, w, gx);
        else
            k_few_dx<T, 1><<<grid(1), kDxThreads, smem, s>>>(a, gy, w, gx);
    });
}

}  // namespace gs
