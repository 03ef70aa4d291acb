// The experts' products on the tensor cores (float16 and bfloat16, widths in
// whole 16-byte vectors).
//
// Three products share one kernel, out[m, n] = sum_k A[m, k] B[n, k]:
//   kForward     A = xs (rows x in),   B = weight[e] (out x in)     sum over in
//   kInputGrad   A = grad_ys (rows x out), B = weight[e]^T (in x out) over out
//   kWeightGrad  A = grad_ys^T (out x rows), B = xs^T (in x rows)   over rows
// The operand whose sum index is not contiguous in memory is handed to the
// matrix instruction as it lies (MN-major), so nothing is transposed.
//
// One block per SM walks output tiles of 128 x kWide: a warp copies 64-term
// slices of A and B into a ring of shared-memory stages (tiled bulk copies),
// a second one issues the matrix instructions, eight more move the finished
// accumulators from tensor memory to the output while the next tile is
// computed in the other half of it (with four, the forward of 262144 rows,
// 512 -> 1024, was bound by them: 235 us).
#include <cstdint>
#include <type_traits>

#include <cuda.h>

#include "expert_rows.cuh"
#include "gs_device.cuh"
#include "gs_head_internal.h"
#include "gs_mma.cuh"
#include "gs_types.cuh"

namespace gs {

namespace {

enum Product { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

constexpr int kHigh = 128;        // rows of an output tile
constexpr int kSlice = 64;        // terms of the sum per stage: 128 bytes
constexpr int kOutWarps = 8;      // two for each quarter of the tile's rows
constexpr int kMmaThreads = 32 * (4 + kOutWarps);  // warps: copy, products, 2 idle, output
constexpr int kAccumulators = 2;

struct ProductArgs {
    const int32_t* offsets;
    int64_t rows;
    int experts;
    int high, width, depth;  // extents: high of the weight gradient, depth of the others
    int chunk;               // weight gradient: rows of a partial sum (0: all of an expert's)
    const void* bias;
    void* out;
    int32_t* d_status;
};

template <int kWide>
struct Shape {
    static constexpr int kBytesA = kHigh * kSlice * 2;
    static constexpr int kBytesB = kWide * kSlice * 2;
    static constexpr int kStageBytes = kBytesA + kBytesB;
    static constexpr int kStages = kWide == 256 ? 4 : 6;
    static constexpr int kStaging = kOutWarps * 32 * 64;
    static constexpr int kColumns = kAccumulators * kWide;
};

struct Bars {
    uint64_t full[8], empty[8], acc_full[kAccumulators], acc_empty[kAccumulators], drain;
    uint32_t tmem;
    int abort;
};

template <int kWide>
constexpr size_t smem_bytes(int experts) {
    using S = Shape<kWide>;
    return 1024 + (size_t)S::kStages * S::kStageBytes + S::kStaging + sizeof(Bars) +
           2 * sizeof(int32_t) * (size_t)(experts + 1);
}

// One output tile of the walk.
struct Tile {
    int expert, piece;
    int row0, row1;  // rows of the output (of the sum, for kWeightGrad)
    int m0, n0;      // first row (kWeightGrad only) and column of the tile
    int slices;      // 64-term slices of the sum
};

template <int kProduct, int kWide>
__device__ __forceinline__ int tiles_per_piece(const ProductArgs& g) {
    const int across = (g.width + kWide - 1) / kWide;
    return kProduct == kWeightGrad ? across * ((g.high + kHigh - 1) / kHigh) : across;
}

template <int kProduct, int kWide>
__device__ __forceinline__ Tile tile_at(const ProductArgs& g, const int32_t* begin,
                                        const int32_t* prefix, int64_t t) {
    const int per = tiles_per_piece<kProduct, kWide>(g);
    const int across = (g.width + kWide - 1) / kWide;
    Tile r;
    r.piece = (int)(t / per);
    const int in = (int)(t - (int64_t)r.piece * per);
    r.n0 = in % across * kWide;
    r.m0 = in / across * kHigh;
    r.expert = expert_of(prefix, g.experts, r.piece);
    const int height = kProduct == kWeightGrad ? g.chunk : kHigh;
    const int b = begin[r.expert], e = begin[r.expert + 1];
    if (height == 0) {
        r.row0 = b;
        r.row1 = e;
    } else {
        r.row0 = b + (r.piece - prefix[r.expert]) * height;
        r.row1 = min(e, r.row0 + height);
    }
    const int terms = kProduct == kWeightGrad ? r.row1 - r.row0 : g.depth;
    r.slices = (terms + kSlice - 1) / kSlice;
    return r;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 rows x 64 bytes of output held one row a lane (four 16-byte vectors),
// turned through shared memory so that four lanes write one row's 64
// contiguous bytes.  valid_rows of the rows and valid_vectors of a row's
// vectors are inside the output.
__device__ __forceinline__ void write_block(char* staging, const uint4* v, char* out,
                                            int64_t pitch, int valid_rows, int valid_vectors) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(staging + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) = v[j];
    __syncwarp();
    const int j = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + lane / 4;
        const uint4 x =
            *reinterpret_cast<const uint4*>(staging + r * 64 + ((j ^ (r >> 1 & 3)) << 4));
        if (r < valid_rows && j < valid_vectors)
            *reinterpret_cast<uint4*>(out + r * pitch + j * 16) = x;
    }
    __syncwarp();
}

// Adds the bias of columns [n, n + 8) to eight sums.
template <typename T>
__device__ __forceinline__ void add_bias(float* v, const T* bias) {
    const uint4 b = *reinterpret_cast<const uint4*>(bias);
    const T* p = reinterpret_cast<const T*>(&b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += to_f(p[i]);
}

// T: element type of the operands; Out: of the output (float for partial sums
// of the weight gradient).
template <typename T, typename Out, int kProduct, int kWide>
__global__ void __launch_bounds__(kMmaThreads, 1)
    k_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ ProductArgs g) {
    using S = Shape<kWide>;
    constexpr bool kMnA = kProduct == kWeightGrad;
    constexpr bool kMnB = kProduct != kForward;
    extern __shared__ char smem_raw[];
    char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    char* staging = smem + S::kStages * S::kStageBytes;
    Bars& bars = *reinterpret_cast<Bars*>(staging + S::kStaging);
    int32_t* begin = reinterpret_cast<int32_t*>(&bars + 1);
    int32_t* prefix = begin + g.experts + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

    if (warp == 0 && lane == 0) {
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < kAccumulators; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], kOutWarps);
        }
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
    }
    if (warp == 1) tmem_alloc(&bars.tmem, S::kColumns);
    if (warp == 2)
        expert_pieces(g.offsets, g.experts, g.rows, kProduct == kWeightGrad ? g.chunk : kHigh,
                      begin, prefix, blockIdx.x == 0 ? g.d_status : nullptr);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem;
    volatile int* abort = &bars.abort;
    const int64_t tiles = (int64_t)prefix[g.experts] * tiles_per_piece<kProduct, kWide>(g);

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const Tile c = tile_at<kProduct, kWide>(g, begin, prefix, t);
                for (int k = 0; k < c.slices; ++k, ++it) {
                    const int s = it % S::kStages;
                    if (it >= S::kStages &&
                        !mbar_wait_limited(&bars.empty[s], (it / S::kStages + 1) & 1, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = smem_u32(smem + s * S::kStageBytes);
                    const uint32_t b = a + S::kBytesA;
                    uint64_t* full = &bars.full[s];
                    mbar_expect_tx(full, S::kStageBytes);
                    if (kProduct == kWeightGrad) {
                        for (int i = 0; i < kHigh / 64; ++i)
                            tma_load_2d(a + i * 64 * 128, &map_a, c.m0 + i * 64,
                                        c.row0 + k * kSlice, full);
                        for (int i = 0; i < kWide / 64; ++i)
                            tma_load_2d(b + i * 64 * 128, &map_b, c.n0 + i * 64,
                                        c.row0 + k * kSlice, full);
                    } else {
                        tma_load_2d(a, &map_a, k * kSlice, c.row0, full);
                        if (kProduct == kForward) {
                            tma_load_3d(b, &map_b, k * kSlice, c.n0, c.expert, full);
                        } else {
                            for (int i = 0; i < kWide / 64; ++i)
                                tma_load_3d(b + i * 64 * 128, &map_b, c.n0 + i * 64, k * kSlice,
                                            c.expert, full);
                        }
                    }
                }
            }
            if (!ok)  // let the copies in flight land before the block goes
                for (uint32_t i = it > S::kStages ? it - S::kStages : 0; i < it; ++i) {
                    int none = 0;
                    mbar_wait_limited(&bars.full[i % S::kStages], (i / S::kStages) & 1, &none);
                }
        }
    } else if (warp == 1) {
        constexpr uint32_t word =
            mma_word(kHigh, kWide, std::is_same<T, __nv_bfloat16>::value, kMnA, kMnB);
        uint32_t it = 0, done = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile c = tile_at<kProduct, kWide>(g, begin, prefix, t);
            if (c.slices == 0) continue;
            const int acc = done % kAccumulators;
            if (done >= kAccumulators)
                ok = warp_wait(&bars.acc_empty[acc], (done / kAccumulators + 1) & 1, abort);
            ++done;
            tmem_fence_after();
            for (int k = 0; k < c.slices && ok; ++k, ++it) {
                const int s = it % S::kStages;
                ok = warp_wait(&bars.full[s], (it / S::kStages) & 1, abort);
                if (!ok) break;
                const uint32_t a = smem_u32(smem + s * S::kStageBytes);
                const uint32_t b = a + S::kBytesA;
                if (kProduct == kWeightGrad && c.row0 + (k + 1) * kSlice > c.row1) {
                    // rows of the next expert in the last slice count as 0,
                    // in both operands: they may hold anything
                    const int first = c.row1 - c.row0 - k * kSlice;
                    for (int i = first * 8 + lane; i < kSlice * 8; i += 32)
                        for (int q = 0; q < (kHigh + kWide) / 64; ++q)
                            *reinterpret_cast<uint4*>(smem + s * S::kStageBytes + q * 64 * 128 +
                                                      i * 16) = uint4{0, 0, 0, 0};
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (lane == 0) {
                    tmem_fence_after();
#pragma unroll
                    for (int j = 0; j < kSlice / 16; ++j) {
                        const uint64_t da = kMnA ? smem_operand(a + j * 2048, 64 * 128, 1024)
                                                 : smem_operand(a + j * 32, 16, 1024);
                        const uint64_t db = kMnB ? smem_operand(b + j * 2048, 64 * 128, 1024)
                                                 : smem_operand(b + j * 32, 16, 1024);
                        mma_f16(tmem + acc * kWide, da, db, word, k > 0 || j > 0);
                    }
                    mma_commit(&bars.empty[s]);
                    if (k + 1 == c.slices) mma_commit(&bars.acc_full[acc]);
                }
                __syncwarp();
            }
        }
        // nothing of this block is still writing tensor memory when it is freed
        if (lane == 0) {
            mma_commit(&bars.drain);
            int none = 0;
            mbar_wait_limited(&bars.drain, 0, &none);
        }
    } else if (warp >= 4) {
        const int q = warp & 3;  // tensor-memory lanes [32 q, 32 q + 32)
        constexpr int kSpan = kWide / (kOutWarps / 4);  // columns of this warp
        const int first = (warp - 4) / 4 * kSpan;
        char* mine = staging + (warp - 4) * 32 * 64;
        constexpr int kVec = 16 / sizeof(Out);  // outputs per 16 bytes
        uint32_t done = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile c = tile_at<kProduct, kWide>(g, begin, prefix, t);
            const int acc = done % kAccumulators;
            const uint32_t from =
                tmem + ((uint32_t)(q * 32) << 16) + acc * kWide + first;
            uint32_t u[2][32] = {};
            if (c.slices > 0) {
                ok = warp_wait(&bars.acc_full[acc], (done / kAccumulators) & 1, abort);
                if (!ok) break;
                ++done;
                tmem_fence_after();
                tmem_load32(from, u[0]);
                tmem_wait_loads();
            }
            char* out;
            int rows;
            if (kProduct == kWeightGrad) {
                const int64_t at = std::is_same<T, Out>::value ? c.expert : c.piece;
                out = static_cast<char*>(g.out) +
                      ((at * g.high + c.m0 + q * 32) * g.width + c.n0) * sizeof(Out);
                rows = g.high - c.m0 - q * 32;
            } else {
                out = static_cast<char*>(g.out) +
                      (((int64_t)c.row0 + q * 32) * g.width + c.n0) * sizeof(Out);
                rows = c.row1 - c.row0 - q * 32;
            }
#pragma unroll
            for (int b = 0; b < kSpan / 32; ++b) {
                const int n = first + b * 32;
                // the next 32 columns come in while these go out
                if (c.slices > 0 && b + 1 < kSpan / 32)
                    tmem_load32(from + (b + 1) * 32, u[(b + 1) & 1]);
                const uint32_t* w = u[b & 1];
                const int left = g.width - c.n0 - n;  // columns from here on
                if (left > 0) {
                    if constexpr (std::is_same<Out, float>::value) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint4 v[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[i] = uint4{w[16 * h + 4 * i], w[16 * h + 4 * i + 1],
                                             w[16 * h + 4 * i + 2], w[16 * h + 4 * i + 3]};
                            write_block(mine, v, out + (n + 16 * h) * sizeof(Out),
                                        (int64_t)g.width * sizeof(Out), rows,
                                        (left - 16 * h + kVec - 1) / kVec);
                        }
                    } else {
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float f[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[8 * i + j]);
                            if (kProduct == kForward && g.bias && i * 8 < left)
                                add_bias(f, static_cast<const T*>(g.bias) +
                                                (int64_t)c.expert * g.width + c.n0 + n + i * 8);
                            v[i] = uint4{pack2<Out>(f[0], f[1]), pack2<Out>(f[2], f[3]),
                                         pack2<Out>(f[4], f[5]), pack2<Out>(f[6], f[7])};
                        }
                        write_block(mine, v, out + n * sizeof(Out),
                                    (int64_t)g.width * sizeof(Out), rows,
                                    (left + kVec - 1) / kVec);
                    }
                }
                if (c.slices > 0) {
                    tmem_wait_loads();
                    if (b + 2 == kSpan / 32 || kSpan == 32) {
                        // the accumulator is read: its next product may begin
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars.acc_empty[acc]);
                    }
                }
            }
        }
        if (kProduct != kWeightGrad) {
            // rows of no expert are 0
            const int64_t per = (int64_t)g.width * sizeof(Out) / 16;
            const int64_t first = (int64_t)begin[g.experts] * per, last = g.rows * per;
            for (int64_t i = first + (int64_t)blockIdx.x * (kOutWarps * 32) + threadIdx.x - 128;
                 i < last; i += (int64_t)gridDim.x * (kOutWarps * 32))
                reinterpret_cast<uint4*>(g.out)[i] = uint4{0, 0, 0, 0};
        }
    }
    __syncthreads();
    if (warp == 1) tmem_free(tmem, S::kColumns);
    if (threadIdx.x == 0 && *abort) report(g.d_status, GS_ERR_TIMEOUT);
}

// grad_weight[e] = sum over the expert's pieces of their partial sums.
template <typename T>
__global__ void __launch_bounds__(256)
    k_sum_pieces(ProductArgs g, const float* __restrict__ partial, T* __restrict__ out) {
    extern __shared__ int32_t pieces[];
    int32_t* prefix = pieces + g.experts + 1;
    if (threadIdx.x < 32)
        expert_pieces(g.offsets, g.experts, g.rows, g.chunk, pieces, prefix, nullptr);
    __syncthreads();
    const int e = blockIdx.y;
    const int64_t size = (int64_t)g.high * g.width / 4;
    const float4* p = reinterpret_cast<const float4*>(partial);
    for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < size; i += (int64_t)gridDim.x * 256) {
        float4 sum{0.f, 0.f, 0.f, 0.f};
        for (int q = prefix[e]; q < prefix[e + 1]; ++q) {
            const float4 v = p[q * size + i];
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
        }
        reinterpret_cast<uint2*>(out)[e * size + i] =
            uint2{pack2<T>(sum.x, sum.y), pack2<T>(sum.z, sum.w)};
    }
}

// cuTensorMapEncodeTiled, found through the runtime (the library does not
// link the driver).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A (rows x columns) matrix, or `count` of them one after the other, copied
// in boxes of box_rows x 64 elements (128 bytes, swizzled).
bool make_map(CUtensorMap* map, int dtype, const void* base, int64_t rows, int64_t columns,
              int count, int box_rows) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)columns, (cuuint64_t)rows, (cuuint64_t)count};
    const cuuint64_t strides[2] = {(cuuint64_t)columns * 2, (cuuint64_t)columns * rows * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, unit[3] = {1, 1, 1};
    return encode(map,
                  dtype == GS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  count > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;
    return n;
}

template <typename T, typename Out, int kProduct, int kWide>
int launch(const CUtensorMap& a, const CUtensorMap& b, const ProductArgs& g, int64_t max_tiles,
           cudaStream_t s) {
    const auto kernel = k_product<T, Out, kProduct, kWide>;
    const size_t smem = smem_bytes<kWide>(g.experts);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
        return GS_ERR_CUDA;
    const int64_t sms = sm_count();
    kernel<<<(unsigned)(max_tiles < sms ? max_tiles : sms), kMmaThreads, smem, s>>>(a, b, g);
    return GS_OK;
}

template <typename T, typename Out, int kProduct>
int launch_wide(const CUtensorMap& a, const CUtensorMap& b, const ProductArgs& g, int64_t pieces,
                cudaStream_t s) {
    const int64_t down = kProduct == kWeightGrad ? (g.high + kHigh - 1) / kHigh : 1;
    const auto tiles = [&](int wide) { return pieces * down * ((g.width + wide - 1) / wide); };
    return g.width > 128 ? launch<T, Out, kProduct, 256>(a, b, g, tiles(256), s)
                         : launch<T, Out, kProduct, 128>(a, b, g, tiles(128), s);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t row_tiles(const LinearArgs& a) {
    return (a.rows + kHigh - 1) / kHigh + a.experts;  // at most one part-filled tile an expert
}

// Rows of one partial sum of the weight gradient, 0 for one sum per expert:
// split when the experts' tiles alone would leave SMs idle.
int weight_grad_chunk(const LinearArgs& a) {
    const int64_t wide = a.in > 128 ? 256 : 128;
    const int64_t tiles = (int64_t)a.experts * ((a.out + kHigh - 1) / kHigh) *
                          ((a.in + wide - 1) / wide);
    if (tiles >= 2 * 152 || a.rows < 2048) return 0;
    const int64_t want = (3 * 152 + tiles - 1) / tiles * a.experts;  // pieces of all experts
    const int64_t chunk = (a.rows / want + kSlice) / kSlice * kSlice;
    return (int)(chunk < 512 ? 512 : chunk);
}

int64_t weight_grad_pieces(const LinearArgs& a, int chunk) {
    return chunk ? a.rows / chunk + a.experts : a.experts;
}

}  // namespace

bool mma_usable(const LinearArgs& a, std::initializer_list<const void*> arrays) {
    if (a.dtype == GS_F32 || a.in % 8 || a.out % 8) return false;
    for (const void* p : arrays)
        if (!aligned16(p)) return false;
    return true;
}

int launch_mma_fwd(const LinearArgs& a, const void* xs, const void* weight, const void* bias,
                   void* ys, cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!make_map(&ma, a.dtype, xs, a.rows, a.in, 0, kHigh) ||
        !make_map(&mb, a.dtype, weight, a.out, a.in, a.experts, a.out > 128 ? 256 : 128))
        return GS_ERR_CUDA;
    const ProductArgs g{a.offsets, a.rows, a.experts, 0, a.out, a.in, 0, bias, ys, a.d_status};
    return a.dtype == GS_F16
               ? launch_wide<__half, __half, kForward>(ma, mb, g, row_tiles(a), s)
               : launch_wide<__nv_bfloat16, __nv_bfloat16, kForward>(ma, mb, g, row_tiles(a), s);
}

int launch_mma_dx(const LinearArgs& a, const void* grad_ys, const void* weight, void* grad_xs,
                  cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!make_map(&ma, a.dtype, grad_ys, a.rows, a.out, 0, kHigh) ||
        !make_map(&mb, a.dtype, weight, a.out, a.in, a.experts, kSlice))
        return GS_ERR_CUDA;
    const ProductArgs g{a.offsets, a.rows, a.experts, 0, a.in, a.out, 0, nullptr, grad_xs,
                        a.d_status};
    return a.dtype == GS_F16
               ? launch_wide<__half, __half, kInputGrad>(ma, mb, g, row_tiles(a), s)
               : launch_wide<__nv_bfloat16, __nv_bfloat16, kInputGrad>(ma, mb, g, row_tiles(a),
                                                                       s);
}

size_t mma_dw_workspace(const LinearArgs& a) {
    const int chunk = weight_grad_chunk(a);
    return chunk ? (size_t)weight_grad_pieces(a, chunk) * a.out * a.in * sizeof(float) : 0;
}

int launch_mma_dw(const LinearArgs& a, const void* grad_ys, const void* xs, void* grad_weight,
                  void* workspace, cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!make_map(&ma, a.dtype, grad_ys, a.rows, a.out, 0, kSlice) ||
        !make_map(&mb, a.dtype, xs, a.rows, a.in, 0, kSlice))
        return GS_ERR_CUDA;
    const int chunk = weight_grad_chunk(a);
    const int64_t pieces = weight_grad_pieces(a, chunk);
    const ProductArgs g{a.offsets, a.rows, a.experts, a.out, a.in, 0, chunk, nullptr,
                        chunk ? workspace : grad_weight, a.d_status};
    int rc = GS_OK;
    const auto run = [&](auto t) {
        using T = decltype(t);
        if (!chunk) {
            rc = launch_wide<T, T, kWeightGrad>(ma, mb, g, pieces, s);
            return;
        }
        rc = launch_wide<T, float, kWeightGrad>(ma, mb, g, pieces, s);
        if (rc != GS_OK) return;
        const int64_t vectors = (int64_t)a.out * a.in / 4;
        k_sum_pieces<T><<<dim3((unsigned)((vectors + 255) / 256 < 64 ? (vectors + 255) / 256 : 64),
                               a.experts),
                          256, 2 * sizeof(int32_t) * (a.experts + 1), s>>>(
            g, static_cast<const float*>(workspace), static_cast<T*>(grad_weight));
    };
    if (a.dtype == GS_F16)
        run(__half{});
    else
        run(__nv_bfloat16{});
    return rc;
}

}  // namespace gs
