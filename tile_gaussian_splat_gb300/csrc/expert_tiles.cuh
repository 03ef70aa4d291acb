// What the tensor-core products share: the walk over stages, the columns of a
// tile that are computed, finished results on their way to the output, and the
// host's side of tiled copies and launches.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda.h>

#include "gs_device.cuh"
#include "gs_mma.cuh"
#include "gs_types.cuh"

namespace gs {

constexpr int kHigh = 128;        // rows of an output tile
constexpr int kOutWarps = 8;      // two for each quarter of the tile's rows

// A place in a ring of kCount stages, and how often it has gone round.
template <int kCount>
struct Ring {
    uint32_t stage = 0, turn = 0;
    __device__ __forceinline__ void advance(int count = kCount) {
        if ((int)++stage == count) {
            stage = 0;
            ++turn;
        }
    }
};

// Columns of a tile from n0 on that are computed: those inside the output, in
// the matrix instruction's steps.
template <int kBlocks, int kWide>
__device__ __forceinline__ int tile_columns(int width, int n0) {
    constexpr int kStep = 16 * kBlocks;
    return min(kWide, (width - n0 + kStep - 1) / kStep * kStep);
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

// Eight results of the output's type in 16 (half types) or 32 bytes.
template <typename Out>
__device__ __forceinline__ void pack8(const float* f, uint4* v) {
    if constexpr (sizeof(Out) == 4) {
        v[0] = uint4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3])};
        v[1] = uint4{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                     __float_as_uint(f[7])};
    } else {
        v[0] = uint4{pack2<Out>(f[0], f[1]), pack2<Out>(f[2], f[3]), pack2<Out>(f[4], f[5]),
                     pack2<Out>(f[6], f[7])};
    }
}

// 32 rows x 64 bytes of output from shared memory (write_block's order), a Word an
// access, several on their way at once (one after the other, 64 odd float32
// columns of a tile took 5000 cycles).
template <typename Word>
__device__ __forceinline__ void write_words(const char* staging, char* out, int64_t pitch_bytes,
                                            int valid_rows, int left_bytes) {
    constexpr int kWords = 64 / (int)sizeof(Word), kStep = 32 / kWords;
    const int lane = threadIdx.x & 31;
    const int byte = lane % kWords * (int)sizeof(Word), j = byte / 16;
#pragma unroll 8
    for (int i = 0; i < 32 / kStep; ++i) {
        const int r = i * kStep + lane / kWords;
        const Word x = *reinterpret_cast<const Word*>(
            staging + r * 64 + ((j ^ (r >> 1 & 3)) << 4) + byte % 16);
        if (r < valid_rows && byte < left_bytes)
            *reinterpret_cast<Word*>(out + r * pitch_bytes + byte) = x;
    }
}

// The widest access of up to 16 bytes, and not below an element, for rows of
// `bytes` bytes on end from p on.
inline int access_bytes(const void* p, size_t bytes, int element) {
    int access = 16;
    while (access > element && (reinterpret_cast<uintptr_t>(p) | bytes) % access) access /= 2;
    return access;
}

// 32 rows x 64 bytes of output held one row a lane (four 16-byte vectors),
// turned through shared memory so that neighbouring lanes write a row's 64
// contiguous bytes, `access` bytes each (16 down to an element: 60000 rows of 8-bit
// products, 512 -> 1004, 1002 and 1001 bfloat16, 60, 69 and 83 us, 90 an element
// each).  valid_rows of the rows and `left` of a row's elements are inside the
// output.
template <typename Out>
__device__ __forceinline__ void write_block(char* staging, const uint4* v, Out* out,
                                            int64_t pitch, int valid_rows, int left,
                                            int access) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(staging + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) = v[j];
    __syncwarp();
    char* to = reinterpret_cast<char*>(out);
    const int64_t pitch_bytes = pitch * (int)sizeof(Out);
    const int left_bytes = left * (int)sizeof(Out);
    if (access == 16)
        write_words<uint4>(staging, to, pitch_bytes, valid_rows, left_bytes);
    else if (access == 8)
        write_words<uint2>(staging, to, pitch_bytes, valid_rows, left_bytes);
    else if (access == 4)
        write_words<uint32_t>(staging, to, pitch_bytes, valid_rows, left_bytes);
    else if constexpr (sizeof(Out) == 2)
        write_words<uint16_t>(staging, to, pitch_bytes, valid_rows, left_bytes);
    __syncwarp();
}

// By the output warps: n elements from `out` on are 0; `at` and `stride`: this
// thread's place among all of them.  Whole vectors between the ends.
template <typename Out>
__device__ __forceinline__ void zero_range(Out* out, int64_t n, int64_t at, int64_t stride) {
    constexpr int kVec = 16 / (int)sizeof(Out);
    const int off = (int)(reinterpret_cast<uintptr_t>(out) & 15u) / (int)sizeof(Out);
    const int64_t head = min(n, (int64_t)((kVec - off) % kVec));
    const int64_t whole = (n - head) / kVec, tail = head + whole * kVec;
    for (int64_t i = at; i < whole; i += stride)
        reinterpret_cast<uint4*>(out + head)[i] = uint4{0, 0, 0, 0};
    for (int64_t i = at; i < head; i += stride) out[i] = from_f<Out>(0.f);
    for (int64_t i = tail + at; i < n; i += stride) out[i] = from_f<Out>(0.f);
}

// cuTensorMapEncodeTiled, found through the runtime (the library does not
// link the driver).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
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

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return n;
}

// Launches `kernel` as a walk over at most max_items tiles: as many clusters of
// kBlocks as are resident at once (an SM without a partner in its cluster's
// reach stays free).  raised, resident: the kernel's own.  most_smem: the
// largest dynamic shared memory it is launched with.
template <int kBlocks, typename K, typename... A>
int launch_walk(PerDevice& raised, PerDevice& resident, K kernel, int threads, size_t smem,
                size_t most_smem, int64_t max_items, cudaStream_t s, const A&... args) {
    if (!raised.get(0, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)most_smem) == cudaSuccess;
        }))
        return GS_ERR_CUDA;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(kBlocks);
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = s;
    cudaLaunchAttribute cluster = {};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = kBlocks;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    config.attrs = &cluster;
    config.numAttrs = 1;
    const int clusters = resident.get(152 / kBlocks, [&] {
        int n = 0;
        return cudaOccupancyMaxActiveClusters(&n, kernel, &config) == cudaSuccess ? n : 0;
    });
    config.gridDim = dim3((unsigned)(std::min<int64_t>(max_items, clusters) * kBlocks));
    return cudaLaunchKernelEx(&config, kernel, args...) == cudaSuccess ? GS_OK : GS_ERR_CUDA;
}

}  // namespace gs
