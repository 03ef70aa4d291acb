// Element types of the feature-head calls: conversions to and from float32
// and 16-byte vectors.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/gs_head.h"

namespace gs {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Calls f with a value of the element type of `dtype` (checked by the caller).
template <typename F>
void with_dtype(int dtype, F&& f) {
    if (dtype == GS_F32)
        f(float{});
    else if (dtype == GS_F16)
        f(__half{});
    else
        f(__nv_bfloat16{});
}

// kVec elements at p as float32: one load of 16 (or 8, 4, 2) bytes.
template <int kBytes>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

template <typename T, int kVec>
using RawVec = typename Raw<(int)sizeof(T) * kVec>::type;

template <typename T, int kVec>
__device__ __forceinline__ RawVec<T, kVec> load_raw(const T* p) {
    return *reinterpret_cast<const RawVec<T, kVec>*>(p);
}
template <typename T, int kVec>
__device__ __forceinline__ void unpack(const RawVec<T, kVec>& raw, float* v) {
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = to_f(e[i]);
}
template <typename T, int kVec>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
    RawVec<T, kVec> raw;
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < kVec; ++i) e[i] = from_f<T>(v[i]);
    *reinterpret_cast<RawVec<T, kVec>*>(p) = raw;
}

// Element i of an array of `dtype` (a uniform branch), for arrays read once.
__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
    if (dtype == GS_F32) return static_cast<const float*>(p)[i];
    if (dtype == GS_F16) return to_f(static_cast<const __half*>(p)[i]);
    return to_f(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float v) {
    if (dtype == GS_F32)
        static_cast<float*>(p)[i] = v;
    else if (dtype == GS_F16)
        static_cast<__half*>(p)[i] = from_f<__half>(v);
    else
        static_cast<__nv_bfloat16*>(p)[i] = from_f<__nv_bfloat16>(v);
}

// Sum over aligned groups of kLanes lanes, in every lane of the group.
template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Threads of a block that works on rows, each row by kLanes of them.
constexpr int kRowThreads = 128;

// Sums over the kLanes lanes of a row of each of kCount values, in every lane.
// A row of the whole block exchanges its warps' sums through `scratch` (two
// halves used in turn, so one barrier a call is enough).
struct RowScratch {
    float part[2][kRowThreads / 32][8];
};

template <int kLanes, int kCount>
__device__ __forceinline__ void row_sums(float* v, RowScratch& scratch, int& half) {
    constexpr int kIn = kLanes < 32 ? kLanes : 32;
#pragma unroll
    for (int k = 0; k < kCount; ++k) v[k] = group_sum<kIn>(v[k]);
    if constexpr (kLanes > 32) {
        static_assert(kLanes == kRowThreads && kCount <= 8, "a row is the block's");
        float(*part)[8] = scratch.part[half];
        half ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < kCount; ++k) part[threadIdx.x / 32][k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kCount; ++k) {
            v[k] = 0.f;
#pragma unroll
            for (int w = 0; w < kRowThreads / 32; ++w) v[k] += part[w][k];
        }
    }
}

// How a kernel works on rows: accesses of kVec elements, kLanes lanes a row,
// kItems accesses a lane, kRows rows of a lane in flight.
template <int kVec_, int kLanes_, int kItems_, int kRows_>
struct Form {
    static constexpr int kVec = kVec_, kLanes = kLanes_, kItems = kItems_, kRows = kRows_;
};

// A number found out (or a thing done) once for every device a process uses.
class PerDevice {
    static constexpr int kMaxDevices = 64;
    std::atomic<int> found_[kMaxDevices] = {};

  public:
    // The current device's: what find() gave, `otherwise` while that is 0 (it
    // is asked again by the next call).
    template <typename F>
    int get(int otherwise, F&& find) {
        int dev = -1;
        const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices;
        int v = known ? found_[dev].load(std::memory_order_acquire) : 0;
        if (v == 0) {
            v = find();
            if (known) found_[dev].store(v, std::memory_order_release);
            if (v == 0) (void)cudaGetLastError();  // not an error of the launch that follows
        }
        return v ? v : otherwise;
    }
};

// Blocks of a kernel that are resident at once on the current device: a walk
// over the rows in equal shares needs exactly those (a second, part-filled wave
// costs a whole one).
template <typename K>
int resident_blocks(PerDevice& resident, K kernel, size_t smem) {
    return resident.get(152, [&] {
        int per = 0, dev = 0, sms = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kRowThreads, smem) !=
                cudaSuccess ||
            cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        return std::max(1, per) * sms;
    });
}

// f(integral constant): the elements of type T in the widest access of 16, 8,
// 4 or 2 bytes that divides all the pointers and distances in bytes or-ed
// together in `all`.
template <typename T, typename F>
void with_width(uintptr_t all, F&& f) {
    constexpr int kSize = (int)sizeof(T);
    if (all % 16 == 0) return f(std::integral_constant<int, 16 / kSize>{});
    if (all % 8 == 0) return f(std::integral_constant<int, 8 / kSize>{});
    if (kSize == 2 && all % 4 == 0) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
}

// A row pointer and distance, for with_width.
template <typename T>
uintptr_t row_bits(const void* p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * sizeof(T));
}

// Whether rows at distance ld from p can be read in 16-byte vectors.
template <typename T>
bool rows_aligned(const void* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * sizeof(T) % 16 == 0;
}

inline size_t dtype_size(int dtype) { return dtype == GS_F32 ? 4 : 2; }

}  // namespace gs
