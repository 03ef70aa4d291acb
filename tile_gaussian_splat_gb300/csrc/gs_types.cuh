// Element types of the feature-head calls: conversions to and from float32
// and 16-byte vectors.
#pragma once

#include <cstdint>
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

// Whether rows at distance ld from p can be read in 16-byte vectors.
template <typename T>
bool rows_aligned(const void* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * sizeof(T) % 16 == 0;
}

inline size_t dtype_size(int dtype) { return dtype == GS_F32 ? 4 : 2; }

}  // namespace gs
