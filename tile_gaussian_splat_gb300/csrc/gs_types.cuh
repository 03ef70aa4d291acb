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

inline size_t dtype_size(int dtype) { return dtype == GS_F32 ? 4 : 2; }

}  // namespace gs
