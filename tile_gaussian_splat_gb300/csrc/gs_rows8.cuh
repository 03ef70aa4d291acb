// The 8-bit rows' elements and scales: e4m3 and powers of two as biased
// exponents (2^(byte - 127), 255 for a NaN).
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/gs_head.h"
#include "gs_head_internal.h"

namespace gs {

// The smallest byte with |v| <= most <= 448 * 2^(byte - 127): 448 is 1.75 * 2^8,
// so the exponent of most less 8, one more above 1.75.
__device__ __forceinline__ int scale_byte(float most) {
    const uint32_t u = __float_as_uint(most);
    const int byte = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(byte, 0);
}

// 2^(byte - 127) for 1 <= byte <= 254.
__device__ __forceinline__ float two_to(int byte) { return __uint_as_float((uint32_t)byte << 23); }

// The same for every byte.
__device__ __forceinline__ float scale_of(int byte) {
    if (byte == 255) return __uint_as_float(0x7fffffffu);
    return byte ? two_to(byte) : __uint_as_float(1u << 22);
}

// Four values rounded to e4m3 (ties to even); at most 448 in size, or NaN.
__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(lo) : "f"(a), "f"(b));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(hi) : "f"(c), "f"(d));
    return (uint32_t)lo | (uint32_t)hi << 16;
}

// Two e4m3 values as float16 (exact).
__device__ __forceinline__ __half2 half2_e4m3(uint16_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    return *reinterpret_cast<const __half2*>(&h);
}

__device__ __forceinline__ void unpack8_e4m3(uint2 q, float* v) {
    const uint32_t word[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(half2_e4m3((uint16_t)(word[i / 2] >> 16 * (i & 1))));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// e4m3 has no infinity, so one that scaling or rounding to T gave came of a
// finite value (65504 in float16 is kept as 65536): the type's largest instead.
template <typename T>
__device__ __forceinline__ float cut_to(float v) {
    constexpr float kMost = sizeof(T) == 4 ? 0x1.fffffep127f
                            : std::is_same<T, __half>::value ? 65504.f : 0x1.fep127f;
    return fabsf(v) > kMost ? copysignf(kMost, v) : v;
}

// The largest byte whose block's values, up to 448 * 2^(byte - 127), T holds.
template <typename T>
constexpr int kSafeByte = std::is_same<T, __half>::value ? 134 : 246;

// By a whole warp: the largest byte of all, from what the blocks of k_top_bytes
// found in their parts.
__device__ __forceinline__ int top_of(const int32_t* parts) {
    int top = 0;
#pragma unroll
    for (int i = 0; i < kTopParts / 32; ++i) top = max(top, parts[i * 32 + (threadIdx.x & 31)]);
    return __reduce_max_sync(0xffffffffu, top);
}

}  // namespace gs
