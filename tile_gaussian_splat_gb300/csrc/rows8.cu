// Rows kept in 8 bits: e4m3 with a power of two for each block of 128
// channels, and back.
//
// A block's power is the smallest with which none of its values is beyond
// e4m3's largest, 448 = 1.75 * 2^8.  Powers of two scale without a rounding of
// their own, and the matrix instruction takes them as they are.  Both ways
// each byte is read and written once: bound by memory bandwidth.  kLanes lanes
// of eight elements each share a block (fewer where a row is short), and
// several blocks are loaded before the first is used.
#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "gs_device.cuh"
#include "gs_head_internal.h"
#include "gs_rows8.cuh"
#include "gs_types.cuh"

namespace gs {

namespace {

constexpr int kThreads8 = 128;
constexpr int kEach = 8;       // elements of a lane
constexpr int kBlocksAhead = 4;  // blocks of a lane in flight

struct Pack8 {
    const void* x;
    uint8_t *q, *scales;
    int64_t ldx, rows;
    int channels, blocks, pitch, scale_pitch;
};

// Eight elements from p on of which `left` are inside the row (0 beyond).
template <typename T, bool kVectors>
__device__ __forceinline__ void load8(const T* p, int left, float* v) {
    constexpr int kVec = 16 / (int)sizeof(T);
    if constexpr (kVectors) {
#pragma unroll
        for (int i = 0; i < kEach / kVec; ++i) {
            RawVec<T, kVec> raw{};
            if (i * kVec < left) raw = load_raw<T, kVec>(p + i * kVec);
            unpack<T, kVec>(raw, v + i * kVec);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i) v[i] = i < left ? to_f(p[i]) : 0.f;
    }
}

template <typename T, int kLanes, bool kVectors>
__global__ void __launch_bounds__(kThreads8) k_pack8(Pack8 a) {
    constexpr int kGroups = kThreads8 / kLanes;
    const int at = threadIdx.x % kLanes;
    const int64_t items = a.rows * a.blocks, step = (int64_t)gridDim.x * kGroups;
    for (int64_t i0 = (int64_t)blockIdx.x * kGroups; i0 < items; i0 += step * kBlocksAhead) {
        float v[kBlocksAhead][kEach];
#pragma unroll
        for (int u = 0; u < kBlocksAhead; ++u) {
            const int64_t item = i0 + u * step + threadIdx.x / kLanes;
            const int64_t r = item / a.blocks;
            const int c = (int)(item - r * a.blocks) * GS_SCALE_BLOCK + at * kEach;
            load8<T, kVectors>(static_cast<const T*>(a.x) + r * a.ldx + c,
                               item < items ? a.channels - c : 0, v[u]);
        }
#pragma unroll
        for (int u = 0; u < kBlocksAhead; ++u) {
            const int64_t item = i0 + u * step + threadIdx.x / kLanes;
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                most = fmaxf(most, fabsf(v[u][j]) <= FLT_MAX ? fabsf(v[u][j]) : 0.f);
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1)
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            if (item >= items) continue;
            const int64_t r = item / a.blocks;
            const int block = (int)(item - r * a.blocks), c = block * GS_SCALE_BLOCK + at * kEach;
            const int power = scale_byte(most);
            const float up = two_to(254 - power);
            if (c < a.pitch) {  // 0 behind the last channel
                uint2 q;
                q.x = pack4_e4m3(v[u][0] * up, v[u][1] * up, v[u][2] * up, v[u][3] * up);
                q.y = pack4_e4m3(v[u][4] * up, v[u][5] * up, v[u][6] * up, v[u][7] * up);
                *reinterpret_cast<uint2*>(a.q + r * a.pitch + c) = q;
            }
            if (at == 0) {
                a.scales[r * a.scale_pitch + block] = (uint8_t)power;
                if (block + 1 == a.blocks)
                    for (int b = a.blocks; b < a.scale_pitch; ++b)
                        a.scales[r * a.scale_pitch + b] = 0;
            }
        }
    }
}

struct Unpack8 {
    const uint8_t *q, *scales;
    void* y;
    int64_t ldy, rows;
    int channels, blocks, pitch, scale_pitch;
};

template <typename T, int kLanes, bool kVectors>
__global__ void __launch_bounds__(kThreads8) k_unpack8(Unpack8 a) {
    constexpr int kGroups = kThreads8 / kLanes, kVec = 16 / (int)sizeof(T);
    const int at = threadIdx.x % kLanes;
    const int64_t items = a.rows * a.blocks, step = (int64_t)gridDim.x * kGroups;
    for (int64_t i0 = (int64_t)blockIdx.x * kGroups; i0 < items; i0 += step * kBlocksAhead) {
        uint2 q[kBlocksAhead];
        int power[kBlocksAhead];
#pragma unroll
        for (int u = 0; u < kBlocksAhead; ++u) {
            const int64_t item = i0 + u * step + threadIdx.x / kLanes;
            const int64_t r = item / a.blocks;
            const int block = (int)(item - r * a.blocks), c = block * GS_SCALE_BLOCK + at * kEach;
            const bool in = item < items && c < a.channels;
            q[u] = in ? *reinterpret_cast<const uint2*>(a.q + r * a.pitch + c) : uint2{0, 0};
            power[u] = in ? a.scales[r * a.scale_pitch + block] : 0;
        }
#pragma unroll
        for (int u = 0; u < kBlocksAhead; ++u) {
            const int64_t item = i0 + u * step + threadIdx.x / kLanes;
            const int64_t r = item / a.blocks;
            const int c = (int)(item - r * a.blocks) * GS_SCALE_BLOCK + at * kEach;
            if (item >= items || c >= a.channels) continue;
            float v[kEach];
            unpack8_e4m3(q[u], v);
            const float size = scale_of(power[u]);
#pragma unroll
            for (int j = 0; j < kEach; ++j) v[j] = cut_to<T>(v[j] * size);
            T* y = static_cast<T*>(a.y) + r * a.ldy + c;
            if constexpr (kVectors) {
#pragma unroll
                for (int i = 0; i < kEach / kVec; ++i)
                    if (c + i * kVec < a.channels) store_vec<T, kVec>(y + i * kVec, v + i * kVec);
            } else {
#pragma unroll
                for (int j = 0; j < kEach; ++j)
                    if (c + j < a.channels) y[j] = from_f<T>(v[j]);
            }
        }
    }
}

// f(lanes a block): rows of up to 32 or 64 channels leave no lane idle.
template <typename F>
void with_lanes(int channels, F&& f) {
    if (channels <= 32) return f(std::integral_constant<int, 4>{});
    if (channels <= 64) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}

template <typename K>
int blocks8(PerDevice& resident, K kernel, int64_t items, int lanes) {
    const int groups = kThreads8 / lanes;
    return (int)std::min<int64_t>((items + groups - 1) / groups,
                                  resident_blocks(resident, kernel, 0));
}

}  // namespace

void launch_pack8(const void* x, int64_t ldx, int64_t rows, int channels, int dtype, uint8_t* q,
                  uint8_t* scales, cudaStream_t s) {
    const int blocks = (channels + GS_SCALE_BLOCK - 1) / GS_SCALE_BLOCK;
    const Pack8 a{x, q, scales, ldx, rows, channels, blocks, GS_ROW8_BYTES(channels),
                  GS_ROW8_SCALES(channels)};
    with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        with_lanes(channels, [&](auto lanes) {
            constexpr int kLanes = decltype(lanes)::value;
            const bool vectors = rows_aligned<T>(x, ldx) && channels * sizeof(T) % 16 == 0;
            const int64_t items = rows * blocks;
            if (vectors) {
                const auto kernel = k_pack8<T, kLanes, true>;
                static PerDevice resident;
                kernel<<<blocks8(resident, kernel, items, kLanes), kThreads8, 0, s>>>(a);
            } else {
                const auto kernel = k_pack8<T, kLanes, false>;
                static PerDevice resident;
                kernel<<<blocks8(resident, kernel, items, kLanes), kThreads8, 0, s>>>(a);
            }
        });
    });
}

void launch_unpack8(const uint8_t* q, const uint8_t* scales, int64_t rows, int channels,
                    int dtype, void* y, int64_t ldy, cudaStream_t s) {
    const int blocks = (channels + GS_SCALE_BLOCK - 1) / GS_SCALE_BLOCK;
    const Unpack8 a{q, scales, y, ldy, rows, channels, blocks, GS_ROW8_BYTES(channels),
                    GS_ROW8_SCALES(channels)};
    with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        with_lanes(channels, [&](auto lanes) {
            constexpr int kLanes = decltype(lanes)::value;
            const bool vectors = rows_aligned<T>(y, ldy) && channels * sizeof(T) % 16 == 0;
            const int64_t items = rows * blocks;
            if (vectors) {
                const auto kernel = k_unpack8<T, kLanes, true>;
                static PerDevice resident;
                kernel<<<blocks8(resident, kernel, items, kLanes), kThreads8, 0, s>>>(a);
            } else {
                const auto kernel = k_unpack8<T, kLanes, false>;
                static PerDevice resident;
                kernel<<<blocks8(resident, kernel, items, kLanes), kThreads8, 0, s>>>(a);
            }
        });
    });
}

}  // namespace gs
