// Rows kept in 8 bits: e4m3 with a power of two for each block of 128
// channels, and back.
//
// A block's power is the smallest with which none of its values is beyond
// e4m3's largest, 448 = 1.75 * 2^8.  Powers of two scale without a rounding of
// their own, and the matrix instruction takes them as they are.  Both ways
// each byte is read and written once: bound by memory bandwidth.  kLanes lanes
// of eight elements each share a block (fewer where a row is short), and
// several blocks are loaded before the first is used.  Where a block lies
// follows from the one before (two 64-bit divisions a block took half of the
// time).  Rows that begin anywhere are read and written as the aligned vectors
// that they lie in, turned by the elements they are off.
// 921600 rows of 128 bfloat16: 54 us there, 56 back by themselves, 6.4 TB/s (96 % of
// a copy's rate; with eight elements a lane 72 and 70, bound by the instructions),
// 58 and 65 among others with all data in memory.  16383 rows of 1021 float16: 17 us
// either way, bound by instructions (element by element 22 and 53).
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
constexpr int kEach = 8;  // elements of an access

// kLanes lanes share a block with kItems accesses each (so that what is done
// once a block is done by few lanes), kAhead blocks of a lane are in flight.
template <int kLanes_, int kItems_, int kAhead_>
struct Share {
    static constexpr int kLanes = kLanes_, kItems = kItems_, kAhead = kAhead_;
};

// The blocks of 128 channels of all rows on end, `step` of them apart.
struct Place {
    int64_t row;
    int block;
    int64_t row_step;
    int block_step, blocks;
    __device__ __forceinline__ Place(int64_t first, int64_t step, int blocks_) : blocks(blocks_) {
        row = first / blocks;
        block = (int)(first - row * blocks);
        row_step = step / blocks;
        block_step = (int)(step - row_step * blocks);
    }
    __device__ __forceinline__ void advance() {
        row += row_step;
        block += block_step;
        if (block >= blocks) {
            block -= blocks;
            ++row;
        }
    }
};

struct Pack8 {
    const void* x;
    uint8_t *q, *scales;
    int64_t ldx, rows;
    int channels, blocks, pitch, scale_pitch;
};

// Eight elements as they lie in memory.
template <typename T>
struct Eight {
    static constexpr int kWords = sizeof(T) * 2;
    uint32_t w[kWords];
};

// Eight elements from p on, of which `left` are inside the row (0 beyond); all
// of [begin, end) may be read.
template <typename T, bool kVectors>
__device__ __forceinline__ Eight<T> load8(const T* p, int left, const T* begin, const T* end) {
    constexpr int kWords = Eight<T>::kWords, kVec = 16 / (int)sizeof(T);
    Eight<T> e{};
    if (left <= 0) return e;
    if constexpr (kVectors) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
            if (i * kVec < left) {
                const uint4 v = *reinterpret_cast<const uint4*>(p + i * kVec);
                e.w[4 * i] = v.x, e.w[4 * i + 1] = v.y, e.w[4 * i + 2] = v.z, e.w[4 * i + 3] = v.w;
            }
        return e;
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const int off = (int)(at & 15u);
    const char* from = reinterpret_cast<const char*>(p) - off;
    if (left < 8 || from < reinterpret_cast<const char*>(begin) ||
        from + 4 * kWords + 16 > reinterpret_cast<const char*>(end)) {
        T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : from_f<T>(0.f);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) e.w[i] = __float_as_uint(to_f(v[i]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                e.w[i] = (uint32_t)*reinterpret_cast<const uint16_t*>(&v[2 * i]) |
                         (uint32_t)*reinterpret_cast<const uint16_t*>(&v[2 * i + 1]) << 16;
        }
        return e;
    }
    uint32_t w[kWords + 4];
#pragma unroll
    for (int i = 0; i < kWords / 4 + 1; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(from + 16 * i);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
    // off = 8 o3 + 4 o2 + 2 o1
#pragma unroll
    for (int i = 0; i < kWords + 2; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < kWords + 1; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < kWords; ++i)
        e.w[i] = sizeof(T) == 2 && (off & 2) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
    return e;
}

template <typename T>
__device__ __forceinline__ void floats8(const Eight<T>& e, float* v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(e.w[i]);
    } else {
        const T* t = reinterpret_cast<const T*>(e.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f(t[i]);
    }
}

// f(how a block is shared): rows of up to 32 or 64 channels leave no lane idle.
template <typename F>
void with_share(int channels, F&& f) {
    if (channels <= 32) return f(Share<4, 1, 4>{});
    if (channels <= 64) return f(Share<8, 1, 4>{});
    return f(Share<8, 2, 2>{});
}

template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <typename T, typename S, bool kVectors>
__global__ void __launch_bounds__(kThreads8) k_pack8(Pack8 a) {
    constexpr int kLanes = S::kLanes, kItems = S::kItems, kGroups = kThreads8 / kLanes;
    const int at = threadIdx.x % kLanes * kEach;
    const T* x = static_cast<const T*>(a.x);
    const T* end = x + (a.rows - 1) * a.ldx + a.channels;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    Place load((int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes, step, a.blocks), p = load;
    // a warp's groups end together: they exchange across all lanes
    const int64_t turns = (a.rows * a.blocks + step - 1) / step;
    for (int64_t t = 0; t < turns; t += S::kAhead) {
        Eight<T> e[S::kAhead][kItems];
#pragma unroll
        for (int u = 0; u < S::kAhead; ++u, load.advance()) {
            const int c = load.block * GS_SCALE_BLOCK + at;
            const T* from = x + load.row * a.ldx + c;
            const int left = load.row < a.rows ? a.channels - c : 0;
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                e[u][i] = load8<T, kVectors>(from + i * kLanes * kEach, left - i * kLanes * kEach,
                                             x, end);
        }
#pragma unroll
        for (int u = 0; u < S::kAhead; ++u, p.advance()) {
            float v[kItems][kEach];
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                floats8(e[u][i], v[i]);
#pragma unroll
                for (int j = 0; j < kEach; ++j) most = fmaxf(most, fabsf(v[i][j]));
            }
            most = lanes_max<kLanes>(most);
            // fmaxf passes over a NaN; an infinity is not counted either
            if (__any_sync(0xffffffffu, most > FLT_MAX)) {
                most = 0.f;
#pragma unroll
                for (int i = 0; i < kItems; ++i)
#pragma unroll
                    for (int j = 0; j < kEach; ++j) {
                        const bool finite = fabsf(v[i][j]) <= FLT_MAX;
                        most = fmaxf(most, finite ? fabsf(v[i][j]) : 0.f);
                        if (!finite) v[i][j] = __uint_as_float(0x7fffffffu);
                    }
                most = lanes_max<kLanes>(most);
            }
            if (p.row >= a.rows) continue;
            const int c = p.block * GS_SCALE_BLOCK + at;
            const int power = scale_byte(most);
            const float up = two_to(254 - power);
            uint8_t* to = a.q + p.row * a.pitch + c;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                if (c + i * kLanes * kEach >= a.pitch) break;  // 0 behind the last channel
                const float* f = v[i];
                *reinterpret_cast<uint2*>(to + i * kLanes * kEach) =
                    uint2{pack4_e4m3(f[0] * up, f[1] * up, f[2] * up, f[3] * up),
                          pack4_e4m3(f[4] * up, f[5] * up, f[6] * up, f[7] * up)};
            }
            if (at == 0) {
                uint8_t* s = a.scales + p.row * a.scale_pitch + p.block;
                // with the zeros behind the last block
                if (p.block + 1 < a.blocks || a.blocks % 4 == 0) {
                    *s = (uint8_t)power;
                } else if (a.blocks % 4 == 1) {
                    *reinterpret_cast<uint32_t*>(s) = (uint32_t)power;
                } else if (a.blocks % 4 == 3) {
                    *reinterpret_cast<uint16_t*>(s) = (uint16_t)power;
                } else {
                    s[0] = (uint8_t)power;
                    *reinterpret_cast<uint16_t*>(s + 1) = 0;
                }
            }
        }
    }
}

struct Unpack8 {
    const uint8_t *q, *scales;
    void* y;
    int64_t ldy, rows;
    int channels, blocks, pitch, scale_pitch;
    const int32_t* used;  // or null: `rows` rows for every expert, those with rows of x
    const int32_t* tops;  // or null: values by lift()'s powers (float16; top_of)
};

// A block's byte once its values are taken as multiples of 2^(top - 134): the
// top's becomes 134, the largest whose values float16 holds.  Values of a byte
// of 64 are 0 in float16, and so are smaller ones; what no expert uses may be
// above the top, and counts for nothing.
__device__ __forceinline__ int lift(int byte, int top) {
    return byte == 255 ? byte : min(max(byte - top + kSafeByte<__half>, 64), kSafeByte<__half>);
}

// Eight values times their scales, as T; kCut: which may be beyond the type.
template <typename T, bool kCut>
__device__ __forceinline__ Eight<T> scaled8(uint2 q, const float* size) {
    float v[8];
    unpack8_e4m3(q, v);
    Eight<T> e;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = kCut ? cut_to<T>(v[j] * size[j]) : v[j] * size[j];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) e.w[j] = __float_as_uint(v[j]);
    } else {
        T* t = reinterpret_cast<T*>(e.w);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = from_f<T>(v[j]);
    }
    return e;
}

template <typename T, typename S>
__global__ void __launch_bounds__(kThreads8) k_unpack8(Unpack8 a) {
    constexpr int kLanes = S::kLanes, kItems = S::kItems, kGroups = kThreads8 / kLanes;
    constexpr int kVec = 16 / (int)sizeof(T);
    const int at = threadIdx.x % kLanes * kEach;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    int top = -1;
    if (std::is_same<T, __half>::value && a.tops) {
        cudaGridDependencySynchronize();  // k_top_bytes may be at work yet
        top = top_of(a.tops);
    }
    if (a.used) {
        // an expert without rows is not looked at; offsets that fall or lie
        // outside are cut where they are used, which leaves no more of them
        if (a.used[blockIdx.y + 1] <= a.used[blockIdx.y]) return;
        a.q += blockIdx.y * a.rows * a.pitch;
        a.scales += blockIdx.y * a.rows * a.scale_pitch;
        a.y = static_cast<T*>(a.y) + blockIdx.y * a.rows * a.ldy;
    }
    Place load((int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes, step, a.blocks), p = load;
    while (p.row < a.rows) {
        uint2 q[S::kAhead][kItems];
        int power[S::kAhead];
#pragma unroll
        for (int u = 0; u < S::kAhead; ++u, load.advance()) {
            const int c = load.block * GS_SCALE_BLOCK + at;
            const uint8_t* from = a.q + load.row * a.pitch + c;
            const bool here = load.row < a.rows;
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                q[u][i] = here && c + i * kLanes * kEach < a.channels
                              ? *reinterpret_cast<const uint2*>(from + i * kLanes * kEach)
                              : uint2{0, 0};
            power[u] = here ? a.scales[load.row * a.scale_pitch + load.block] : 0;
        }
#pragma unroll
        for (int u = 0; u < S::kAhead; ++u, p.advance()) {
            if (p.row >= a.rows) continue;
            const int c = p.block * GS_SCALE_BLOCK + at;
            T* to = static_cast<T*>(a.y) + p.row * a.ldy + c;
            if (top >= 0) power[u] = lift(power[u], top);
            const float one = scale_of(power[u]);
            const float size[8] = {one, one, one, one, one, one, one, one};
            const auto write = [&](auto cut) {
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    const int left = a.channels - c - i * kLanes * kEach;
                    const Eight<T> e = scaled8<T, decltype(cut)::value>(q[u][i], size);
                    uint4* y = reinterpret_cast<uint4*>(to + i * kLanes * kEach);
#pragma unroll
                    for (int k = 0; k < kEach / kVec; ++k)
                        if (k * kVec < left)
                            y[k] = uint4{e.w[4 * k], e.w[4 * k + 1], e.w[4 * k + 2],
                                         e.w[4 * k + 3]};
                }
            };
            if (power[u] > kSafeByte<T>)
                write(std::true_type{});
            else
                write(std::false_type{});
        }
    }
}

// Rows of y that begin anywhere: a thread has the eight elements of one or two
// aligned vectors of a row, of which the first and last may lie across its
// ends.  They take eight bytes of q from two aligned words of eight, and at
// most two blocks' scales.
template <typename T>
__global__ void __launch_bounds__(kThreads8) k_unpack8_any(Unpack8 a, int vectors) {
    Place p((int64_t)blockIdx.x * kThreads8 + threadIdx.x, (int64_t)gridDim.x * kThreads8, vectors);
    for (; p.row < a.rows; p.advance()) {
        T* row = static_cast<T*>(a.y) + p.row * a.ldy;
        // first channel of this thread: at most 0
        const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
        const int c = p.block * kEach - off;
        if (c >= a.channels) continue;
        const uint8_t* q = a.q + p.row * a.pitch;
        const int lo = (c >> 3) * 8, turn = (c - lo) * 8;  // eight bytes from lo on, bits off
        const uint2 w0 = lo >= 0 ? *reinterpret_cast<const uint2*>(q + lo) : uint2{0, 0};
        const uint2 w1 =
            lo + 8 < a.pitch ? *reinterpret_cast<const uint2*>(q + lo + 8) : uint2{0, 0};
        uint32_t w[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
        for (int i = 0; i < 3; ++i) w[i] = turn & 32 ? w[i + 1] : w[i];
        const uint2 v{__funnelshift_r(w[0], w[1], turn & 31), __funnelshift_r(w[1], w[2], turn & 31)};
        const uint8_t* s = a.scales + p.row * a.scale_pitch;
        const int block = max(c, 0) / GS_SCALE_BLOCK;
        const bool both = (block + 1) * GS_SCALE_BLOCK < min(c + kEach, a.channels);
        const int p0 = s[block], p1 = both ? s[block + 1] : p0;
        const float here = scale_of(p0), next = scale_of(p1);
        const int mine = (block + 1) * GS_SCALE_BLOCK - c;  // elements of the first of them
        float size[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) size[j] = j < mine ? here : next;
        const Eight<T> e = max(p0, p1) > kSafeByte<T> ? scaled8<T, true>(v, size)
                                                      : scaled8<T, false>(v, size);
        if (c >= 0 && c + kEach <= a.channels) {
#pragma unroll
            for (int i = 0; i < Eight<T>::kWords / 4; ++i)
                reinterpret_cast<uint4*>(row + c)[i] =
                    uint4{e.w[4 * i], e.w[4 * i + 1], e.w[4 * i + 2], e.w[4 * i + 3]};
        } else {
            const T* t = reinterpret_cast<const T*>(e.w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j >= 0 && c + j < a.channels) row[c + j] = t[j];
        }
    }
}

// The largest byte, 255 apart, of the blocks that the experts' products use: of
// xs' rows and of the weights of experts that have rows (each null: not wanted),
// what every block of threads found in tops (top_of).  A row a thread: a byte for
// 128 elements, small beside what unpacks them, which is launched while this is
// at work.  The gradients of 131072 rows, 512 -> 1024, take 277 us, 272 without it
// (285 with one maximum for all, set to 0 before), those of 20014 rows 259 -> 131
// 71 and 68, those of 921600 rows 128 -> 64 228 and 218 (238 a word at a time).
constexpr int kTopThreads = 256;

__global__ void __launch_bounds__(kTopThreads)
    k_top_bytes(const uint32_t* xs, const uint32_t* weight, const int32_t* offsets, int64_t rows,
                int experts, int out, int blocks, int32_t* tops) {
    __shared__ int begin, kept, found[2];
    cudaTriggerProgrammaticLaunchCompletion();  // k_unpack8 may come up, and wait
    if (threadIdx.x == 0) kept = found[0] = found[1] = 0;
    __syncthreads();
    // the experts' ranges never fall: they end at the largest offset
    for (int e = threadIdx.x; e <= experts; e += kTopThreads) {
        const int at = (int)min(max((int64_t)offsets[e], (int64_t)0), rows);
        if (e == 0) begin = at;
        atomicMax(&kept, at);
    }
    __syncthreads();
    const int words = (blocks + 3) / 4;
    // bytes behind the last block count for nothing
    const uint32_t last = 0xffffffffu >> (words * 4 - blocks) * 8;
    const int64_t first = (int64_t)blockIdx.x * kTopThreads + threadIdx.x;
    constexpr int64_t kStep = (int64_t)kTopParts * kTopThreads;
    // the largest of every byte of the words of rows [r, end) that are used,
    // eight of them on their way at once
    const auto largest = [&](const uint32_t* p, int64_t r, int64_t end, auto used) {
        uint32_t most = 0;
        for (; r < end; r += 8 * kStep)
            for (int w = 0; w < words; ++w) {
                uint32_t v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int64_t row = r + k * kStep;
                    v[k] = row < end && used(row) ? p[row * words + w] : 0;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    v[k] &= w + 1 == words ? last : 0xffffffffu;
                    most = __vmaxu4(most, v[k] & ~__vcmpeq4(v[k], 0xffffffffu));
                }
            }
        most = __vmaxu4(most, most >> 16);
        return __vmaxu4(most, most >> 8) & 255u;
    };
    uint32_t most[2] = {0, 0};
    if (xs) most[0] = largest(xs, begin + first, kept, [](int64_t) { return true; });
    if (weight)
        most[1] = largest(weight, first, (int64_t)experts * out, [&](int64_t row) {
            const int e = (int)((uint32_t)row / (uint32_t)out);
            return offsets[e + 1] > offsets[e];
        });
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, most[i]);
        if ((threadIdx.x & 31) == 0) atomicMax(found + i, (int)top);
    }
    __syncthreads();
    if (threadIdx.x < 2) tops[threadIdx.x * kTopParts + blockIdx.x] = found[threadIdx.x];
}

template <typename K>
int blocks8(PerDevice& resident, K kernel, int64_t items, int lanes) {
    const int groups = kThreads8 / lanes;
    return (int)std::min<int64_t>((items + groups - 1) / groups,
                                  resident_blocks(resident, kernel, 0));
}

static_assert(kThreads8 == kRowThreads, "resident blocks are asked for of these");

}  // namespace

void launch_pack8(const void* x, int64_t ldx, int64_t rows, int channels, int dtype, uint8_t* q,
                  uint8_t* scales, cudaStream_t s) {
    const int blocks = (channels + GS_SCALE_BLOCK - 1) / GS_SCALE_BLOCK;
    const Pack8 a{x, q, scales, ldx, rows, channels, blocks, GS_ROW8_BYTES(channels),
                  GS_ROW8_SCALES(channels)};
    with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        with_share(channels, [&](auto share) {
            using S = decltype(share);
            const int64_t items = rows * blocks;
            if (rows_aligned<T>(x, ldx) && channels * sizeof(T) % 16 == 0) {
                const auto kernel = k_pack8<T, S, true>;
                static PerDevice resident;
                kernel<<<blocks8(resident, kernel, items, S::kLanes), kThreads8, 0, s>>>(a);
            } else {
                const auto kernel = k_pack8<T, S, false>;
                static PerDevice resident;
                kernel<<<blocks8(resident, kernel, items, S::kLanes), kThreads8, 0, s>>>(a);
            }
        });
    });
}

void launch_top_bytes(const LinearArgs& a, const uint8_t* xs, const uint8_t* weight,
                      int32_t* tops, cudaStream_t s) {
    k_top_bytes<<<kTopParts, kTopThreads, 0, s>>>(
        reinterpret_cast<const uint32_t*>(xs), reinterpret_cast<const uint32_t*>(weight),
        a.offsets, a.rows, a.experts, a.out, (a.in + GS_SCALE_BLOCK - 1) / GS_SCALE_BLOCK, tops);
}

void launch_unpack8(const uint8_t* q, const uint8_t* scales, int64_t rows, int channels,
                    int dtype, void* y, int64_t ldy, cudaStream_t s, const int32_t* offsets,
                    int experts, const int32_t* tops) {
    const int blocks = (channels + GS_SCALE_BLOCK - 1) / GS_SCALE_BLOCK;
    const Unpack8 a{q, scales, y, ldy, rows, channels, blocks, GS_ROW8_BYTES(channels),
                    GS_ROW8_SCALES(channels), offsets, tops};
    with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        if (!rows_aligned<T>(y, ldy) || channels * sizeof(T) % 16 != 0) {
            // elements before a row's first in its first vector: at most 16 bytes
            const int vectors = (channels + 16 / (int)sizeof(T) - 1 + kEach - 1) / kEach;
            static PerDevice resident;
            k_unpack8_any<T><<<blocks8(resident, k_unpack8_any<T>, rows * vectors, 1), kThreads8,
                               0, s>>>(a, vectors);
            return;
        }
        with_share(channels, [&](auto share) {
            using S = decltype(share);
            static PerDevice resident;
            const auto kernel = k_unpack8<T, S>;
            const int all = blocks8(resident, kernel, rows * blocks, S::kLanes);
            // which experts have rows is not known here: each has the blocks for
            // its part, at least some where few have any
            const int each = offsets ? std::min(all, std::max(all / experts, 32)) : all;
            const dim3 grid(each, offsets ? experts : 1);
            if (!tops) {
                kernel<<<grid, kThreads8, 0, s>>>(a);
                return;
            }
            cudaLaunchConfig_t config = {};
            config.gridDim = grid;
            config.blockDim = dim3(kThreads8);
            config.stream = s;
            cudaLaunchAttribute early = {};
            early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            early.val.programmaticStreamSerializationAllowed = 1;
            config.attrs = &early;
            config.numAttrs = 1;
            (void)cudaLaunchKernelEx(&config, kernel, a);
        });
    });
}

}  // namespace gs
