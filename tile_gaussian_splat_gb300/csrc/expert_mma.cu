// The experts' products on the tensor cores.
//
// Three products share one kernel, out[m, n] = sum_k A[m, k] B[n, k]:
//   kForward     A = xs (rows x in),   B = weight[e] (out x in)     sum over in
//   kInputGrad   A = grad_ys (rows x out), B = weight[e]^T (in x out) over out
//   kWeightGrad  A = grad_ys^T (out x rows), B = xs^T (in x rows)   over rows
// The operand whose sum index is not contiguous in memory is handed to the
// matrix instruction as it lies (MN-major), so nothing is transposed.
//
// float32 operands are first written as three bfloat16 planes, a = a0 + a1 +
// a2, each the nearest to what is left (exact), and a product is six sums,
// a2 b0 + a0 b2 + a1 b1 + a1 b0 + a0 b1 + a0 b0, small ones first; the terms
// left out are of either sign and at most 2^-24 of |a b|, half a unit of the
// last place (planes cut off left out up to 2^-21, always towards zero).  Half-type operands whose rows are not
// whole 16-byte vectors are copied to rows that are (one plane).
//
// The accumulators cut off where float32 sums round (1.2e-8 of the result per
// 16 terms on random data: 3.8e-6 over 5000), always towards zero, so every few
// slices they are added to a running sum, kept in the other half of tensor
// memory, and start anew.  (Added to the output itself, that traffic took as
// long as the products.)
//
// Two neighbouring blocks work as one on output tiles of 256 x 256 (each
// block holds half of the rows of A and of B, so every byte copied into shared
// memory serves twice the products; a single block on tiles of 128 x 256 was
// bound by those copies: 15 TB/s out of the L2).  Narrow outputs and few rows
// take one block and 128-row tiles.  In every block a warp copies 64-term
// slices into a ring of shared-memory stages (tiled bulk copies, counted on
// the first block's barrier), one warp of the first block issues the matrix
// instructions, and eight warps move finished accumulators from tensor memory
// to the output while the next tile is computed in the other half of it.
// 16 experts, bf16: 262144 rows, 512 -> 1024, 194 us (1420 TFLOP/s) where the
// experts have equal shares and 222 us (1240) where a router spreads them and
// passes follow each other; the stores bind (without them 147 of 195 us).  The
// input gradient of 131072 rows 94 us (1460 TFLOP/s), their weight gradient 126
// us (1090), with the bias gradient 143.
//
// The weight gradient's sums run over an expert's rows, of which there are
// many for few output tiles.  The rows of all experts, end to end, are cut
// into g.groups equal shares; a share's tiles (one per tile of a weight
// matrix) walk it side by side, so the rows are read from memory once.  An
// expert that lies within one share is written at once; one that crosses a
// cut leaves partial sums, added up in the order of the shares afterwards.
// Four helper warps take the bias gradient's column sums from the same stages,
// each of a weight matrix' column tiles those of its part of the slices: the
// copies and the products alone keep shared memory busy, and one tile in two
// taking all of the sums cost 38 us on 95.  One of them also clears the rows
// of the next expert in an expert's last slice.
#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include <cuda.h>

#include "expert_rows.cuh"
#include "expert_tiles.cuh"
#include "gs_device.cuh"
#include "gs_head_internal.h"
#include "gs_mma.cuh"
#include "gs_rows8.cuh"
#include "gs_types.cuh"

namespace gs {

namespace {

enum Product { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

constexpr int kSlice = 64;        // terms of the sum per stage: 128 bytes
// Warps: 0 copies, 1 issues products, 2 and 3 (and two after the output warps)
// help with the weight gradient, from 4 on they write the output.
template <int kProduct>
constexpr int kMmaThreads = 32 * (4 + kOutWarps + (kProduct == kWeightGrad ? 2 : 0));
constexpr int kAccumulators = 2;
// Slices summed in an accumulator before they are added to the running sum:
// of a0 b0 (float32), and of half types over features and over rows.  Over
// 131072 rows in nine shares, 1024 x 512 bfloat16, 0.39 % of the gradients were
// not the nearest to the exact sum without rounds (0.05 % of sums in float32),
// 0.12 % with rounds of 32, 0.064 % of 16 and 0.035 % of 8, in 141, 142, 145
// and 151 us.  Rounds of 16 cost products over 2048 features 16 % (82 -> 96 us),
// of 32 nothing there and 7 to 10 % over 4096; 32768 positive float16 products
// came out 1.9e-4 too small on average without rounds and 1.3e-5 with 32.
constexpr int kRound = 8, kHalfRound = 32, kHalfRowsRound = 16;

struct ProductArgs {
    const int32_t* offsets;
    int64_t rows;
    int experts;
    int high, width, depth;  // extents: high of the weight gradient, depth of the others
    int groups;              // weight gradient: shares of the rows
    int pairs;               // sums over plane pairs: 1, for float32 6 (3 with 8-bit rows)
    int round;               // slices summed before they are added to the running sum
    int rounds;              // some sums take several rounds
    int access;              // bytes at which the output's rows can be written
    const int32_t* tops;     // or null: sums are multiples of 2^(top_of - 134) (float16)
    const void* bias;        // kForward
    void* out;
    void* bias_grad;         // kWeightGrad, or null
    float* partial;          // kWeightGrad: two tiles an item (see Walk)
    float* bias_partial;     // two tile heights an item, then one per expert and tile
    int32_t* d_status;
};

// kBlocks blocks share a tile of kHigh * kBlocks rows and kWide columns.
template <int kBlocks, int kWide>
struct Shape {
    static constexpr int kTileHigh = kHigh * kBlocks;
    static constexpr int kBytesA = kHigh * kSlice * 2;
    static constexpr int kPartB = kWide / kBlocks;  // columns of B a block holds, at most
    static constexpr int kBytesB = kPartB * kSlice * 2;
    static constexpr int kStageBytes = kBytesA + kBytesB;
    static constexpr int kStages = kStageBytes > 32768 ? 4 : 6;
    static constexpr int kStaging = kOutWarps * 32 * 64;
    static constexpr int kSpan = kWide / (kOutWarps / 4);  // columns an output warp writes
    static constexpr int kBias = kOutWarps * kSpan * 4;     // their biases as float32
    static constexpr int kColumns = kAccumulators * kWide;
};

struct Bars {
    // of the first block: a stage's data is there (in all blocks), its rows of
    // another expert are cleared, the accumulators may be overwritten
    uint64_t full[6], cleared, acc_empty[kAccumulators];
    // of each block: the helpers may read a stage, it may be overwritten, the
    // accumulators are finished
    uint64_t landed[6], empty[6], acc_full[kAccumulators], drain;
    uint32_t tmem;
    int abort;
};

template <int kBlocks, int kWide>
constexpr size_t smem_bytes(int experts) {
    using S = Shape<kBlocks, kWide>;
    return 1024 + (size_t)S::kStages * S::kStageBytes + S::kStaging + S::kBias +
           sizeof(Bars) +
           2 * sizeof(int32_t) * (size_t)(experts + 1);
}

// Planes of A and B in sum number `sum` of g.pairs, small terms first (three
// pairs: B has one plane).
__device__ __forceinline__ int plane_a(int pairs, int sum) {
    if (pairs == 3) return 2 - sum;
    return 0x001102 >> 4 * (6 - pairs + sum) & 15;  // 2, 0, 1, 1, 0, 0
}
__device__ __forceinline__ int plane_b(int pairs, int sum) {
    if (pairs == 3) return 0;
    return 0x010120 >> 4 * (6 - pairs + sum) & 15;  // 0, 2, 1, 0, 1, 0
}

// One output tile, or one expert's part of it (kWeightGrad).
struct Tile {
    int expert;
    int row0, row1;  // rows of the output (of the sum, for kWeightGrad)
    int m0, n0;      // first row (kWeightGrad only) and column of the tile
    int count;       // 64-term slices of the sum
    int q0, q1;      // of the slices of all sums over plane pairs, those of one round
    int tile;        // kWeightGrad: which tile of the weight matrix
    bool whole;      // kWeightGrad: all of the expert's rows
    int64_t slot;    // kWeightGrad: where a partial sum goes
};

__device__ __forceinline__ int64_t share_begin(int64_t total, int groups, int group) {
    return total * group / groups;
}

// The tiles of one pair of blocks (or block), in order; every warp of it walks
// the same ones.  kForward, kInputGrad: item = (piece of an expert's rows,
// column tile).  kWeightGrad: item = (share of the rows, tile of the weight
// matrix), its experts one after the other; begin and prefix count slices.
template <int kProduct, int kBlocks, int kWide>
struct Walk {
    using S = Shape<kBlocks, kWide>;
    const ProductArgs& g;
    const int32_t *begin, *prefix;
    int64_t item, items, mine = 0, pos = 0, end = 0;
    int step, across, per;

    __device__ __forceinline__ Walk(const ProductArgs& g_, const int32_t* begin_,
                                    const int32_t* prefix_)
        : g(g_), begin(begin_), prefix(prefix_) {
        item = blockIdx.x / kBlocks;
        step = gridDim.x / kBlocks;
        across = (g.width + kWide - 1) / kWide;
        per = kProduct == kWeightGrad ? across * ((g.high + S::kTileHigh - 1) / S::kTileHigh)
                                      : across;
        items = (int64_t)(kProduct == kWeightGrad ? g.groups : prefix[g.experts]) * per;
    }

    // The slices of the next round of a tile; false after the last.
    __device__ __forceinline__ bool next_round(Tile& c) const {
        const int all = c.count * g.pairs;
        c.q0 = c.q1;
        c.q1 = min(all, max(c.q0, all - c.count) + g.round);
        return c.q0 < all;
    }

    // c: as the call before left it (count and q1 0 before the first).
    __device__ __forceinline__ bool next(Tile& c) {
        if (next_round(c)) return true;
        if constexpr (kProduct == kWeightGrad) {
            const int64_t total = prefix[g.experts];
            while (pos >= end) {
                if (item >= items) return false;
                mine = item;
                item += step;
                pos = share_begin(total, g.groups, (int)(mine / per));
                end = share_begin(total, g.groups, (int)(mine / per) + 1);
            }
            const int in = c.tile = (int)(mine % per);
            c.m0 = in / across * S::kTileHigh;
            c.n0 = in % across * kWide;
            c.expert = expert_of(prefix, g.experts, (int)pos);
            const int first = prefix[c.expert], count = prefix[c.expert + 1] - first;
            const int k0 = (int)pos - first, k1 = (int)min(end - first, (int64_t)count);
            c.row0 = begin[c.expert] + k0 * kSlice;
            c.row1 = min(begin[c.expert + 1], begin[c.expert] + k1 * kSlice);
            c.count = k1 - k0;
            c.whole = c.count == count;
            c.slot = mine * 2 + (k0 > 0 ? 0 : 1);
            pos += c.count;
        } else {
            if (item >= items) return false;
            const int piece = (int)(item / per);
            c.m0 = 0;
            c.n0 = (int)(item - (int64_t)piece * per) * kWide;
            c.expert = expert_of(prefix, g.experts, piece);
            c.row0 = begin[c.expert] + (piece - prefix[c.expert]) * S::kTileHigh;
            c.row1 = min(begin[c.expert + 1], c.row0 + S::kTileHigh);
            c.count = (g.depth + kSlice - 1) / kSlice;
            c.tile = 0;
            c.whole = true;
            c.slot = 0;
            item += step;
        }
        c.q1 = 0;
        return next_round(c);
    }
};

// By a whole warp: what sums are multiples of: planes of 8-bit rows in float16 leave a common
// power of two out.  (Sums are below 2^63: times 2^-126 they are 0 in float16.)
template <typename Out>
__device__ __forceinline__ float unit_of(const ProductArgs& g) {
    if (!std::is_same<Out, __half>::value || !g.tops) return 1.f;
    return two_to(max(top_of(g.tops) - 7, 1));
}

// T: type of the planes; Out: of the output and of bias.
template <typename T, typename Out, int kProduct, int kBlocks, int kWide>
__global__ void __launch_bounds__(kMmaThreads<kProduct>, 1)
    k_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ ProductArgs g) {
    using S = Shape<kBlocks, kWide>;
    constexpr bool kMnA = kProduct == kWeightGrad;
    constexpr bool kMnB = kProduct != kForward;
    extern __shared__ char smem_raw[];
    char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    char* staging = smem + S::kStages * S::kStageBytes;
    Bars& bars = *reinterpret_cast<Bars*>(staging + S::kStaging + S::kBias);
    int32_t* begin = reinterpret_cast<int32_t*>(&bars + 1);
    int32_t* prefix = begin + g.experts + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int rank = kBlocks == 2 ? (int)cluster_rank() : 0;
    // the helpers read the stages too where the bias gradient is asked for
    const bool columns = kProduct == kWeightGrad && g.bias_grad;

    if (warp == 0 && lane == 0) {
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.landed[i], 1);
            mbar_init(&bars.empty[i], kProduct == kWeightGrad ? (columns ? 5 : 2) : 1);
        }
        for (int i = 0; i < kAccumulators; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], kOutWarps * kBlocks);
        }
        mbar_init(&bars.cleared, kBlocks);
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
    }
    if (warp == 1) tmem_alloc<kBlocks>(&bars.tmem, S::kColumns);
    if (warp == 2)
        expert_pieces(g.offsets, g.experts, g.rows,
                      kProduct == kWeightGrad ? kSlice : S::kTileHigh, begin, prefix,
                      blockIdx.x == 0 ? g.d_status : nullptr);
    tmem_fence_before();
    __syncthreads();
    if (kBlocks == 2) cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem, base = smem_u32(smem);
    volatile int* abort = &bars.abort;
    Walk<kProduct, kBlocks, kWide> walk(g, begin, prefix);
    Tile c{};
    // where a running sum takes the second accumulator's place
    const int accumulators = g.rounds ? 1 : kAccumulators;

    if (warp == 0) {
        Ring<S::kStages> at;
        bool ok = true;
        while (ok && walk.next(c)) {
            const int n0 =
                c.n0 + rank * (tile_columns<kBlocks, kWide>(g.width, c.n0) / kBlocks);
            int sum = c.q0 / c.count, k = c.q0 % c.count;
            for (int q = c.q0; q < c.q1; ++q, at.advance()) {
                const int row_a = plane_a(g.pairs, sum) * (int)g.rows + c.row0;
                const int row_b = plane_b(g.pairs, sum) * (int)g.rows + c.row0;
                const int matrix = plane_b(g.pairs, sum) * g.experts + c.expert;
                ok = at.turn == 0 || warp_wait(&bars.empty[at.stage], (at.turn + 1) & 1, abort);
                if (!ok) break;
                const uint32_t a = base + at.stage * S::kStageBytes;
                const uint32_t b = a + S::kBytesA;
                const uint32_t full = kBlocks == 2 ? mbar_at(&bars.full[at.stage], 0)
                                                   : smem_u32(&bars.full[at.stage]);
                if (elect_one()) {
                    if (rank == 0)
                        mbar_expect_tx(&bars.full[at.stage], S::kStageBytes * kBlocks);
                    if (kProduct == kWeightGrad) {
                        const int m0 = c.m0 + rank * kHigh;
#pragma unroll
                        for (int i = 0; i < kHigh / 64; ++i)
                            tma_load_2d<kBlocks>(a + i * 64 * 128, &map_a, m0 + i * 64,
                                                 row_a + k * kSlice, full);
#pragma unroll
                        for (int i = 0; i < S::kPartB / 64; ++i)
                            tma_load_2d<kBlocks>(b + i * 64 * 128, &map_b, n0 + i * 64,
                                                 row_b + k * kSlice, full);
                    } else {
                        tma_load_2d<kBlocks>(a, &map_a, k * kSlice, row_a + rank * kHigh, full);
                        if (kProduct == kForward) {
                            tma_load_3d<kBlocks>(b, &map_b, k * kSlice, n0, matrix, full);
                        } else {
#pragma unroll
                            for (int i = 0; i < S::kPartB / 64; ++i)
                                tma_load_3d<kBlocks>(b + i * 64 * 128, &map_b, n0 + i * 64,
                                                     k * kSlice, matrix, full);
                        }
                    }
                }
                __syncwarp();
                if (++k == c.count) {
                    k = 0;
                    ++sum;
                }
            }
        }
        if (!ok && rank == 0)  // let the copies in flight land before the blocks go
            for (int i = 0; i < S::kStages; ++i) {
                // stages [stage, ...) were last filled one turn ago
                const uint32_t turn = i < (int)at.stage ? at.turn : at.turn - 1;
                int none = 0;
                if (turn != ~0u) mbar_wait_limited(&bars.full[i], turn & 1, &none);
            }
    } else if (warp == 1) {
        constexpr uint32_t word0 =
            mma_word(S::kTileHigh, 0, std::is_same<T, __nv_bfloat16>::value, kMnA, kMnB);
        const uint64_t from_a =
            kMnA ? smem_operand(base, 64 * 128, 1024) : smem_operand(base, 16, 1024);
        const uint64_t from_b = kMnB ? smem_operand(base + S::kBytesA, 64 * 128, 1024)
                                     : smem_operand(base + S::kBytesA, 16, 1024);
        Ring<S::kStages> at;
        Ring<kAccumulators> acc;
        uint32_t cut = 0;
        bool ok = rank == 0;
        while (ok && walk.next(c)) {
            if (acc.turn > 0) ok = warp_wait(&bars.acc_empty[acc.stage], (acc.turn + 1) & 1, abort);
            tmem_fence_after();
            const uint32_t d = tmem + acc.stage * kWide;
            const uint32_t word =
                word0 | (uint32_t)(tile_columns<kBlocks, kWide>(g.width, c.n0) >> 3) << 17;
            int k = kProduct == kWeightGrad ? c.q0 % c.count : 0;
            for (int q = c.q0; q < c.q1 && ok; ++q, at.advance()) {
                ok = warp_wait(&bars.full[at.stage], at.turn & 1, abort);
                if (!ok) break;
                if (kProduct == kWeightGrad) {
                    if (lane < kBlocks) mbar_arrive_at(&bars.landed[at.stage], lane);
                    if (c.row1 - c.row0 < (k + 1) * kSlice) {
                        ok = warp_wait<kBlocks == 2>(&bars.cleared, cut++ & 1, abort);
                        if (!ok) break;
                    }
                    __syncwarp();
                }
                const uint64_t da = from_a + at.stage * (S::kStageBytes >> 4);
                const uint64_t db = from_b + at.stage * (S::kStageBytes >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < kSlice / 16; ++j)
                        mma_f16<kBlocks>(d, da + j * ((kMnA ? 2048 : 32) >> 4),
                                         db + j * ((kMnB ? 2048 : 32) >> 4), word,
                                         q > c.q0 || j > 0);
                    mma_commit<kBlocks>(&bars.empty[at.stage]);
                    if (q + 1 == c.q1) mma_commit<kBlocks>(&bars.acc_full[acc.stage]);
                }
                __syncwarp();
                if (kProduct == kWeightGrad && ++k == c.count) k = 0;
            }
            acc.advance(accumulators);
        }
        // nothing is still writing tensor memory when it is freed
        if (rank == 0) {
            if (elect_one()) mma_commit<kBlocks>(&bars.drain);
            __syncwarp();
            int none = 0;
            mbar_wait_limited(&bars.drain, 0, &none);
        }
    } else if (kProduct == kWeightGrad && (warp == 2 || (columns && (warp == 3 || warp > 11)))) {
        const int helper = warp < 4 ? warp - 2 : warp - 10;  // 32 columns each
        // of eight rows, lanes that read together take rows four apart: their
        // halves of the swizzled 128 bytes differ
        const int row8 = (lane >> 3) | (lane >> 2 & 1) << 2, unit = (helper & 1) * 4 + (lane & 3);
        Ring<S::kStages> at;
        bool ok = true;
        float sum[8] = {};  // of eight columns of A over every eighth row
        while (ok && walk.next(c)) {
            int sums = c.q0 / c.count, k = c.q0 % c.count;
            for (int q = c.q0; q < c.q1; ++q, at.advance()) {
                ok = warp_wait(&bars.landed[at.stage], at.turn & 1, abort);
                if (!ok) break;
                char* a = smem + at.stage * S::kStageBytes;
                const int valid = min(kSlice, c.row1 - c.row0 - k * kSlice);
                if (warp == 2 && valid < kSlice) {
                    // rows of the next expert count as 0, in both operands:
                    // they may hold anything
                    for (int i = valid * 8 + lane; i < kSlice * 8; i += 32)
                        for (int q = 0; q < S::kStageBytes / (64 * 128); ++q)
                            *reinterpret_cast<uint4*>(a + q * 64 * 128 + i * 16) =
                                uint4{0, 0, 0, 0};
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_release_at(&bars.cleared, 0);
                }
                // every plane of A once: where it meets plane 0 of B
                if (columns && plane_b(g.pairs, sums) == 0 &&
                    (c.row0 / kSlice + k) % walk.across == c.n0 / kWide) {
                    const char* p = a + helper / 2 * 64 * 128;
#pragma unroll
                    for (int r = row8; r < kSlice; r += 8) {
                        if (r >= valid) break;
                        float v[8];
                        unpack<T, 8>(*reinterpret_cast<const uint4*>(
                                         p + r * 128 + ((unit ^ (r & 7)) << 4)),
                                     v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum[i] += v[i];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_at(&bars.empty[at.stage], rank);
                if (++k == c.count) {
                    k = 0;
                    ++sums;
                }
            }
            if (ok && columns && c.q1 == c.count * g.pairs) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 4);
                    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 8);
                    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 16);
                }
                const int in = rank * kHigh + helper * 32 + lane * 8;
                const int64_t slot =
                    c.whole ? 2 * walk.items + (int64_t)c.expert * walk.per + c.tile : c.slot;
                float4* p = reinterpret_cast<float4*>(g.bias_partial + slot * S::kTileHigh + in);
                if (lane < 4) {
                    p[0] = float4{sum[0], sum[1], sum[2], sum[3]};
                    p[1] = float4{sum[4], sum[5], sum[6], sum[7]};
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = 0.f;
            }
        }
    } else if (warp >= 4 && warp < 4 + kOutWarps) {
        const int q = warp & 3;  // tensor-memory lanes [32 q, 32 q + 32)
        constexpr int kSpan = S::kSpan;
        // half types over features: the next 32 columns come in while these go
        // out (float32 has six times the products to hide behind, the weight
        // gradient long sums, and no registers to spare)
        constexpr int kAhead = sizeof(Out) == 4 || kProduct == kWeightGrad ? 0 : 1;
        float* bias = reinterpret_cast<float*>(staging + S::kStaging) + (warp - 4) * kSpan;
        const int first = (warp - 4) / 4 * kSpan;
        char* mine = staging + (warp - 4) * 32 * 64;
        const float unit = kProduct == kForward ? 1.f : unit_of<Out>(g);
        Ring<kAccumulators> acc;
        bool ok = true;
        for (; ok && walk.next(c); acc.advance(accumulators)) {
            const uint32_t from =
                tmem + ((uint32_t)(q * 32) << 16) + acc.stage * kWide + first;
            uint32_t u[1 + kAhead][32];
            if (kProduct == kForward && g.bias) {
                const Out* p = static_cast<const Out*>(g.bias) + (int64_t)c.expert * g.width;
#pragma unroll
                for (int i = lane; i < kSpan; i += 32) {
                    const int n = c.n0 + first + i;
                    bias[i] = n < g.width ? to_f(p[n]) : 0.f;
                }
                __syncwarp();
            }
            ok = warp_wait(&bars.acc_full[acc.stage], acc.turn & 1, abort);
            if (!ok) break;
            tmem_fence_after();
            if (kAhead) {
                tmem_load32(from, u[0]);
                tmem_wait_loads();
            }
            const int row = rank * kHigh + q * 32;  // first row in the tile
            const bool partial = kProduct == kWeightGrad && !c.whole;
            float* part = nullptr;
            Out* out = static_cast<Out*>(g.out);
            int rows;
            if (partial) {
                part = g.partial + (c.slot * S::kTileHigh + row) * kWide;
                rows = 32;
            } else if (kProduct == kWeightGrad) {
                out += ((int64_t)c.expert * g.high + c.m0 + row) * g.width + c.n0;
                rows = g.high - c.m0 - row;
            } else {
                out += ((int64_t)c.row0 + row) * g.width + c.n0;
                rows = c.row1 - c.row0 - row;
            }
#pragma unroll
            for (int b = 0; b < kSpan / 32; ++b) {
                const int n = first + b * 32;
                if (b + kAhead < kSpan / 32)
                    tmem_load32(from + (b + kAhead) * 32, u[(b + 1) & kAhead]);
                if (!kAhead) tmem_wait_loads();
                uint32_t* w = u[b & kAhead];
                const bool last = c.q1 == c.count * g.pairs;
                const uint32_t sum = from + kWide + b * 32;
                if (c.q0 > 0) {
                    uint32_t was[32];
                    tmem_load32(sum, was);
                    tmem_wait_loads();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        w[i] = __float_as_uint(__uint_as_float(was[i]) + __uint_as_float(w[i]));
                }
                if (!last) {
                    tmem_store32(sum, w);
                    tmem_wait_stores();
                }
                const int left = g.width - c.n0 - n;  // columns from here on
                if (!last) {
                    // kept in tensor memory
                } else if (partial) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = uint4{w[16 * h + 4 * i], w[16 * h + 4 * i + 1],
                                         w[16 * h + 4 * i + 2], w[16 * h + 4 * i + 3]};
                        write_block<float>(mine, v, part + n + 16 * h, kWide, rows, 16, 16);
                    }
                } else if (left > 0) {
                    constexpr int kRow = 64 / (int)sizeof(Out);  // columns written at a time
#pragma unroll
                    for (int h = 0; h < 32 / kRow; ++h) {
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < kRow / 8; ++i) {
                            float f[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                f[j] = __uint_as_float(w[kRow * h + 8 * i + j]);
                                if constexpr (kProduct != kForward &&
                                              std::is_same<Out, __half>::value)
                                    f[j] *= unit;
                            }
                            if (kProduct == kForward && g.bias) {
                                const float4* p = reinterpret_cast<const float4*>(
                                    bias + b * 32 + kRow * h + 8 * i);
                                const float4 lo = p[0], hi = p[1];
                                f[0] += lo.x, f[1] += lo.y, f[2] += lo.z, f[3] += lo.w;
                                f[4] += hi.x, f[5] += hi.y, f[6] += hi.z, f[7] += hi.w;
                            }
                            pack8<Out>(f, v + i * (int)sizeof(Out) / 2);
                        }
                        write_block<Out>(mine, v, out + n + kRow * h, g.width, rows,
                                         left - kRow * h, g.access);
                    }
                }
                tmem_wait_loads();
                if (b + 1 + kAhead == kSpan / 32) {
                    // the accumulator is read: its next product may begin
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_at(&bars.acc_empty[acc.stage], 0);
                }
            }
        }
        // rows of no expert, and the gradients of experts without rows, are 0
        const int64_t at = (int64_t)blockIdx.x * (kOutWarps * 32) + threadIdx.x - 128;
        const int64_t stride = (int64_t)gridDim.x * (kOutWarps * 32);
        Out* out = static_cast<Out*>(g.out);
        if (kProduct != kWeightGrad) {
            const int64_t kept = begin[g.experts];
            zero_range(out + kept * g.width, (g.rows - kept) * g.width, at, stride);
        } else {
            const int64_t size = (int64_t)g.high * g.width;
            for (int e = 0; e < g.experts; ++e)
                if (prefix[e] == prefix[e + 1])
                    zero_range(out + e * size, size, at, stride);
        }
    }
    __syncthreads();
    if (kBlocks == 2) cluster_sync();  // the other block's arrivals and products are over too
    if (warp == 1) tmem_free<kBlocks>(tmem, S::kColumns);
    if (threadIdx.x == 0 && *abort) report(g.d_status, GS_ERR_TIMEOUT);
}

constexpr int kSlabs = 16;  // blocks that add up a tile of partial sums

// What was left in parts.  For every cut between shares, kSlabs blocks per
// tile: the expert that it (and no cut before it) cuts, grad_weight[e] = its
// partial sums in the order of the shares.  Then for every expert ceil(high /
// 256) blocks: grad_bias[e] = the sums of its column tiles and shares.
template <typename Out, int kBlocks, int kWide>
__global__ void __launch_bounds__(256)
    k_sum_parts(const __grid_constant__ ProductArgs g, int tiles) {
    using S = Shape<kBlocks, kWide>;
    constexpr int kSlab = S::kTileHigh / kSlabs;
    extern __shared__ int32_t begin[];
    int32_t* prefix = begin + g.experts + 1;
    if (threadIdx.x < 32)
        expert_pieces(g.offsets, g.experts, g.rows, kSlice, begin, prefix, nullptr);
    __syncthreads();
    const int64_t total = prefix[g.experts];
    const int across = (g.width + kWide - 1) / kWide;
    const auto share_of = [&](int64_t pos) {
        int s = (int)(pos * g.groups / total);
        while (share_begin(total, g.groups, s) > pos) --s;
        while (share_begin(total, g.groups, s + 1) <= pos) ++s;
        return s;
    };
    // shares without a slice there are only where there are more shares than
    // slices (asked of every share for every sum, two 64-bit divisions each took
    // as long as the sums)
    const bool gaps = total < g.groups;
    const auto empty = [&](int s) {
        return gaps && share_begin(total, g.groups, s) == share_begin(total, g.groups, s + 1);
    };
    // an expert's part in share s, of the shares s0 .. that it lies in
    const auto slot = [&](int s, int s0, int tile) {
        return ((int64_t)s * tiles + tile) * 2 + (s == s0 ? 1 : 0);
    };
    int block = blockIdx.x;
    const float unit = unit_of<Out>(g);
    const int cut_blocks = (g.groups - 1) * tiles * kSlabs;
    if (block < cut_blocks) {
        const int cut = block / (tiles * kSlabs) + 1, tile = block / kSlabs % tiles;
        const int64_t pos = share_begin(total, g.groups, cut);
        if (total == 0 || pos >= total) return;
        const int e = expert_of(prefix, g.experts, (int)pos);
        if (prefix[e] == pos) return;  // between two experts
        const int s0 = share_of(prefix[e]);
        if (cut != s0 + 1) return;  // an earlier cut's blocks do this expert
        const int s1 = share_of((int64_t)prefix[e + 1] - 1);
        const int m0 = tile / across * S::kTileHigh + block % kSlabs * kSlab;
        const int n0 = tile % across * kWide;
        for (int i = threadIdx.x; i < kSlab * kWide / 4; i += 256) {
            const int row = i / (kWide / 4), col = i % (kWide / 4) * 4;
            if (m0 + row >= g.high || n0 + col >= g.width) continue;
            float4 sum{0.f, 0.f, 0.f, 0.f};
            // four shares' parts on their way at once, added in order
            for (int s = s0; s <= s1; s += 4) {
                float4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = float4{0.f, 0.f, 0.f, 0.f};
                    if (s + k <= s1 && !empty(s + k))
                        v[k] = *reinterpret_cast<const float4*>(
                            g.partial + (slot(s + k, s0, tile) * S::kTileHigh +
                                         block % kSlabs * kSlab + row) * kWide + col);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sum.x += v[k].x;
                    sum.y += v[k].y;
                    sum.z += v[k].z;
                    sum.w += v[k].w;
                }
            }
            Out* out = static_cast<Out*>(g.out) + ((int64_t)e * g.high + m0 + row) * g.width +
                       n0 + col;
            const float v[4] = {sum.x * unit, sum.y * unit, sum.z * unit, sum.w * unit};
            if (g.access >= 4 * (int)sizeof(Out)) {
                store_vec<Out, 4>(out, v);
            } else {
                for (int j = 0; j < min(4, g.width - n0 - col); ++j) out[j] = from_f<Out>(v[j]);
            }
        }
        return;
    }
    block -= cut_blocks;
    const int per = (g.high + 255) / 256, e = block / per;
    const int m = block % per * 256 + threadIdx.x;
    if (m >= g.high) return;
    float sum = 0.f;
    if (prefix[e] < prefix[e + 1]) {
        const int s0 = share_of(prefix[e]), s1 = share_of((int64_t)prefix[e + 1] - 1);
        const int row = m % S::kTileHigh, tile0 = m / S::kTileHigh * across;
        for (int s = s0; s <= s1; ++s) {
            if (empty(s)) continue;
            for (int n = tile0; n < tile0 + across; ++n) {
                const int64_t at = s0 == s1 ? 2 * (int64_t)g.groups * tiles + e * tiles + n
                                            : slot(s, s0, n);
                sum += g.bias_partial[at * S::kTileHigh + row];
            }
        }
    }
    static_cast<Out*>(g.bias_grad)[(int64_t)e * g.high + m] = from_f<Out>(sum);
}

// A (rows x columns) matrix as planes of rows of `pitch` elements (a multiple
// of 8): float32 as three of bfloat16, half types copied.  Reads once, writes once.
constexpr int kPlaneThreads = 256;

// a = a0 + a1 + a2, each the nearest bfloat16 to what is left: at most 2^-8,
// then 2^-17 of the power of two below |a|, whose last six bits a2 holds (from
// |a| of 2^-110 on; below, a2 loses what is under 2^-133).
// An infinity is +-1, 0 and itself: a2 meets b0 alone, which is 0 only where b
// is (below 2^-133), so every product but that with 0 is infinite, and one of
// two infinities too, by a2 b0 and a0 b2.  (In a0 it would meet b1 and b2,
// which are 0 for many b.)  A NaN is in a2 as well.
__device__ __forceinline__ void split3(float a, uint16_t* p) {
    const bool finite = fabsf(a) <= FLT_MAX;
    __nv_bfloat16 a0 = __float2bfloat16_rn(finite ? a : copysignf(1.f, a));
    // the largest values would round to infinity: cut off
    if (finite && fabsf(__bfloat162float(a0)) > FLT_MAX) a0 = __float2bfloat16_rz(a);
    const float r1 = finite ? a - __bfloat162float(a0) : 0.f;
    const __nv_bfloat16 a1 = __float2bfloat16_rn(r1);
    const __nv_bfloat16 a2 = __float2bfloat16_rn(finite ? r1 - __bfloat162float(a1) : a);
    p[0] = __bfloat16_as_ushort(a0);
    p[1] = __bfloat16_as_ushort(a1);
    p[2] = __bfloat16_as_ushort(a2);
}

// 2^lanes threads a row, at most 32, of eight elements each (four 2^lanes
// apart where rows are not whole vectors, so that reads are contiguous, took
// 19 us where this takes 15: three planes of 2-byte writes).  With whole vectors
// eight blocks an SM are worth a few spilled registers (242486 x 136 float32:
// 59 us, 65 with six blocks; odd rows 17 us and 14).
template <typename T, typename Plane, bool kVectors>
__global__ void __launch_bounds__(kPlaneThreads, kVectors ? 8 : 6)
    k_planes(const T* __restrict__ x, int64_t rows, int columns, int pitch, int lanes,
             Plane* __restrict__ out) {
    constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1, kEach = 8;
    const int at = threadIdx.x & ((1 << lanes) - 1), height = kPlaneThreads >> lanes;
    const int c0 = (blockIdx.x * 32 + at) * kEach;
    if (c0 >= pitch) return;
    const int64_t plane = rows * pitch;
    for (int64_t r = (int64_t)blockIdx.y * height + (threadIdx.x >> lanes); r < rows;
         r += (int64_t)gridDim.y * height) {
        const T* from = x + r * columns + c0;
        uint16_t* to = reinterpret_cast<uint16_t*>(out) + r * pitch + c0;
        __align__(16) T v[kEach];
        if constexpr (kVectors) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(from)[i];
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                v[i] = c0 + i < columns ? from[i] : from_f<T>(0.f);
        }
        __align__(16) uint16_t p[kPlanes][kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if constexpr (sizeof(T) == 4) {
                uint16_t part[3];
                split3(v[i], part);
#pragma unroll
                for (int k = 0; k < kPlanes; ++k) p[k][i] = part[k];
            } else {
                p[0][i] = *reinterpret_cast<const uint16_t*>(&v[i]);
            }
        }
#pragma unroll
        for (int k = 0; k < kPlanes; ++k)
            *reinterpret_cast<uint4*>(to + k * plane) = *reinterpret_cast<const uint4*>(p[k]);
    }
}

// An operand as the tiled copies read it.
struct Planes {
    const void* base;
    int64_t rows;  // of one plane
    int columns, pitch, count;
};

// Whether rows of `columns` elements from p on can be copied as they lie.
bool copyable(int dtype, const void* p, int columns) {
    return dtype != GS_F32 && columns % 8 == 0 && aligned16(p);
}

size_t plane_bytes(int dtype, int64_t rows, int columns) {
    const size_t bytes = (size_t)(dtype == GS_F32 ? 3 : 1) * rows * ceil_div(columns, 8) * 16;
    return (bytes + 255) / 256 * 256;
}

// The operand itself, or its planes at *workspace (which moves behind them).
Planes prepare(int dtype, const void* x, int64_t rows, int columns, char** workspace,
               cudaStream_t s) {
    if (copyable(dtype, x, columns)) return Planes{x, rows, columns, columns, 1};
    const int pitch = (int)ceil_div(columns, 8) * 8, count = dtype == GS_F32 ? 3 : 1;
    void* out = *workspace;
    *workspace += plane_bytes(dtype, rows, columns);
    // whole vectors of 8 elements, so that the last is whole too
    const bool vectors = aligned16(x) && columns % 8 == 0;
    int lanes = 0;
    while (lanes < 5 && (8 << lanes) < pitch) ++lanes;
    const dim3 grid((unsigned)ceil_div(pitch, 256),
                    (unsigned)std::min<int64_t>(ceil_div(rows, kPlaneThreads >> lanes), 152 * 8));
    with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        using Plane = typename std::conditional<sizeof(T) == 4, __nv_bfloat16, T>::type;
        const T* from = static_cast<const T*>(x);
        Plane* to = static_cast<Plane*>(out);
        if (vectors)
            k_planes<T, Plane, true>
                <<<grid, kPlaneThreads, 0, s>>>(from, rows, columns, pitch, lanes, to);
        else
            k_planes<T, Plane, false>
                <<<grid, kPlaneThreads, 0, s>>>(from, rows, columns, pitch, lanes, to);
    });
    return Planes{out, rows, columns, pitch, count};
}

// A matrix (experts = 0), or one matrix an expert, copied in boxes of
// box_rows x 64 elements (128 bytes, swizzled).
bool make_map(CUtensorMap* map, int dtype, const Planes& p, int experts, int box_rows) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const int64_t all = p.rows * p.count, one = experts ? p.rows / experts : all;
    const cuuint64_t dims[3] = {(cuuint64_t)p.columns, (cuuint64_t)one,
                                (cuuint64_t)(experts * p.count)};
    const cuuint64_t strides[2] = {(cuuint64_t)p.pitch * 2, (cuuint64_t)p.pitch * one * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, unit[3] = {1, 1, 1};
    return encode(map,
                  dtype == GS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  experts > 0 ? 3 : 2, const_cast<void*>(p.base), dims, strides, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, typename Out, int kProduct, int kBlocks, int kWide>
int launch(const CUtensorMap& a, const CUtensorMap& b, const ProductArgs& g, int64_t max_items,
           cudaStream_t s) {
    static PerDevice raised, resident;
    return launch_walk<kBlocks>(raised, resident, k_product<T, Out, kProduct, kBlocks, kWide>,
                                kMmaThreads<kProduct>, smem_bytes<kBlocks, kWide>(g.experts),
                                smem_bytes<kBlocks, kWide>(GS_MAX_EXPERTS), max_items, s, a, b, g);
}

// Two blocks a tile of 256 x 256 where those fill every pair of SMs twice, or
// the product is float32's six; one block a tile of 128 x 256 else.  16
// experts, 512 -> 1024 bf16: 65536 rows 53 us in pairs and 62 single, 16384
// 18.6 and 20.3, 8192 12.1 both, 2048 9.1 and 8.1; float32 59 and 62 for 8192.
bool use_pairs(const LinearArgs& a, int width) {
    const int64_t tiles = (a.rows / 256 + a.experts / 2) * ceil_div(width, 256);
    return width > 128 && (a.dtype == GS_F32 || tiles >= sm_count());
}

// Columns of B in one box of a tiled copy.
int box_b(bool pairs, int width) { return !pairs && width > 128 ? 256 : 128; }

template <typename T, typename Out, int kProduct>
int launch_rows(const CUtensorMap& a, const CUtensorMap& b, const ProductArgs& g, bool pairs,
                cudaStream_t s) {
    // at most one part-filled tile an expert
    const int64_t pieces = g.rows / (pairs ? 256 : 128) + g.experts;
    if (pairs) return launch<T, Out, kProduct, 2, 256>(a, b, g, pieces * ceil_div(g.width, 256), s);
    if (g.width > 128)
        return launch<T, Out, kProduct, 1, 256>(a, b, g, pieces * ceil_div(g.width, 256), s);
    return launch<T, Out, kProduct, 1, 128>(a, b, g, pieces, s);
}

// Sums over plane pairs: the planes of float32 gradients meet one plane of
// 8-bit rows.
int plane_pairs(const LinearArgs& a) { return a.dtype != GS_F32 ? 1 : a.packed ? 3 : 6; }

// How the weight gradient is cut up.
struct GradPlan {
    bool pairs;
    int high, wide;    // of a tile
    int64_t tiles;     // of a weight matrix
    int groups;        // shares of the rows
};

GradPlan grad_plan(const LinearArgs& a) {
    GradPlan p{};
    p.pairs = a.out > 128 && a.in > 128;
    p.high = p.pairs ? 256 : 128;
    p.wide = a.in > 128 ? 256 : 128;
    p.tiles = ceil_div(a.out, p.high) * ceil_div(a.in, p.wide);
    const int64_t units = sm_count() / (p.pairs ? 2 : 1);
    // Shares: more of them occupy more units and fill the last round of them
    // better, but each leaves partial sums (two tiles an item, written and
    // read).  The least time by this estimate of a unit's walk: 0.35 us a
    // slice (of each of a float32 product's sums), 2 us for an expert's
    // part to come out, and the sums at 5 TB/s (where experts are longer than a
    // slice, so that a cut falls inside one).  16 experts of 8192 rows, 1024
    // x 512: 126 us in 9 shares, 150 in 19, 170 in 5.
    const double slices = a.rows / (double)kSlice + 0.5 * a.experts;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>((int64_t)slices, 2 * units));
    double best = 0.0;
    for (int64_t g = 1; g <= most; ++g) {
        const int64_t items = g * p.tiles;
        const double walk = slices / g * 0.35 * plane_pairs(a) +
                            2.0 * (a.experts / (double)g + 1);
        const double inside = std::max(0.0, 1.0 - a.experts / slices);
        const double sums = g > 1 ? 3.0 + inside * 16.0 * items * p.high * p.wide / 5e6 : 0.0;
        const double time = walk * ceil_div(items, units) + sums;
        if (g == 1 || time < best) {
            best = time;
            p.groups = (int)g;
        }
    }
    return p;
}

size_t partial_floats(const GradPlan& p) {
    return p.groups > 1 ? (size_t)(2 * p.groups * p.tiles) * p.high * p.wide : 0;
}

size_t bias_floats(const GradPlan& p, int experts) {
    return (size_t)((2 * p.groups + experts) * p.tiles) * p.high;
}

template <typename T, typename Out, int kBlocks, int kWide>
int launch_weight_grad(const CUtensorMap& a, const CUtensorMap& b, const ProductArgs& g,
                       const GradPlan& p, cudaStream_t s) {
    const int rc =
        launch<T, Out, kWeightGrad, kBlocks, kWide>(a, b, g, (int64_t)p.groups * p.tiles, s);
    const int64_t blocks = (int64_t)(p.groups - 1) * p.tiles * kSlabs +
                           (g.bias_grad ? g.experts * ceil_div(g.high, 256) : 0);
    if (rc == GS_OK && blocks > 0)
        k_sum_parts<Out, kBlocks, kWide>
            <<<(unsigned)blocks, 256, 2 * sizeof(int32_t) * (g.experts + 1), s>>>(g,
                                                                                 (int)p.tiles);
    return rc;
}

template <typename T, typename Out>
int weight_grad_of(const CUtensorMap& a, const CUtensorMap& b, const ProductArgs& g,
                   const GradPlan& p, cudaStream_t s) {
    if (p.pairs) return launch_weight_grad<T, Out, 2, 256>(a, b, g, p, s);
    if (p.wide == 256) return launch_weight_grad<T, Out, 1, 256>(a, b, g, p, s);
    return launch_weight_grad<T, Out, 1, 128>(a, b, g, p, s);
}

// depth: terms of a sum, 0 where the caller says how long a tile's part is.
ProductArgs product_args(const LinearArgs& a, void* out, int width, int depth) {
    ProductArgs g{};
    g.offsets = a.offsets;
    g.rows = a.rows;
    g.experts = a.experts;
    g.width = width;
    g.depth = depth;
    g.pairs = plane_pairs(a);
    g.round = a.dtype == GS_F32 ? kRound : kHalfRound;
    g.rounds = ceil_div(depth, kSlice) > g.round;
    const int size = (int)dtype_size(a.dtype);
    g.access = access_bytes(out, (size_t)width * size, size);
    g.out = out;
    g.d_status = a.d_status;
    return g;
}

// f(type of the planes, type of the output)
template <typename F>
int with_types(int dtype, F&& f) {
    if (dtype == GS_F32) return f(__nv_bfloat16{}, float{});
    if (dtype == GS_F16) return f(__half{}, __half{});
    return f(__nv_bfloat16{}, __nv_bfloat16{});
}

}  // namespace

size_t linear_fwd_workspace(const LinearArgs& a, const void* xs, const void* weight) {
    size_t n = 0;
    if (few_rows(a, copyable(a.dtype, weight, a.in))) return n;
    if (!copyable(a.dtype, xs, a.in)) n += plane_bytes(a.dtype, a.rows, a.in);
    if (!copyable(a.dtype, weight, a.in))
        n += plane_bytes(a.dtype, (int64_t)a.experts * a.out, a.in);
    return n;
}

int launch_linear_fwd(const LinearArgs& a, const void* xs, const void* weight, const void* bias,
                      void* ys, void* workspace, cudaStream_t s) {
    if (few_rows(a, copyable(a.dtype, weight, a.in))) {
        launch_few_fwd(a, xs, weight, bias, ys, s);
        return GS_OK;
    }
    const bool pairs = use_pairs(a, a.out);
    char* ws = static_cast<char*>(workspace);
    const Planes pa = prepare(a.dtype, xs, a.rows, a.in, &ws, s);
    const Planes pb = prepare(a.dtype, weight, (int64_t)a.experts * a.out, a.in, &ws, s);
    CUtensorMap ma, mb;
    if (!make_map(&ma, a.dtype, pa, 0, kHigh) ||
        !make_map(&mb, a.dtype, pb, a.experts, box_b(pairs, a.out)))
        return GS_ERR_CUDA;
    ProductArgs g = product_args(a, ys, a.out, a.in);
    g.bias = bias;
    return with_types(a.dtype, [&](auto t, auto o) {
        return launch_rows<decltype(t), decltype(o), kForward>(ma, mb, g, pairs, s);
    });
}

namespace {

// The input gradient of few rows: only where the weights would be rewritten
// (as they lie, the tensor cores were never slower).
bool few_dx(const LinearArgs& a, const void* weight) {
    return !copyable(a.dtype, weight, a.in) && few_rows(a, false);
}

// The gradients of weight and bias from the rows' planes, of map_dtype.  tops: of x.
int launch_grad_of_weight(const LinearArgs& a, int map_dtype, const Planes& gy, const Planes& x,
                          const int32_t* tops, void* grad_weight, void* grad_bias, float* sums,
                          cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!make_map(&ma, map_dtype, gy, 0, kSlice) || !make_map(&mb, map_dtype, x, 0, kSlice))
        return GS_ERR_CUDA;
    const GradPlan p = grad_plan(a);
    ProductArgs g = product_args(a, grad_weight, a.in, 0);
    g.high = a.out;
    g.groups = p.groups;
    if (a.dtype != GS_F32) g.round = kHalfRowsRound;
    // no part of a sum is longer than a share, nor than all the rows
    g.rounds = std::min(ceil_div(a.rows, kSlice),
                        ceil_div(a.rows / kSlice + a.experts, p.groups)) > g.round;
    g.tops = tops;
    g.bias_grad = grad_bias;
    g.partial = sums;
    g.bias_partial = sums + partial_floats(p);
    return with_types(a.dtype, [&](auto t, auto o) {
        return weight_grad_of<decltype(t), decltype(o)>(ma, mb, g, p, s);
    });
}

size_t grad_sums_bytes(const LinearArgs& a) {
    const GradPlan p = grad_plan(a);
    const size_t n = (partial_floats(p) + bias_floats(p, a.experts)) * sizeof(float);
    return (n + 255) / 256 * 256;
}

}  // namespace

size_t linear_bwd_workspace(const LinearArgs& a, const void* grad_ys, const void* xs,
                            const void* weight) {
    size_t n = grad_sums_bytes(a);
    if (!copyable(a.dtype, grad_ys, a.out)) n += plane_bytes(a.dtype, a.rows, a.out);
    if (!copyable(a.dtype, xs, a.in)) n += plane_bytes(a.dtype, a.rows, a.in);
    if (!copyable(a.dtype, weight, a.in) && !few_dx(a, weight))
        n += plane_bytes(a.dtype, (int64_t)a.experts * a.out, a.in);
    return n;
}

int launch_linear_bwd(const LinearArgs& a, const void* grad_ys, const void* xs,
                      const void* weight, void* grad_xs, void* grad_weight, void* grad_bias,
                      void* workspace, cudaStream_t s) {
    char* ws = static_cast<char*>(workspace);
    float* sums = reinterpret_cast<float*>(ws);
    ws += grad_sums_bytes(a);
    Planes gy{};
    if (grad_weight || !few_dx(a, weight)) gy = prepare(a.dtype, grad_ys, a.rows, a.out, &ws, s);
    CUtensorMap ma, mb;
    if (grad_xs && few_dx(a, weight)) {
        launch_few_dx(a, grad_ys, weight, grad_xs, s);
    } else if (grad_xs) {
        const bool pairs = use_pairs(a, a.in);
        const Planes w = prepare(a.dtype, weight, (int64_t)a.experts * a.out, a.in, &ws, s);
        if (!make_map(&ma, a.dtype, gy, 0, kHigh) || !make_map(&mb, a.dtype, w, a.experts, kSlice))
            return GS_ERR_CUDA;
        const ProductArgs g = product_args(a, grad_xs, a.in, a.out);
        const int rc = with_types(a.dtype, [&](auto t, auto o) {
            return launch_rows<decltype(t), decltype(o), kInputGrad>(ma, mb, g, pairs, s);
        });
        if (rc != GS_OK) return rc;
    }
    if (!grad_weight) return GS_OK;
    const Planes x = prepare(a.dtype, xs, a.rows, a.in, &ws, s);
    return launch_grad_of_weight(a, a.dtype, gy, x, nullptr, grad_weight, grad_bias, sums, s);
}

namespace {

// 8-bit rows as rows of half types: bfloat16 holds the values of bytes 3 to 246
// (4 bits from 2^-133 to 448 * 2^119); above it is cut to its largest, as
// gs_rows_unpack8 does, below what is finer than 2^-133 is rounded.
// float16 takes the elements as multiples of a power of two that all of the rows
// (of the weights) have in common, by which the sums are multiplied: the largest
// byte's lie just within it, those of up to 22 bytes below are exact, and what is
// smaller is off by at most 2^-25 there, 2^-39 of the largest.
constexpr int plane_dtype(int dtype) { return dtype == GS_F16 ? GS_F16 : GS_BF16; }

size_t unpacked_bytes(int64_t rows, int columns) { return plane_bytes(GS_BF16, rows, columns); }

// At the front of the workspace, of float16: what launch_top_bytes leaves.
size_t tops_bytes(int dtype) { return dtype == GS_F16 ? 2 * kTopParts * sizeof(int32_t) : 0; }

// offsets: x are weights, of which only experts that have rows are needed.
Planes unpacked(int dtype, Rows8 x, int64_t rows, int columns, const int32_t* offsets, int experts,
                const int32_t* tops, char** workspace, cudaStream_t s) {
    // the zeros behind the last column too, up to whole vectors: they lie in
    // the same block and row of 16 bytes
    const int pitch = (int)ceil_div(columns, 8) * 8;
    void* out = *workspace;
    *workspace += unpacked_bytes(rows, columns);
    launch_unpack8(x.q, x.scales, offsets ? rows / experts : rows, pitch, dtype, out, pitch, s,
                   offsets, experts, tops);
    return Planes{out, rows, columns, pitch, 1};
}

}  // namespace

size_t linear8_bwd_workspace(const LinearArgs& a, const void* grad_ys) {
    size_t n = tops_bytes(a.dtype) + grad_sums_bytes(a);
    if (!copyable(a.dtype, grad_ys, a.out)) n += plane_bytes(a.dtype, a.rows, a.out);
    return n + unpacked_bytes(a.rows, a.in) + unpacked_bytes((int64_t)a.experts * a.out, a.in);
}

int launch_linear8_bwd(const LinearArgs& a, const void* grad_ys, Rows8 xs, Rows8 weight,
                       void* grad_xs, void* grad_weight, void* grad_bias, void* workspace,
                       cudaStream_t s) {
    const int planes = plane_dtype(a.dtype);
    char* ws = static_cast<char*>(workspace);
    int32_t* tops = a.dtype == GS_F16 ? reinterpret_cast<int32_t*>(ws) : nullptr;
    ws += tops_bytes(a.dtype);
    float* sums = reinterpret_cast<float*>(ws);
    ws += grad_sums_bytes(a);
    const Planes gy = prepare(a.dtype, grad_ys, a.rows, a.out, &ws, s);
    if (tops)
        launch_top_bytes(a, grad_weight ? xs.scales : nullptr, grad_xs ? weight.scales : nullptr,
                         tops, s);
    if (grad_xs) {
        const bool pairs = use_pairs(a, a.in);
        const Planes w = unpacked(planes, weight, (int64_t)a.experts * a.out, a.in, a.offsets,
                                  a.experts, tops ? tops + kTopParts : nullptr, &ws, s);
        CUtensorMap ma, mb;
        if (!make_map(&ma, planes, gy, 0, kHigh) || !make_map(&mb, planes, w, a.experts, kSlice))
            return GS_ERR_CUDA;
        ProductArgs g = product_args(a, grad_xs, a.in, a.out);
        g.tops = tops ? tops + kTopParts : nullptr;
        const int rc = with_types(a.dtype, [&](auto t, auto o) {
            return launch_rows<decltype(t), decltype(o), kInputGrad>(ma, mb, g, pairs, s);
        });
        if (rc != GS_OK) return rc;
    }
    if (!grad_weight) return GS_OK;
    const Planes x = unpacked(planes, xs, a.rows, a.in, nullptr, 0, tops, &ws, s);
    return launch_grad_of_weight(a, planes, gy, x, tops, grad_weight, grad_bias, sums, s);
}

}  // namespace gs
