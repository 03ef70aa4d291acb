// The experts' products of 8-bit rows on the tensor cores:
//   ys[r, n] = sum over blocks b of 128 channels of
//              2^(sx[r, b] + sw[n, b]) * sum over the block of qx[r, k] qw[n, k]
//
// The matrix instruction takes the powers of two itself: for every row of
// either operand a byte in tensor memory, picked out of a word of four by the
// instruction, so a word a row serves 512 channels, and the elements go from
// memory to the tensor cores as they lie, at one byte each.  (Its blocks are
// of 32 channels: four in turn take the same byte.)
//
// In every block a warp copies slices of 128 channels into a ring of
// shared-memory stages (tiled bulk copies), four warps read the rows' words of
// powers and write them to tensor memory (each to its own quarter of the lanes:
// the instruction wants them in all four), one warp of the first block issues
// the matrix instructions, and eight warps move finished accumulators to the
// output while the next tile is computed in the other ones.  The second
// accumulators leave no room for the powers beside 256 columns each, so tiles
// are 192 columns wide.
#include <algorithm>
#include <cstdint>

#include <cuda.h>

#include "expert_rows.cuh"
#include "expert_tiles.cuh"
#include "gs_device.cuh"
#include "gs_head_internal.h"
#include "gs_mma.cuh"
#include "gs_types.cuh"

namespace gs {

namespace {

constexpr int kDeep = 128;          // channels a stage: 128 bytes
constexpr int kGroup = 4;           // stages a word of powers serves
constexpr int kAccumulators = 2;
// Warps: 0 copies, 1 issues products, 2, 3, 12 and 13 write powers (the
// quarters 2, 3, 0 and 1 of the lanes), 4 to 11 write the output.
constexpr int kThreads = 32 * 14;
// Columns of tensor memory: the accumulators, then the powers of kBuffers
// groups, those of A in four columns and those of B, a column for 32 of its
// rows, from the eighth on.
constexpr int kColumns = 512, kPowers = 16, kBuffers = 4, kPowersB = 8;
// Slices summed in an accumulator before they are added to the running sum: as
// many instructions as a round of half types over features.
constexpr int kRound = 32;
static_assert(kRound % kGroup == 0, "a round begins with a word of powers");

struct Product8Args {
    const int32_t* offsets;
    const uint32_t *powers_a, *powers_b;  // a row's words: `words` each
    int64_t rows;
    int experts, width, depth, words;
    int rounds;   // sums take several rounds
    int vectors;  // output rows are whole 16-byte vectors
    const void* bias;
    void* out;
    int32_t* d_status;
};

template <int kBlocks, int kWide>
struct Shape8 {
    static constexpr int kTileHigh = kHigh * kBlocks;
    static constexpr int kBytesA = kHigh * kDeep;
    static constexpr int kPartB = kWide / kBlocks;
    static constexpr int kBytesB = kPartB * kDeep;
    static constexpr int kStageBytes = kBytesA + kBytesB;
    static constexpr int kStages = 6;
    static constexpr int kStaging = kOutWarps * 32 * 64;
    static constexpr int kSpan = kWide / (kOutWarps / 4);  // columns an output warp writes
    static constexpr int kBias = kOutWarps * kSpan * 4;
    static_assert(kStageBytes % 1024 == 0, "swizzled rows begin on 1024 bytes");
    static_assert(kAccumulators * kWide + kBuffers * kPowers <= kColumns, "tensor memory");
    static_assert(kWide / 32 <= kPowers - kPowersB, "powers of B");
};

struct Bars8 {
    // of the first block: a stage's data, a buffer's powers are there (in all
    // blocks), the accumulators may be overwritten
    uint64_t full[6], powers_full[kBuffers], acc_empty[kAccumulators];
    // of each block: a stage, a buffer of powers may be overwritten, the
    // accumulators are finished
    uint64_t empty[6], powers_empty[kBuffers], acc_full[kAccumulators], drain;
    uint32_t tmem;
    int abort;
};

template <int kBlocks, int kWide>
constexpr size_t smem_bytes8(int experts) {
    using S = Shape8<kBlocks, kWide>;
    return 1024 + (size_t)S::kStages * S::kStageBytes + S::kStaging + S::kBias + sizeof(Bars8) +
           2 * sizeof(int32_t) * (size_t)(experts + 1);
}

struct Tile8 {
    int expert;
    int row0, row1;  // rows of the output
    int n0;          // first column
    int q0, q1;      // slices of one round
};

// The tiles of one pair of blocks (or block), in order; every warp of it walks
// the same ones: item = (piece of an expert's rows, column tile).
template <int kBlocks, int kWide>
struct Walk8 {
    using S = Shape8<kBlocks, kWide>;
    const Product8Args& g;
    const int32_t *begin, *prefix;
    int64_t item, items;
    int step, across, count;

    __device__ __forceinline__ Walk8(const Product8Args& g_, const int32_t* begin_,
                                     const int32_t* prefix_)
        : g(g_), begin(begin_), prefix(prefix_) {
        item = blockIdx.x / kBlocks;
        step = gridDim.x / kBlocks;
        across = (g.width + kWide - 1) / kWide;
        count = (g.depth + kDeep - 1) / kDeep;
        items = (int64_t)prefix[g.experts] * across;
    }

    // c: as the call before left it (q1 = count before the first).
    __device__ __forceinline__ bool next(Tile8& c) {
        if (c.q1 == count) {
            if (item >= items) return false;
            const int piece = (int)(item / across);
            c.n0 = (int)(item - (int64_t)piece * across) * kWide;
            c.expert = expert_of(prefix, g.experts, piece);
            c.row0 = begin[c.expert] + (piece - prefix[c.expert]) * S::kTileHigh;
            c.row1 = min(begin[c.expert + 1], c.row0 + S::kTileHigh);
            c.q1 = 0;
            item += step;
        }
        c.q0 = c.q1;
        c.q1 = min(count, c.q0 + kRound);
        return true;
    }
};

template <typename Out, int kBlocks, int kWide>
__global__ void __launch_bounds__(kThreads, 1)
    k_product8(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ Product8Args g) {
    using S = Shape8<kBlocks, kWide>;
    extern __shared__ char smem_raw[];
    char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    char* staging = smem + S::kStages * S::kStageBytes;
    Bars8& bars = *reinterpret_cast<Bars8*>(staging + S::kStaging + S::kBias);
    int32_t* begin = reinterpret_cast<int32_t*>(&bars + 1);
    int32_t* prefix = begin + g.experts + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int rank = kBlocks == 2 ? (int)cluster_rank() : 0;

    if (warp == 0 && lane == 0) {
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(&bars.powers_full[i], 4 * kBlocks);
            mbar_init(&bars.powers_empty[i], 1);
        }
        for (int i = 0; i < kAccumulators; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], kOutWarps * kBlocks);
        }
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
    }
    if (warp == 1) tmem_alloc<kBlocks>(&bars.tmem, kColumns);
    if (warp == 2)
        expert_pieces(g.offsets, g.experts, g.rows, S::kTileHigh, begin, prefix,
                      blockIdx.x == 0 ? g.d_status : nullptr);
    tmem_fence_before();
    __syncthreads();
    if (kBlocks == 2) cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem, base = smem_u32(smem);
    const uint32_t powers = tmem + kAccumulators * kWide;
    volatile int* abort = &bars.abort;
    Walk8<kBlocks, kWide> walk(g, begin, prefix);
    Tile8 c{};
    c.q1 = walk.count;
    // where a running sum takes the second accumulator's place
    const int accumulators = g.rounds ? 1 : kAccumulators;

    if (warp == 0) {
        Ring<S::kStages> at;
        bool ok = true;
        while (ok && walk.next(c)) {
            const int n0 =
                c.n0 + rank * (tile_columns<kBlocks, kWide>(g.width, c.n0) / kBlocks);
            for (int q = c.q0; q < c.q1; ++q, at.advance()) {
                ok = at.turn == 0 || warp_wait(&bars.empty[at.stage], (at.turn + 1) & 1, abort);
                if (!ok) break;
                const uint32_t a = base + at.stage * S::kStageBytes;
                const uint32_t full = kBlocks == 2 ? mbar_at(&bars.full[at.stage], 0)
                                                   : smem_u32(&bars.full[at.stage]);
                if (elect_one()) {
                    if (rank == 0)
                        mbar_expect_tx(&bars.full[at.stage], S::kStageBytes * kBlocks);
                    tma_load_2d<kBlocks>(a, &map_a, q * kDeep, c.row0 + rank * kHigh, full);
                    tma_load_3d<kBlocks>(a + S::kBytesA, &map_b, q * kDeep, n0, c.expert, full);
                }
                __syncwarp();
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
        constexpr uint32_t word0 = mma_word_e4m3(S::kTileHigh);
        const uint64_t from_a = smem_operand(base, 16, 1024);
        const uint64_t from_b = smem_operand(base + S::kBytesA, 16, 1024);
        Ring<S::kStages> at;
        Ring<kAccumulators> acc;
        Ring<kBuffers> buffer;
        bool ok = rank == 0;
        while (ok && walk.next(c)) {
            if (acc.turn > 0) ok = warp_wait(&bars.acc_empty[acc.stage], (acc.turn + 1) & 1, abort);
            tmem_fence_after();
            const uint32_t d = tmem + acc.stage * kWide;
            const uint32_t word =
                word0 | (uint32_t)(tile_columns<kBlocks, kWide>(g.width, c.n0) >> 3) << 17;
            for (int q = c.q0; q < c.q1 && ok; ++q, at.advance()) {
                if (q % kGroup == 0) {
                    ok = warp_wait(&bars.powers_full[buffer.stage], buffer.turn & 1, abort);
                    if (!ok) break;
                    tmem_fence_after();
                }
                ok = warp_wait(&bars.full[at.stage], at.turn & 1, abort);
                if (!ok) break;
                const uint64_t da = from_a + at.stage * (S::kStageBytes >> 4);
                const uint64_t db = from_b + at.stage * (S::kStageBytes >> 4);
                const uint32_t from = powers + buffer.stage * kPowers;
                const uint32_t byte = q % kGroup;
                const bool last = q % kGroup == kGroup - 1 || q + 1 == c.q1;
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < kDeep / 32; ++j)
                        mma_e4m3<kBlocks>(d, da + j * (32 >> 4), db + j * (32 >> 4),
                                          word | byte << 4 | byte << 29, from, from + kPowersB,
                                          q > c.q0 || j > 0);
                    mma_commit<kBlocks>(&bars.empty[at.stage]);
                    if (last) mma_commit<kBlocks>(&bars.powers_empty[buffer.stage]);
                    if (q + 1 == c.q1) mma_commit<kBlocks>(&bars.acc_full[acc.stage]);
                }
                __syncwarp();
                if (last) buffer.advance();
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
    } else if (warp < 4 || warp >= 4 + kOutWarps) {
        const uint32_t mine = powers + ((uint32_t)((warp & 3) * 32) << 16);
        Ring<kBuffers> buffer;
        bool ok = true;
        while (ok && walk.next(c)) {
            const int row = c.row0 + rank * kHigh + lane;
            const uint32_t* a = g.powers_a + (int64_t)row * g.words;
            const uint32_t* b =
                g.powers_b + ((int64_t)c.expert * g.width + c.n0 + lane) * g.words;
            for (int q = c.q0; q < c.q1; q += kGroup, buffer.advance()) {
                uint32_t v[kPowers] = {};
                const int word = q / kGroup;
#pragma unroll
                for (int i = 0; i < kHigh / 32; ++i)
                    if (row + i * 32 < c.row1) v[i] = a[(int64_t)i * 32 * g.words + word];
#pragma unroll
                for (int i = 0; i < kWide / 32; ++i)
                    if (c.n0 + lane + i * 32 < g.width)
                        v[kPowersB + i] = b[(int64_t)i * 32 * g.words + word];
                ok = buffer.turn == 0 ||
                     warp_wait(&bars.powers_empty[buffer.stage], (buffer.turn + 1) & 1, abort);
                if (!ok) break;
                tmem_fence_after();
                tmem_store16(mine + buffer.stage * kPowers, v);
                tmem_wait_stores();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(&bars.powers_full[buffer.stage], 0);
            }
        }
    } else {
        const int q = warp & 3;  // tensor-memory lanes [32 q, 32 q + 32)
        constexpr int kSpan = S::kSpan;
        // the next 32 columns come in while these go out (float32 has no
        // registers to spare)
        constexpr int kAhead = sizeof(Out) == 4 ? 0 : 1;
        float* bias = reinterpret_cast<float*>(staging + S::kStaging) + (warp - 4) * kSpan;
        const int first = (warp - 4) / 4 * kSpan;
        char* mine = staging + (warp - 4) * 32 * 64;
        Ring<kAccumulators> acc;
        bool ok = true;
        for (; ok && walk.next(c); acc.advance(accumulators)) {
            const uint32_t from =
                tmem + ((uint32_t)(q * 32) << 16) + acc.stage * kWide + first;
            uint32_t u[1 + kAhead][32];
            if (g.bias) {
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
            Out* out = static_cast<Out*>(g.out) + ((int64_t)c.row0 + row) * g.width + c.n0;
            const int rows = c.row1 - c.row0 - row;
            const bool last = c.q1 == walk.count;
#pragma unroll
            for (int b = 0; b < kSpan / 32; ++b) {
                const int n = first + b * 32;
                if (b + kAhead < kSpan / 32)
                    tmem_load32(from + (b + kAhead) * 32, u[(b + 1) & kAhead]);
                if (!kAhead) tmem_wait_loads();
                uint32_t* w = u[b & kAhead];
                const uint32_t sum = from + kWide + b * 32;
                if (c.q0 > 0) {
                    uint32_t was[32];
                    tmem_load32(sum, was);
                    tmem_wait_loads();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        w[i] = __float_as_uint(__uint_as_float(was[i]) + __uint_as_float(w[i]));
                }
                const int left = g.width - c.n0 - n;  // columns from here on
                if (!last) {
                    tmem_store32(sum, w);
                    tmem_wait_stores();
                } else if (left > 0) {
                    constexpr int kRow = 64 / (int)sizeof(Out);  // columns written at a time
#pragma unroll
                    for (int h = 0; h < 32 / kRow; ++h) {
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < kRow / 8; ++i) {
                            float f[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                f[j] = __uint_as_float(w[kRow * h + 8 * i + j]);
                            if (g.bias) {
                                const float4* p = reinterpret_cast<const float4*>(
                                    bias + b * 32 + kRow * h + 8 * i);
                                const float4 lo = p[0], hi = p[1];
                                f[0] += lo.x, f[1] += lo.y, f[2] += lo.z, f[3] += lo.w;
                                f[4] += hi.x, f[5] += hi.y, f[6] += hi.z, f[7] += hi.w;
                            }
                            pack8<Out>(f, v + i * (int)sizeof(Out) / 2);
                        }
                        write_block<Out>(mine, v, out + n + kRow * h, g.width, rows,
                                         left - kRow * h, g.vectors);
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
        // rows of no expert are 0
        const int64_t kept = begin[g.experts];
        zero_range(static_cast<Out*>(g.out) + kept * g.width, (g.rows - kept) * g.width,
                   (int64_t)blockIdx.x * (kOutWarps * 32) + threadIdx.x - 128,
                   (int64_t)gridDim.x * (kOutWarps * 32), g.vectors);
    }
    __syncthreads();
    if (kBlocks == 2) cluster_sync();  // the other block's arrivals and products are over too
    if (warp == 1) tmem_free<kBlocks>(tmem, kColumns);
    if (threadIdx.x == 0 && *abort) report(g.d_status, GS_ERR_TIMEOUT);
}

// Rows of `columns` bytes (experts = 0), or a matrix of them an expert, copied
// in boxes of box_rows x 128 bytes, swizzled; zeros behind the last column.
bool make_map8(CUtensorMap* map, const uint8_t* base, int64_t rows, int columns, int experts,
               int box_rows) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t pitch = GS_ROW8_BYTES(columns);
    const cuuint64_t dims[3] = {(cuuint64_t)columns, (cuuint64_t)rows, (cuuint64_t)experts};
    const cuuint64_t strides[2] = {pitch, pitch * (cuuint64_t)rows};
    const cuuint32_t box[3] = {kDeep, (cuuint32_t)box_rows, 1}, unit[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, experts > 0 ? 3 : 2,
                  const_cast<uint8_t*>(base), dims, strides, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Out, int kBlocks, int kWide>
int launch_shape(const LinearArgs& a, Rows8 xs, Rows8 weight, const Product8Args& g,
                 cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!make_map8(&ma, xs.q, a.rows, a.in, 0, kHigh) ||
        !make_map8(&mb, weight.q, a.out, a.in, a.experts, kWide / kBlocks))
        return GS_ERR_CUDA;
    // at most one part-filled tile an expert
    const int64_t items =
        (a.rows / (kHigh * kBlocks) + a.experts) * ceil_div(g.width, kWide);
    static PerDevice raised, resident;
    return launch_walk<kBlocks>(raised, resident, k_product8<Out, kBlocks, kWide>, kThreads,
                                smem_bytes8<kBlocks, kWide>(g.experts),
                                smem_bytes8<kBlocks, kWide>(GS_MAX_EXPERTS), items, s, ma, mb, g);
}

}  // namespace

int launch_linear8_fwd(const LinearArgs& a, Rows8 xs, Rows8 weight, const void* bias, void* ys,
                       cudaStream_t s) {
    Product8Args g{};
    g.offsets = a.offsets;
    g.powers_a = reinterpret_cast<const uint32_t*>(xs.scales);
    g.powers_b = reinterpret_cast<const uint32_t*>(weight.scales);
    g.rows = a.rows;
    g.experts = a.experts;
    g.width = a.out;
    g.depth = a.in;
    g.words = GS_ROW8_SCALES(a.in) / 4;
    g.rounds = ceil_div(a.in, kDeep) > kRound;
    g.vectors = aligned16(ys) && (size_t)a.out * dtype_size(a.dtype) % 16 == 0;
    g.bias = bias;
    g.out = ys;
    g.d_status = a.d_status;
    const int64_t tiles = (a.rows / 256 + a.experts / 2) * ceil_div(a.out, 192);
    int rc = GS_OK;
    with_dtype(a.dtype, [&](auto o) {
        using Out = decltype(o);
        if (a.out > 128 && tiles >= sm_count())
            rc = launch_shape<Out, 2, 192>(a, xs, weight, g, s);
        else
            rc = launch_shape<Out, 1, 128>(a, xs, weight, g, s);
    });
    return rc;
}

}  // namespace gs
