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
// Two neighbouring blocks work as one on output tiles of 256 x 192 (each holds
// half of the rows of A and of B).  In every block a warp copies slices of 256
// channels into shared memory (tiled bulk copies; the slices of A stay there for
// all column tiles of a piece where they fit), another the rows' words of powers,
// in the order of tensor memory, and the tile's bias comes through a third; one
// warp of the first block issues the matrix instructions, and eight or twelve
// warps move finished accumulators to the output, in boxes (tiled bulk copies
// again) where its rows are whole vectors, while the next tile is computed in the
// other accumulators.  Those leave no room for the powers beside 256 columns
// each, so tiles are 192 columns wide.
//
// 262144 rows, 16 experts, 512 -> 1024, bfloat16 out: 143 us (1920 TFLOP/s, 4.8
// TB/s; the bytes alone take 100 us), float32 229 (178); 65536 rows 1024 -> 1024,
// bfloat16, float16 and float32 out: 72, 76 and 87 us.  Nothing is saturated (131072
// of the first: tensor pipe 37 %, memory 49 %, L2 44 %, issue 46 %); 512 threads
// leave 128 registers each, 32 bytes short (float32 52).  At 137 us, before the
// release below, it took 105 without the output, 133 without the products and 93
// without both.  What is left is the issuing warp's own time,
// 2000 cycles a tile beside 1536 of products (an instruction 42, a commit 90, a
// wait that is over 40), and slices of A that come late from memory behind the
// output's writes.  Steps: powers written to tensor memory from registers by four
// warps 218 us; with the bias read ahead and arrivals that do not wait for the
// writes to global memory 157 (a release at cluster scope by one warp, one a tile,
// cost 35 us for the bias and 35 for the powers, which need it); slices of 256
// channels, A kept, boxes, no division a tile 147; a third slice of A 140; its
// slices on the barrier of B's 137; the second block's powers released at cluster
// scope 143.  Not kept: whole 32-byte sectors stored from
// registers (178 against 159 at that step), prefetches of the next piece's A into
// the L2 (155 against 147).  Two warps that issue in turn are
// unsound as long as each waits only for its own tiles' slices: a barrier's
// parity then stands for two phases.
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

constexpr int kDeep = 256;          // channels a slice: two boxes of 128 bytes a row
constexpr int kHalf = kDeep / 2;
constexpr int kGroup = 2;           // slices a word of powers serves
constexpr int kAccumulators = 2;
constexpr int kSpan = 64;           // columns an output warp writes
constexpr int kRowBytes = 64;       // of the boxes they leave in
// Warps: 0 copies rows, 1 issues products (of a second block: copies powers with
// 2), 2 copies powers, 3 the bias, from 4 on they write the output.
template <int kWide>
constexpr int kOutputs = 4 * kWide / kSpan;
template <int kWide>
constexpr int kThreads = 32 * (4 + kOutputs<kWide>);
// Columns of tensor memory: the accumulators, then the powers of kBuffers
// groups, those of A's rows in four columns and those of B's, 128 rows in four.
constexpr int kColumns = 512, kBuffers = 4, kPowersB = 4;
constexpr int kChunk = 512;         // bytes of 128 rows' words
// Slices summed in an accumulator before they are added to the running sum: as
// many instructions as a round of half types over features.
constexpr int kRound = 16;
static_assert(kRound % kGroup == 0, "a round begins with a word of powers");

struct Product8Args {
    const int32_t* offsets;
    const uint32_t *powers_a, *powers_b;  // a row's words: `words` each
    int64_t rows;
    int experts, width, depth, words;
    int rounds;   // sums take several rounds
    int access;   // bytes at which the output's rows can be written
    const void* bias;
    void* out;
    int32_t* d_status;
};

struct Bars8 {
    // of the first block: a slice of B, and of A where it comes with it, a
    // buffer's words of powers are there (in all blocks), the accumulators may
    // be overwritten
    uint64_t full[4], words_full[kBuffers], acc_empty[kAccumulators];
    // of each block: a slice may be overwritten, powers are in tensor memory,
    // a buffer of them may be overwritten, the accumulators are finished, a
    // tile's bias is there, and may be overwritten
    uint64_t empty_a[4], empty_b[4], powers_full[kBuffers], powers_empty[kBuffers],
        acc_full[kAccumulators], bias_full[kAccumulators], bias_empty[kAccumulators], drain;
    uint32_t tmem;
    int abort;
};

// kSlots, kStages: slices of A and of B in shared memory.  512 channels leave a
// slot of three for the next piece's first slice, whose 1 to 2 us from memory
// under the output's writes are else waited for at every piece (262144 rows 512
// -> 1024, at that step: 140 us with 3 and 4, 150 with 2 and 4, 147 with 2 and 5,
// 152 with 3 and 3, 175 with 4 and 2).
template <int kBlocks_, int kWide_, int kSlots_, int kStages_>
struct Shape8 {
    static constexpr int kBlocks = kBlocks_, kWide = kWide_, kSlots = kSlots_;
    static constexpr int kStages = kStages_;
    static constexpr int kTileHigh = kHigh * kBlocks;
    static constexpr int kBytesA = kHigh * kDeep;
    static constexpr int kPartB = kWide / kBlocks;
    static constexpr int kBytesB = kPartB * kDeep;
    static constexpr int kChunksB = (kWide + 127) / 128;
    static constexpr int kPowers = 4 * (1 + kChunksB);  // columns of a buffer
    static constexpr int kPowerBytes = (1 + kChunksB) * kChunk;
    static constexpr int kStaging = kOutputs<kWide> * 32 * kRowBytes;
    static constexpr int kBias = kAccumulators * kWide * 4;
    // most experts whose ranges fit beside the rest
    static constexpr int kRest = 1024 + kSlots * kBytesA + kStages * kBytesB + kStaging +
                                 kBuffers * kPowerBytes + kBias + sizeof(Bars8);
    static constexpr int kExperts = std::min(GS_MAX_EXPERTS, (232448 - kRest) / 8 - 1);
    static_assert(kPartB * kHalf % 1024 == 0, "swizzled rows begin on 1024 bytes");
    static_assert(kAccumulators * kWide + kBuffers * kPowers <= kColumns, "tensor memory");
};

template <typename S>
constexpr size_t smem_bytes8(int experts) {
    return S::kRest + 2 * sizeof(int32_t) * (size_t)(experts + 1);
}

struct Tile8 {
    int expert;
    int row0, row1;  // rows of the output
    int n0;          // first column
    int q0, q1;      // slices of one round
    bool first, final;  // of the tiles that share their slices of A
};

// The tiles of one pair of blocks (or block), in order; every warp of it walks
// the same ones: an equal share of the items (piece of an expert's rows, column
// tile), column tiles of a piece on end.  They share the slices of A, which stay
// in shared memory, where kSlots hold them all.
// (Where a tile is follows from the one before: a division and a search of the
// experts for each took a third of a tile's time, in every warp.)
template <typename S>
struct Walk8 {
    const int32_t* begin;
    int64_t left;                      // items to come
    int across, count, experts;
    int column = 0, expert = 0, row0 = 0;  // of the next tile
    bool fresh = true;

    __device__ __forceinline__ Walk8(const Product8Args& g, const int32_t* begin_,
                                     const int32_t* prefix)
        : begin(begin_), experts(g.experts) {
        across = (g.width + S::kWide - 1) / S::kWide;
        count = (g.depth + kDeep - 1) / kDeep;
        const int64_t items = (int64_t)prefix[g.experts] * across;
        const int shares = gridDim.x / S::kBlocks, share = blockIdx.x / S::kBlocks;
        const int64_t item = items * share / shares;
        left = items * (share + 1) / shares - item;
        if (left <= 0) return;
        const int piece = (int)(item / across);
        column = (int)(item - (int64_t)piece * across);
        expert = expert_of(prefix, experts, piece);
        row0 = begin[expert] + (piece - prefix[expert]) * S::kTileHigh;
    }

    // c: as the call before left it (q1 = count before the first).
    __device__ __forceinline__ bool next(Tile8& c) {
        if (c.q1 == count) {
            if (left <= 0) return false;
            --left;
            c.n0 = column * S::kWide;
            c.expert = expert;
            c.row0 = row0;
            c.row1 = min(begin[expert + 1], row0 + S::kTileHigh);
            c.q1 = 0;
            c.first = fresh || count > S::kSlots;
            fresh = ++column == across;
            c.final = fresh || left == 0 || count > S::kSlots;
            if (fresh) {
                column = 0;
                row0 += S::kTileHigh;
                if (row0 >= begin[expert + 1]) {
                    do ++expert;
                    while (expert < experts && begin[expert] == begin[expert + 1]);
                    row0 = begin[expert];
                }
            }
        }
        c.q0 = c.q1;
        c.q1 = min(count, c.q0 + kRound);
        return true;
    }
};

// The slices of A in order, a slot for each: `at` of the first of a tile.
template <int kSlots>
struct Slots {
    uint32_t at = 0;
    __device__ __forceinline__ uint32_t slot(int q) const { return (at + q) % kSlots; }
    __device__ __forceinline__ uint32_t turn(int q) const { return (at + q) / kSlots; }
};

template <typename Out, typename S>
__global__ void __launch_bounds__(kThreads<S::kWide>, 1)
    k_product8(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_out, const __grid_constant__ Product8Args g) {
    constexpr int kBlocks = S::kBlocks, kWide = S::kWide;
    extern __shared__ char smem_raw[];
    char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    char* staging = smem + S::kSlots * S::kBytesA + S::kStages * S::kBytesB;
    char* words = staging + S::kStaging;
    float* biases = reinterpret_cast<float*>(words + kBuffers * S::kPowerBytes);
    Bars8& bars = *reinterpret_cast<Bars8*>(biases + kAccumulators * kWide);
    int32_t* begin = reinterpret_cast<int32_t*>(&bars + 1);
    int32_t* prefix = begin + g.experts + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int rank = kBlocks == 2 ? (int)cluster_rank() : 0;

    if (warp == 0 && lane == 0) {
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
        if (g.access == 16) tma_prefetch(&map_out);
        for (int i = 0; i < S::kSlots; ++i) mbar_init(&bars.empty_a[i], 1);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty_b[i], 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(&bars.words_full[i], kBlocks);
            mbar_init(&bars.powers_full[i], 1);
            mbar_init(&bars.powers_empty[i], 1);
        }
        for (int i = 0; i < kAccumulators; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], kOutputs<kWide> * kBlocks);
            mbar_init(&bars.bias_full[i], 1);
            mbar_init(&bars.bias_empty[i], kOutputs<kWide>);
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
    const uint32_t base_b = base + S::kSlots * S::kBytesA;
    const uint32_t powers = tmem + kAccumulators * kWide;
    volatile int* abort = &bars.abort;
    Walk8<S> walk(g, begin, prefix);
    Tile8 c{};
    c.q1 = walk.count;
    // where a running sum takes the second accumulator's place
    const int accumulators = g.rounds ? 1 : kAccumulators;

    if (warp == 0) {
        Ring<S::kStages> at;
        Slots<S::kSlots> slots;
        bool ok = true;
        while (ok && walk.next(c)) {
            const int n0 =
                c.n0 + rank * (tile_columns<kBlocks, kWide>(g.width, c.n0) / kBlocks);
            for (int q = c.q0; q < c.q1; ++q, at.advance()) {
                // a last slice of up to 128 channels is one box
                const int boxes = g.depth - q * kDeep > kHalf ? 2 : 1;
                const uint32_t slot = slots.slot(q), turn = slots.turn(q);
                if (c.first && turn > 0) ok = warp_wait(&bars.empty_a[slot], (turn + 1) & 1, abort);
                if (ok && at.turn > 0)
                    ok = warp_wait(&bars.empty_b[at.stage], (at.turn + 1) & 1, abort);
                if (!ok) break;
                const uint32_t full = kBlocks == 2 ? mbar_at(&bars.full[at.stage], 0)
                                                   : smem_u32(&bars.full[at.stage]);
                if (elect_one()) {
                    if (rank == 0)
                        mbar_expect_tx(&bars.full[at.stage],
                                       boxes * kBlocks *
                                           (S::kBytesB / 2 + (c.first ? S::kBytesA / 2 : 0)));
                    for (int i = 0; i < boxes && c.first; ++i)
                        tma_load_2d<kBlocks>(base + slot * S::kBytesA + i * S::kBytesA / 2, &map_a,
                                             q * kDeep + i * kHalf, c.row0 + rank * kHigh, full);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_3d<kBlocks>(base_b + at.stage * S::kBytesB + i * S::kBytesB / 2,
                                             &map_b, q * kDeep + i * kHalf, n0, c.expert, full);
                }
                __syncwarp();
            }
            if (c.final && c.q1 == walk.count) slots.at += walk.count;
        }
        if (!ok && rank == 0)  // let the copies in flight land before the blocks go
            for (int i = 0; i < S::kStages; ++i) {
                // stages [stage, ...) were last filled one turn ago
                const uint32_t turn = i < (int)at.stage ? at.turn : at.turn - 1;
                int none = 0;
                if (turn != ~0u) mbar_wait_limited(&bars.full[i], turn & 1, &none);
            }
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t word0 = mma_word_e4m3(S::kTileHigh);
        const uint64_t from_a = smem_operand(base, 16, 1024);
        const uint64_t from_b = smem_operand(base_b, 16, 1024);
        Ring<S::kStages> at;
        Slots<S::kSlots> slots;
        Ring<kAccumulators> acc;
        Ring<kBuffers> buffer;
        bool ok = true;
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
                const uint32_t slot = slots.slot(q);
                ok = warp_wait(&bars.full[at.stage], at.turn & 1, abort);
                if (!ok) break;
                const uint64_t da = from_a + slot * (S::kBytesA >> 4);
                const uint64_t db = from_b + at.stage * (S::kBytesB >> 4);
                const uint32_t from = powers + buffer.stage * S::kPowers;
                const bool last = q % kGroup == kGroup - 1 || q + 1 == c.q1;
                // 32 channels an instruction, four in turn with the same byte
                const uint32_t turned = word | (uint32_t)(q % kGroup) << 5 |
                                        (uint32_t)(q % kGroup) << 30;
                const auto product = [&](int j) {
                    constexpr int kJumpA = S::kBytesA / 2 >> 4, kJumpB = S::kBytesB / 2 >> 4;
                    mma_e4m3<kBlocks>(d, da + j / 4 * kJumpA + j % 4 * (32 >> 4),
                                      db + j / 4 * kJumpB + j % 4 * (32 >> 4),
                                      turned | (uint32_t)(j / 4) << 4 | (uint32_t)(j / 4) << 29,
                                      from, from + kPowersB, q > c.q0 || j > 0);
                };
                const int steps = (g.depth - q * kDeep + 31) / 32;
                if (elect_one()) {
                    if (steps >= kDeep / 32) {
#pragma unroll
                        for (int j = 0; j < kDeep / 32; ++j) product(j);
                    } else {
                        for (int j = 0; j < steps; ++j) product(j);
                    }
                    mma_commit<kBlocks>(&bars.empty_b[at.stage]);
                    if (c.final) mma_commit<kBlocks>(&bars.empty_a[slot]);
                    if (last) mma_commit<kBlocks>(&bars.powers_empty[buffer.stage]);
                    if (q + 1 == c.q1) mma_commit<kBlocks>(&bars.acc_full[acc.stage]);
                }
                __syncwarp();
                if (last) buffer.advance();
            }
            acc.advance(accumulators);
            if (c.final && c.q1 == walk.count) slots.at += walk.count;
        }
        // nothing is still writing tensor memory when it is freed
        if (elect_one()) mma_commit<kBlocks>(&bars.drain);
        __syncwarp();
        int none = 0;
        mbar_wait_limited(&bars.drain, 0, &none);
    } else if (warp == 2 || (warp == 1 && rank != 0)) {
        // words of powers, a buffer a group; the first block's warp has all of
        // them copied into tensor memory when the copies of two more groups are
        // on their way (the warp that issues the products lost a fifth of its
        // time to that).  The second block's words are read by the first one's
        // instructions: they are fenced for those and released at cluster scope,
        // which takes as long as a tile, so two warps do it in turn, each with
        // half of the buffers (262144 rows 512 -> 1024: 143 us, 180 with one; 153
        // with one that releases two buffers together; 155 with copies of the next
        // words on their way, which the release waits for too; 166 with all words
        // written from the first block into the second's shared memory).
        constexpr int kBehind = 2;
        static_assert(kBehind < kBuffers, "a buffer that is not passed on is not waited for");
        Ring<kBuffers> buffer, next;
        bool ok = true;
        int waiting = 0;
        const auto pass_on = [&] {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.words_full[next.stage]);
            ok = warp_wait<kBlocks == 2>(&bars.words_full[next.stage], next.turn & 1, abort);
            if (!ok) return;
            tmem_fence_after();
            const uint32_t chunk = smem_u32(words) + next.stage * S::kPowerBytes;
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < 1 + S::kChunksB; ++j)
                    tmem_copy_32x16<kBlocks>(powers + next.stage * S::kPowers + j * 4,
                                             chunk + j * kChunk);
                mma_commit<kBlocks>(&bars.powers_full[next.stage]);
            }
            __syncwarp();
            next.advance();
        };
        while (ok && walk.next(c)) {
            const int row = c.row0 + rank * kHigh + lane, n = c.n0 + lane;
            const uint32_t* a = g.powers_a + (int64_t)row * g.words;
            const uint32_t* b = g.powers_b + ((int64_t)c.expert * g.width + n) * g.words;
            for (int q = c.q0; q < c.q1; q += kGroup, buffer.advance()) {
                if (rank != 0 && (buffer.stage & 1) != (warp & 1)) continue;
                ok = buffer.turn == 0 ||
                     warp_wait(&bars.powers_empty[buffer.stage], (buffer.turn + 1) & 1, abort);
                if (!ok) break;
                const int word = q / kGroup;
                // row r's word at 16 (r % 32) + 4 (r / 32): tensor memory's order
                const uint32_t to =
                    smem_u32(words) + buffer.stage * S::kPowerBytes + lane * 16;
#pragma unroll
                for (int i = 0; i < kHigh / 32; ++i) {
                    const bool in = row + i * 32 < c.row1;
                    copy_word(to + i * 4, in ? a + (int64_t)i * 32 * g.words + word : g.powers_a,
                              in);
                }
#pragma unroll
                for (int i = 0; i < kWide / 32; ++i) {
                    const bool in = n + i * 32 < g.width;
                    copy_word(to + (1 + i / 4) * kChunk + i % 4 * 4,
                              in ? b + (int64_t)i * 32 * g.words + word : g.powers_b, in);
                }
                copy_group();
                if (rank != 0) {
                    copy_wait<0>();
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_release_at(&bars.words_full[buffer.stage], 0);
                } else if (waiting == kBehind) {
                    copy_wait<kBehind>();
                    pass_on();
                    if (!ok) break;
                } else {
                    ++waiting;
                }
            }
        }
        copy_wait<0>();
        for (; ok && waiting > 0; --waiting) pass_on();
        if (!ok && rank == 0) {  // let the copies into tensor memory end
            int none = 0;
            for (int i = 0; i < kBuffers; ++i) {
                const uint32_t turn = i < (int)next.stage ? next.turn : next.turn - 1;
                if (turn != ~0u) mbar_wait_limited(&bars.powers_full[i], turn & 1, &none);
            }
        }
    } else if (warp == 3) {
        Ring<kAccumulators> at;
        bool ok = g.bias != nullptr;
        while (ok && walk.next(c)) {
            if (c.q1 < walk.count) continue;  // added to what the last round leaves
            if (at.turn > 0) ok = warp_wait(&bars.bias_empty[at.stage], (at.turn + 1) & 1, abort);
            if (!ok) break;
            const Out* p = static_cast<const Out*>(g.bias) + (int64_t)c.expert * g.width;
#pragma unroll
            for (int i = lane; i < kWide; i += 32)
                biases[at.stage * kWide + i] = c.n0 + i < g.width ? to_f(p[c.n0 + i]) : 0.f;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.bias_full[at.stage]);
            at.advance();
        }
    } else {
        const int q = warp & 3;  // tensor-memory lanes [32 q, 32 q + 32)
        const int first = (warp - 4) / 4 * kSpan;
        char* mine = staging + (warp - 4) * 32 * kRowBytes;
        constexpr int kRow = kRowBytes / (int)sizeof(Out);  // columns written at a time
        constexpr int kVectors = kRowBytes / 16;
        Ring<kAccumulators> acc, added;
        bool ok = true;
        for (; ok && walk.next(c); acc.advance(accumulators)) {
            const uint32_t from =
                tmem + ((uint32_t)(q * 32) << 16) + acc.stage * kWide + first;
            const int row = rank * kHigh + q * 32;  // first row in the tile
            Out* out = static_cast<Out*>(g.out) + ((int64_t)c.row0 + row) * g.width + c.n0 + first;
            const int rows = c.row1 - c.row0 - row;
            const bool last = c.q1 == walk.count, with_bias = last && g.bias;
            ok = warp_wait(&bars.acc_full[acc.stage], acc.turn & 1, abort);
            if (!ok) break;
            tmem_fence_after();
            if (with_bias) {
                ok = warp_wait(&bars.bias_full[added.stage], added.turn & 1, abort);
                if (!ok) break;
            }
            const float* bias = biases + added.stage * kWide + first;
            uint32_t u[kSpan];
#pragma unroll
            for (int i = 0; i < kSpan; i += 32) tmem_load32(from + i, u + i);
            tmem_wait_loads();
            const uint32_t sum = from + kWide;
            if (c.q0 > 0) {
#pragma unroll
                for (int i = 0; i < kSpan; i += 32) {
                    uint32_t was[32];
                    tmem_load32(sum + i, was);
                    tmem_wait_loads();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        u[i + j] = __float_as_uint(__uint_as_float(was[j]) +
                                                   __uint_as_float(u[i + j]));
                }
            }
            if (!last) {
#pragma unroll
                for (int i = 0; i < kSpan; i += 32) tmem_store32(sum + i, u + i);
                tmem_wait_stores();
            }
            // the accumulator is read: its next product may begin
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(&bars.acc_empty[acc.stage], 0);
            const int left = g.width - c.n0 - first;  // columns from here on
            // whole rows of whole vectors go out as boxes
            const bool boxed = g.access == 16 && rows >= 32;
            const auto write = [&](auto biased) {
#pragma unroll
                for (int b = 0; b < kSpan / kRow; ++b) {
                    if (b * kRow >= left) break;
                    uint4 v[kVectors];
#pragma unroll
                    for (int i = 0; i < kRow / 8; ++i) {
                        float f[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(u[b * kRow + 8 * i + j]);
                        if constexpr (decltype(biased)::value) {
                            const float4* p =
                                reinterpret_cast<const float4*>(bias + b * kRow + 8 * i);
                            const float4 lo = p[0], hi = p[1];
                            f[0] += lo.x, f[1] += lo.y, f[2] += lo.z, f[3] += lo.w;
                            f[4] += hi.x, f[5] += hi.y, f[6] += hi.z, f[7] += hi.w;
                        }
                        pack8<Out>(f, v + i * (int)sizeof(Out) / 2);
                    }
                    // the box before has left
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
                    if (boxed) {
#pragma unroll
                        for (int j = 0; j < kVectors; ++j)
                            *reinterpret_cast<uint4*>(mine + lane * kRowBytes +
                                                      ((j ^ (lane >> 1 & 3)) << 4)) = v[j];
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0)
                            tma_store_2d(&map_out, smem_u32(mine), c.n0 + first + b * kRow,
                                         c.row0 + row);
                    } else {
                        write_block<Out>(mine, v, out + b * kRow, g.width, rows, left - b * kRow,
                                         g.access);
                    }
                }
            };
            if (with_bias)
                write(std::true_type{});
            else if (last)
                write(std::false_type{});
            if (with_bias) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.bias_empty[added.stage]);
                added.advance();
            }
        }
        if (lane == 0) bulk_wait();
        // rows of no expert are 0
        const int64_t kept = begin[g.experts];
        zero_range(static_cast<Out*>(g.out) + kept * g.width, (g.rows - kept) * g.width,
                   (int64_t)blockIdx.x * (kOutputs<kWide> * 32) + threadIdx.x - 128,
                   (int64_t)gridDim.x * (kOutputs<kWide> * 32));
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
    const cuuint32_t box[3] = {kHalf, (cuuint32_t)box_rows, 1}, unit[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, experts > 0 ? 3 : 2,
                  const_cast<uint8_t*>(base), dims, strides, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output in boxes of 32 rows x kRowBytes, swizzled.
bool make_out_map(CUtensorMap* map, int dtype, void* ys, int64_t rows, int width) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const size_t size = dtype_size(dtype);
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, pitch = width * size;
    const cuuint32_t box[2] = {(cuuint32_t)(kRowBytes / size), 32}, unit[2] = {1, 1};
    return encode(map,
                  dtype == GS_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                  : dtype == GS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  2, ys, dims, &pitch, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Out, typename S>
int launch_shape(const LinearArgs& a, Rows8 xs, Rows8 weight, const Product8Args& g,
                 cudaStream_t s) {
    CUtensorMap ma, mb, mo{};
    if (g.access == 16 && !make_out_map(&mo, a.dtype, g.out, a.rows, a.out))
        return GS_ERR_CUDA;
    if (!make_map8(&ma, xs.q, a.rows, a.in, 0, kHigh) ||
        !make_map8(&mb, weight.q, a.out, a.in, a.experts, S::kPartB))
        return GS_ERR_CUDA;
    // at most one part-filled tile an expert
    const int64_t items = (a.rows / S::kTileHigh + a.experts) * ceil_div(g.width, S::kWide);
    static PerDevice raised, resident;
    return launch_walk<S::kBlocks>(raised, resident, k_product8<Out, S>, kThreads<S::kWide>,
                                   smem_bytes8<S>(g.experts), smem_bytes8<S>(S::kExperts),
                                   items, s, ma, mb, mo, g);
}

}  // namespace

int launch_linear8_fwd(const LinearArgs& a, Rows8 xs, Rows8 weight, const void* bias, void* ys,
                       cudaStream_t s) {
    if (few_rows(a, true)) {
        launch_few8_fwd(a, xs, weight, bias, ys, s);
        return GS_OK;
    }
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
    const int size = (int)dtype_size(a.dtype);
    g.access = access_bytes(ys, (size_t)a.out * size, size);
    g.bias = bias;
    g.out = ys;
    g.d_status = a.d_status;
    // Two blocks a tile of 256 x 192 where those fill every pair of SMs twice,
    // one block a tile of 128 x 128 else (512 -> 1024 bf16: 40000 rows 33 us in
    // pairs and 33 single, 4000 12.3 and 10.3).
    const int64_t tiles = (a.rows / 256 + a.experts / 2) * ceil_div(a.out, 192);
    int rc = GS_OK;
    with_dtype(a.dtype, [&](auto o) {
        using Out = decltype(o);
        if (a.out <= 128 || tiles < sm_count())
            rc = launch_shape<Out, Shape8<1, 128, 3, 3>>(a, xs, weight, g, s);
        else if (a.experts <= Shape8<2, 192, 3, 4>::kExperts)
            rc = launch_shape<Out, Shape8<2, 192, 3, 4>>(a, xs, weight, g, s);
        else
            rc = launch_shape<Out, Shape8<2, 192, 3, 3>>(a, xs, weight, g, s);
    });
    return rc;
}

}  // namespace gs
