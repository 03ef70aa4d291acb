// The instructions the tensor-core products are built from: bounded waits,
// tiled bulk copies, tensor memory and its matrix instruction (sm_103a).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "gs_device.cuh"

namespace gs {

// A wait on an mbarrier gives up after this long; a tile's copies and
// products take microseconds, so it only ends a wait that nothing will meet.
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// kCluster: what threads of the other block released (mbar_release_at) is seen
// after the wait too, not only what this block's did.
template <bool kCluster>
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    if constexpr (kCluster)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    return done != 0;
}

// Waits for phase `parity`; false once *abort is set (by any waiter of the
// block that gave up) or the limit has passed.  The clock is looked at every
// 256 polls only: reading the global timer takes as long as a slice's
// products.
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait_limited(uint64_t* bar, uint32_t parity,
                                                  volatile int* abort) {
    uint64_t start = 0;
    for (uint32_t polls = 1;; ++polls) {
        if (mbar_try<kCluster>(bar, parity)) return true;
        if (polls % 256) continue;
        if (*abort) return false;
        const uint64_t now = now_ns();
        if (start == 0) start = now;
        if (now - start > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
}

// The same for a whole warp, with one answer.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait_limited<kCluster>(bar, parity, abort));
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Arrives on a barrier of this block, after which this thread's writes to its
// shared memory are seen by whoever in the block waited for it.
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Arrives on the barrier at the same place in block `rank` of the cluster.
// What such arrivals hand to the other block was written by bulk copies or read
// from tensor memory, which barriers and fences of their own order: the arrival
// releases nothing else.  (A release at cluster scope takes 1 us beside other
// traffic and waits for the warp's copies on their way.)
__device__ __forceinline__ void mbar_arrive_at(uint64_t* bar, uint32_t rank) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar)),
        "r"(rank)
        : "memory");
}

// The same, after which this warp's writes to its own shared memory are seen
// by whoever in the cluster waited for it (with kCluster): for what threads of
// one block write and the other block's instructions read.
__device__ __forceinline__ void mbar_release_at(uint64_t* bar, uint32_t rank) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar)),
        "r"(rank)
        : "memory");
}

__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// The barrier at the same place in block `rank` of the cluster.
__device__ __forceinline__ uint32_t mbar_at(uint64_t* bar, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(bar)), "r"(rank));
    return a;
}

// True in one lane of the (converged) warp.  Copies and matrix instructions
// take their operands from registers of the whole warp: issued under this, in
// code that the warp runs together, they need no moves between the two kinds
// (under a test of the lane's number an instruction's issue cost 60 cycles).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Box of a two- or three-dimensional array into shared memory; c0 is the
// innermost coordinate (a multiple of 16 bytes).  bar: a shared address, with
// kBlocks = 2 of either block's barrier.
template <int kBlocks>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            uint32_t bar) {
    if constexpr (kBlocks == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}
template <int kBlocks>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint32_t bar) {
    if constexpr (kBlocks == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
            : "memory");
}

// A box from shared memory to a two-dimensional array (what lies beyond its
// extents is not written), a group of its own among the thread's bulk copies.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
        "cp.async.bulk.commit_group;" ::"l"(map),
        "r"(c0), "r"(c1), "r"(src)
        : "memory");
}
// Until the thread's bulk stores have read shared memory, or are over.
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// By one warp of each of the kBlocks (1 or 2) blocks whose products share
// instructions.
template <int kBlocks>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
    if constexpr (kBlocks == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(where)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(where)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <int kBlocks>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
    if constexpr (kBlocks == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base),
                     "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base),
                     "r"(columns));
}
__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 columns of the warp's 32 lanes: v[i] is this lane's value of column i.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
          "=r"(v[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
        "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
        "r"(v[30]), "r"(v[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_stores() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_loads() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 32 x 16 bytes that lie on end in shared memory (of each of the blocks) into
// four columns of tensor memory: 16 bytes a lane, the same for every quarter of
// the lanes.  Products issued afterwards by the same thread find them there.
template <int kBlocks>
__device__ __forceinline__ void tmem_copy_32x16(uint32_t to, uint32_t smem) {
    const uint64_t from = (uint64_t)((smem & 0x3ffffu) >> 4) | (uint64_t)(128 >> 4) << 16 |
                          (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
    if constexpr (kBlocks == 2)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(from)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(from)
                     : "memory");
}

// Four bytes from global into shared memory without a register between, zeros
// where !in (the address is then not read).
__device__ __forceinline__ void copy_word(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the newest kLeft groups of copies are there.
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Shared-memory operand of the matrix instruction: 128-byte rows, swizzled as
// the tiled copies write them.  With the sum's index contiguous (K-major)
// `stride` is the distance of groups of 8 rows; with it outermost (MN-major)
// `stride` is that of groups of 8 terms and `lead` that of 64-element columns.
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lead >> 4) << 16 |
           (uint64_t)(stride >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction word of kind::f16 with float32 accumulators.
// columns: a multiple of 16 (of 32 with two blocks).
__device__ __forceinline__ constexpr uint32_t mma_word(int rows, int columns, bool bf16,
                                                       bool a_mn, bool b_mn) {
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) |
           (b_mn ? 1u << 16 : 0u) | (uint32_t)(columns >> 3) << 17 | (uint32_t)(rows >> 4) << 24;
}

// With two blocks: each holds half of A's rows, half of B's columns and its
// rows of the result, all at the same places; one block issues.
template <int kBlocks>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t word,
                                        bool accumulate) {
    if constexpr (kBlocks == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate)
            : "memory");
}

// Instruction word of kind::mxf8f6f4, e4m3 operands (K-major) with powers of
// two for every 32 terms of a row, float32 accumulators.  To be added: columns
// >> 3 at bit 17 (columns as mma_word's), and which byte of the words of powers
// is taken at bits 4 (B's) and 29 (A's).
__device__ __forceinline__ constexpr uint32_t mma_word_e4m3(int rows) {
    return 1u << 23 | (uint32_t)(rows >> 4) << 24;
}

// 32 terms; power_a, power_b: the first column of the rows' words in tensor
// memory, row r at lane r % 32 (of every quarter of the lanes) and column r / 32.
template <int kBlocks>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t word,
                                         uint32_t power_a, uint32_t power_b, bool accumulate) {
    if constexpr (kBlocks == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], "
            "p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate), "r"(power_a), "r"(power_b)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], "
            "p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate), "r"(power_a), "r"(power_b)
            : "memory");
}

// Arrives on `bar` (in every one of the blocks) once all products issued so
// far by this thread are done.
template <int kBlocks>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    if constexpr (kBlocks == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_u32(bar))
            : "memory");
}

}  // namespace gs
