/*
 * tcgen05.cuh -- the matrix unit of sm_103a as head_loss.cu uses it: a pair of blocks on two SMs
 * works on one tile, shared-memory operand tiles brought in by TMA, accumulators in tensor
 * memory, mbarriers with bounded waits.
 *
 * Operands are 16-bit tiles under the 128-byte swizzle, cut into boxes of 128 rows of 128 bytes
 * (16 KB, one TMA copy each; a copy takes the SM's TMA unit about 70 cycles and 1.36 a row, so
 * that boxes of 64 rows, measured, bring in 53 bytes a cycle and of 128 rows 67, against the 64
 * that the matrix unit uses up on tiles of 256 x 256):
 *   K-major   a box is 128 rows of the operand by 64 of K; 8-row groups lie 1,024 bytes apart, a
 *             step of 16 along K is 32 bytes, the next 64 of K are the next box
 *   MN-major  a box is 128 of K by 64 of the operand's rows: each K row holds 64 neighbours.
 *             The next 64 lie a box further, the next 8 of K 1,024 bytes, a step of 16 along
 *             K 2,048 bytes
 */
#pragma once

#include "rows.cuh"

#include <cuda.h>

namespace zero {
namespace {

constexpr uint32_t kBoxRows = 128, kBoxBytes = 128 * kBoxRows;

__device__ __forceinline__ uint64_t operand_desc(uint32_t smem, bool mn_major)
{
    const uint64_t lead = mn_major ? kBoxBytes / 16 : 1;
    return (uint64_t)((smem & 0x3ffff) >> 4) | lead << 16 | (uint64_t)(1024 / 16) << 32 | 1ull << 46 | 2ull << 61;
}

/* Bytes / 16 to step q of 16 along K. */
__device__ __forceinline__ uint32_t k_step(bool mn_major, uint32_t q)
{
    return mn_major ? 128 * q : q / 4 * (kBoxBytes / 16) + q % 4 * 2;
}

/* fp32 accumulation of an M x N tile; A and B both bf16 or both fp16. */
__device__ __forceinline__ uint32_t instr_desc(bool f16, bool a_mn, bool b_mn, uint32_t m, uint32_t n)
{
    const uint32_t type = f16 ? 0 : 1;
    return 1u << 4 | type << 7 | type << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (n / 8) << 17 |
           (m / 16) << 24;
}

/* One 256 x N x 16 step by the pair of blocks: each holds its 128 rows of A and of D and half of
 * B's rows, at the same shared and tensor memory addresses; the first block issues. */
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                 "r"(accumulate)
                 : "memory");
}

/* Arrives on the mbarrier at this address in both blocks once every MMA issued so far by this
 * thread has finished. */
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc(uint32_t smem, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns));
}

/* 32 columns of the warp's 32 accumulator rows: thread l gets row l.  The whole warp executes the
 * load together (.aligned), so it is brought together first: what comes before may have taken lanes
 * apart (a row's end, the lane that sends a bulk copy). */
__device__ __forceinline__ void tmem_load32(uint32_t at, float (&v)[32])
{
    uint32_t r[32];
    __syncwarp();
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
}

/* The same of 16 columns. */
__device__ __forceinline__ void tmem_load16(uint32_t at, float (&v)[16])
{
    uint32_t r[16];
    __syncwarp();
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(r[i]);
}

/* One box at (x: the contiguous dimension, y: the rows); what lies outside the tensor is 0.
 * x is a multiple of 8 elements.  bar: of either block of the pair. */
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void map_prefetch(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

/* A warp's finished columns on their way out: written row by row (thread l: row l) under the
 * swizzle of a tensor map whose box is 32 rows of kBytes, then one bulk copy, which what lies
 * outside the tensor is cut from.  The lane that issues it also waits before the next one.  v: the
 * row's N pieces of 16 bytes from `first` on. */
template <uint32_t kBytes, uint32_t N>
__device__ __forceinline__ void stage_row(uint32_t smem, uint32_t lane, const uint4 (&v)[N], uint32_t first = 0)
{
    static_assert(kBytes == 128 || kBytes == 64, "the swizzle of 128 or of 64 bytes");
    const uint32_t turn = kBytes == 128 ? lane & 7 : lane >> 1 & 3;
#pragma unroll
    for (uint32_t q = 0; q < N; ++q)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(smem + lane * kBytes + (((first + q) ^ turn) << 4)),
                     "r"(v[q].x), "r"(v[q].y), "r"(v[q].z), "r"(v[q].w)
                     : "memory");
}

__device__ __forceinline__ void stage_wait(uint32_t lane)
{
    if (lane == 0)
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

__device__ __forceinline__ void stage_send(uint32_t smem, uint32_t lane, const CUtensorMap* map, uint32_t x, uint32_t y,
                                           bool add)
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
        if (add)
            asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                         "r"(x), "r"(y), "r"(smem)
                         : "memory");
        else
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                         "r"(x), "r"(y), "r"(smem)
                         : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

/* A shared address of this block as the pair's first block has it. */
__device__ __forceinline__ uint32_t of_first(uint32_t addr)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(0));
    return r;
}

/* True in one lane of the (converged) warp: the compiler then knows that what the lane issues
 * has the warp's uniform operands, which a test of the lane's number does not tell it. */
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p;
}

__device__ __forceinline__ uint32_t block_of_pair()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void pair_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n"
                 "barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}

/* On a barrier of either block (of_first). */
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool bar_done(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok;
}

/* The same without waiting. */
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok;
}

__device__ __noinline__ bool bar_wait_bounded(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up)
{
    const long long t0 = clock64();
    while (!bar_done(bar, parity)) {
        if (*gave_up)
            return false;
        if (clock64() - t0 > 4000000000LL) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

/* A wait of at most ~2 s, cut short where another thread of the block has given up. */
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up)
{
    return bar_done(bar, parity) || bar_wait_bounded(bar, parity, gave_up);
}

/* The same by a whole warp, with one answer. */
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up)
{
    return __all_sync(0xffffffffu, bar_wait(bar, parity, gave_up));
}

/* A row-major tensor of elements of type t, for boxes of box_cols (64 or 128 bytes, the swizzle)
 * by box_rows.  False where the driver refuses it (the address, the stride and the extents are
 * checked by the callers). */
bool tensor_map(CUtensorMap* map, const void* p, zero_dtype_t t, uint64_t cols, uint64_t rows, uint64_t stride,
                uint32_t box_cols, uint32_t box_rows);

}  // namespace
}  // namespace zero
