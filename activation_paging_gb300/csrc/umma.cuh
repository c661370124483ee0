// Tensor-core building blocks of the experts' products: barriers with bounded
// waits, tensor maps and their copies, operand descriptors, and the products
// and read-out of accumulators in tensor memory.
#pragma once

#include <cuda.h>

#include "ap_common.cuh"

namespace ap {
namespace umma {

// ---- barriers in shared memory ---------------------------------------------------
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_done()
{
    asm volatile("fence.mbarrier_init.release.cluster;\n\tfence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits for the phase of this parity to end; gives up after a number of tries
// (each of which may sleep for a while), or once another wait of the block gave
// up (*dead).  A million tries take some ten milliseconds at the least, which is
// no limit to a wait for work whose length the sizes give: such a wait names a
// count that moves while the work does (*moved), and the tries are those without
// a move.
constexpr uint32_t kTries = 1u << 20;
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *dead, const volatile uint32_t *moved = nullptr)
{
    uint32_t ok = 0, seen = moved ? *moved : 0;
    for (uint32_t i = 0; i < kTries; ++i) {
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
        if (ok) return true;
        if ((i & 255) != 255) continue;
        if (*dead) return false;
        if (moved && *moved != seen) {
            seen = *moved;
            i = 0;
        }
    }
    *dead = 1;
    return false;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
    return one;
}
// The same barrier in another block of the cluster: its address, and an arrival there.
__device__ __forceinline__ void bar_arrive_at(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// ---- copies by tensor map ---------------------------------------------------------
// PAIR: the barrier may be the other block's of a pair (a cluster address).
template <bool PAIR> __device__ __forceinline__ void tma_2d(uint32_t to, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                     "[%0], [%1, {%2, %3}], [%4];" ::"r"(to),
                     "l"(map), "r"(x), "r"(y), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                         to),
                     "l"(map), "r"(x), "r"(y), "r"(bar)
                     : "memory");
}
template <bool PAIR> __device__ __forceinline__ void tma_3d(uint32_t to, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                     "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(to),
                     "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(to),
                     "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                     : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tma_5d(uint32_t to, const CUtensorMap *map, int x, int y, int z, int u, int v, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                     "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(to),
                     "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(to),
                     "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar)
                     : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// What threads wrote to shared memory becomes visible to the tensor cores.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tensor memory ------------------------------------------------------------------
// (one whole warp each; PAIR: of both blocks of a pair, which do it together)
template <bool PAIR> __device__ __forceinline__ void tmem_alloc(uint32_t to, uint32_t columns)
{
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <bool PAIR> __device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Operands lie in shared memory as lines of 128 bytes, eight lines to a
// swizzled atom of 1024 bytes.
// Contiguous along the contraction ("K"): a line is 64 values of one row; the
// next eight rows lie `next` = 1024 bytes on.  16 values further along the
// contraction: 32 bytes.
// Contiguous along the rows ("MN"): a line is 64 rows' values at one place of
// the contraction; eight places on: 1024 bytes; 64 rows on: `chunk` bytes.  16
// places further: 2048 bytes.
__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t chunk)
{
    return (uint64_t)((at & 0x3ffff) >> 4) | (uint64_t)(chunk >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// BF16 operands, FP32 accumulators, m x n.
__device__ __forceinline__ uint32_t shape_of(int m, int n, bool a_mn, bool b_mn)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(m >> 4) << 24;
}
// acc (+)= A B^T over 16 places of the contraction (one thread).  PAIR: the first
// block of a pair multiplies for both: each has half of A's rows and the
// accumulator's lanes for them, and half of B's.
template <bool PAIR> __device__ __forceinline__ void mma(uint32_t acc, uint64_t a, uint64_t b, uint32_t shape, bool add)
{
    if constexpr (PAIR)
        asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(acc),
                     "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
                     : "memory");
    else
        asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(acc),
                     "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
                     : "memory");
}
// The barrier (PAIR: of both blocks) gets one arrival when all products that this thread asked for are done.
template <bool PAIR> __device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"((uint16_t)3)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void acc_load(uint32_t at, float (&v)[32])
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                   "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(at)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The same 32 lanes and columns as two halves of 16 lanes in the layout of 8 x 8
// matrices: v[h][4 i + 2 s + c] is lane 16 h + 8 s + l / 4 and column 8 i +
// 2 (l % 4) + c of the warp's lane l.
__device__ __forceinline__ void acc_load_tiles(uint32_t at, float (&v)[2][16])
{
    uint32_t r[2][16];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                     "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                     : "=r"(r[h][0]), "=r"(r[h][1]), "=r"(r[h][2]), "=r"(r[h][3]), "=r"(r[h][4]), "=r"(r[h][5]), "=r"(r[h][6]),
                       "=r"(r[h][7]), "=r"(r[h][8]), "=r"(r[h][9]), "=r"(r[h][10]), "=r"(r[h][11]), "=r"(r[h][12]),
                       "=r"(r[h][13]), "=r"(r[h][14]), "=r"(r[h][15])
                     : "r"(at + ((uint32_t)h << 20))
                     : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[h][i] = __uint_as_float(r[h][i]);
}

// The same 32 lanes and columns of one place added to those of another (add) or
// put there: columns that no product writes.  acc_folded() ends the stores.
__device__ __forceinline__ void acc_fold(uint32_t from, uint32_t to, bool add)
{
    uint32_t r[32], q[32];
    if (add) {
        asm volatile(
                     "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%64];\n\t"
                     "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%65];\n\t"
                     "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47}, [%66];\n\t"
                     "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%67];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                       "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
                       "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15]),
                       "=r"(q[16]), "=r"(q[17]), "=r"(q[18]), "=r"(q[19]), "=r"(q[20]), "=r"(q[21]), "=r"(q[22]), "=r"(q[23]), "=r"(q[24]), "=r"(q[25]), "=r"(q[26]), "=r"(q[27]), "=r"(q[28]), "=r"(q[29]), "=r"(q[30]), "=r"(q[31])
                     : "r"(from), "r"(from + (1u << 20)), "r"(to), "r"(to + (1u << 20))
                     : "memory");
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) + __uint_as_float(q[i]));
    } else {
        float v[2][16];
        acc_load_tiles(from, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i / 16][i % 16]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
                     "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(to + ((uint32_t)h << 20)),
                     "r"(r[h * 16 + 0]), "r"(r[h * 16 + 1]), "r"(r[h * 16 + 2]), "r"(r[h * 16 + 3]), "r"(r[h * 16 + 4]), "r"(r[h * 16 + 5]), "r"(r[h * 16 + 6]), "r"(r[h * 16 + 7]), "r"(r[h * 16 + 8]), "r"(r[h * 16 + 9]), "r"(r[h * 16 + 10]), "r"(r[h * 16 + 11]), "r"(r[h * 16 + 12]), "r"(r[h * 16 + 13]), "r"(r[h * 16 + 14]), "r"(r[h * 16 + 15])
                     : "memory");
}
__device__ __forceinline__ void acc_folded() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- 8 x 8 matrices of 16-bit values, transposed on their way --------------------------
// Lane l gives the address of row l % 8 of matrix l / 8 in memory; a lane holds
// two neighbours of a column there.
__device__ __forceinline__ void matrices_store(uint32_t at, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void matrices_load(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

// ---- host ---------------------------------------------------------------------------
// A map of BF16 values, innermost first, with lines of 128 bytes, swizzled;
// pitches in elements for the dimensions after the first.
bool make_map(CUtensorMap *map, const void *base, int dims, const uint64_t *extent, const uint64_t *pitch, const uint32_t *box);

} // namespace umma
} // namespace ap
