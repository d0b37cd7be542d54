// tcgen05.cuh -- thin inline-PTX wrappers of the 5th-generation tensor cores
// for a pair of CTAs (cta_group::2): tensor memory, matrix instructions and
// their completion, the tensor copies that feed them, and the descriptors of
// operands in shared memory.
#pragma once

#include <cstdint>
#include <cuda.h>  // CUtensorMap only; no libcuda symbol is linked
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace nqg {

// True in one lane of a converged warp.  Copies and matrix instructions are issued under it by a warp that stays together:
// their operands then go to uniform registers as they are.
__device__ __forceinline__ bool elect_lane()
{
    uint32_t yes;
    asm volatile("{ .reg .pred p;\n"
                 "  elect.sync _|p, 0xffffffff;\n"
                 "  selp.u32 %0, 1, 0, p; }"
                 : "=r"(yes));
    return yes != 0;
}

// ---------------------------------------------------------------- tensor memory

// One warp of each CTA of the pair, all lanes; the address is written to shared memory.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void tmem_free_pair(uint32_t at, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}

__device__ __forceinline__ void tcgen05_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of 16 lanes, as fragments of 8 x 8: v[4 b + 2 s + i] is column 8 b + 2 (lane % 4) + i of lane 8 s + lane / 4.
__device__ __forceinline__ void tmem_load_fragments(uint32_t at, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
                   "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(at)
                 : "memory");
}

// The same for 64 columns.
__device__ __forceinline__ void tmem_load_fragments(uint32_t at, uint32_t (&v)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
                   "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
                   "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
                   "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
                 : "r"(at)
                 : "memory");
}

// Four fragments of 8 x 8 16-bit values (two of a row a thread) to shared memory as rows of 16 bytes, or (across) their
// transposes: thread L gives the address of row L % 8 of fragment L / 8.
template <bool ACROSS>
__device__ __forceinline__ void store_fragments(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    if constexpr (ACROSS)
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
    else
        asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------- matrix instructions

// D[256, N] (+)= A[256, 16] B[N, 16]^T over the pair: each CTA holds 128 rows of A and of D and N / 2 rows of B.
__device__ __forceinline__ void mma_pair_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{ .reg .pred p;\n"
                 "  setp.ne.u32 p, %4, 0;\n"
                 "  tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
                 : "memory");
}

// Arrives at the barrier of this offset in the cluster's CTAs of `ctas` (a bit each: the pair's two) once every matrix
// instruction this thread has issued is complete.
__device__ __forceinline__ void mma_pair_commit(uint32_t bar, uint32_t ctas)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(static_cast<uint16_t>(ctas))
                 : "memory");
}

// fp32 sums of 16-bit operands; an operand is "across" where its rows run along the contraction (MN-major).
__host__ __device__ constexpr uint32_t mma_f16_descriptor(bool bf16, bool a_across, bool b_across, uint32_t M, uint32_t N)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_across ? 1u << 15 : 0u) | (b_across ? 1u << 16 : 0u) |
           ((N >> 3) << 17) | ((M >> 4) << 24);
}

// An operand in shared memory in 128-byte lines with the 128-byte swizzle, 1024-byte aligned.  Along: a line is 64
// elements of the contraction of one row, eight rows a group.  Across: a line is 64 rows at one place of the
// contraction, eight places a group, and the next 64 rows lie `chunk` bytes on.
__device__ __forceinline__ uint64_t operand_along(uint32_t at)
{
    return static_cast<uint64_t>((at >> 4) & 0x3FFFu) | (uint64_t{1} << 16) | (uint64_t{1024 >> 4} << 32) | (uint64_t{1} << 46) |
           (uint64_t{2} << 61);
}

__device__ __forceinline__ uint64_t operand_across(uint32_t at, uint32_t chunk)
{
    return static_cast<uint64_t>((at >> 4) & 0x3FFFu) | (static_cast<uint64_t>(chunk >> 4) << 16) | (uint64_t{1024 >> 4} << 32) |
           (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// ----------------------------------------------------------------- the pair's barriers

// Arrives at a barrier of either CTA (address from cluster_map).  These order nothing beyond this CTA: what they announce is
// tensor memory (with its own fences) or a copy's data (whose transaction bytes say when it is there).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// A float to shared memory of a CTA of the cluster (address from cluster_map).
__device__ __forceinline__ void store_cluster(uint32_t at, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// A box of a three- or four-dimensional tensor to this CTA's shared memory, counted on a barrier of either CTA.
__device__ __forceinline__ void tensor_load_pair(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tensor_load_pair(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z, int32_t u, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

} // namespace nqg
