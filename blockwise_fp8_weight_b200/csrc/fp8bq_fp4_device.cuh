// fp8bq_fp4_device.cuh -- the sm_100a instructions of the 4-bit products:
// tensor memory, block-scaled tcgen05.mma, their completion barriers, and
// thread-block cluster access.
#pragma once

#include "fp8bq_device.cuh"
#include "fp8bq_fp4.h"

namespace fp8bq {
namespace dev {

// True in one lane of the (whole) warp.  The tensor core's and the copy engine's
// instructions take their operands from the warp's uniform registers; behind
// this, unlike behind a test of the lane's number, the compiler knows that one
// lane runs, and keeps the operands there.  Measured on B200: 128 clocks an
// instruction of 256 x 256 x 64, the tensor cores' rate, instead of 150 to 200.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r));
    return r != 0;
}

// ---------------------------------------------------------------- tensor memory

// One warp; CG CTAs of a pair allocate together (each has a warp make the
// call).  The base address lands in *dst (shared memory).
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(dst)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(dst)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t base, uint32_t cols) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 16 columns of this warp's 32 lanes (lane i of the warp gets lane i of its
// quarter), and the wait for them.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- shared-memory operands

// Descriptor of a K-major operand of 128-byte rows in the 128-byte swizzle
// (groups of eight rows 1024 bytes apart), starting at a 1024-byte boundary;
// 32 bytes (64 codes) along K are two units of its address field.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) |
           (2ull << 61);
}
// ---------------------------------------------------------------- block-scaled MMA

// Instruction word: e2m1 operands, fp32 sums, both K-major, tile m x n, e8m0
// or e4m3 scales; byte `id` of a scale column begins the instruction's.
__host__ __device__ constexpr uint32_t mma_word(int format, int m, int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
           ((format == FP8BQ_MXFP4 ? 1u : 0u) << 23) | ((uint32_t)(m >> 7) << 27);
}
__device__ __forceinline__ uint32_t mma_word_id(uint32_t word, uint32_t id) {
    return word | (id << 4) | (id << 29);
}

template <int FMT, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t word,
                                        uint32_t sa, uint32_t sb, bool add) {
#define FP4_MMA(CGS, VEC)                                                                     \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"                             \
                 "tcgen05.mma.cta_group::" CGS ".kind::mxf4nvf4.block_scale.scale_vec::" VEC  \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(word), \
                 "r"(sa), "r"(sb), "r"((uint32_t)add)                                          \
                 : "memory")
    if constexpr (CG == 1 && FMT == FP8BQ_MXFP4) FP4_MMA("1", "2X");
    else if constexpr (CG == 1) FP4_MMA("1", "4X");
    else if constexpr (FMT == FP8BQ_MXFP4) FP4_MMA("2", "2X");
    else FP4_MMA("2", "4X");
#undef FP4_MMA
}

// Arrive on `bar` once everything this thread has issued to the tensor cores
// is done; CG == 2: on the barrier at this place in both CTAs of the pair.
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_addr(bar)) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                     ".multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)), "h"((uint16_t)3)
                     : "memory");
}

// The same on this CTA's barrier alone.
__device__ __forceinline__ void mma_commit_pair_here(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_addr(bar)) : "memory");
}

// 8 columns of this warp's 32 lanes, and the wait for the stores.
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint4 &a, const uint4 &b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                     addr),
                 "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrive on a barrier of the cluster (an address from peer_addr).  What it
// announces is tensor memory, which the tcgen05 fences order; a release at
// cluster scope would wait for far more (measured: 1 us an arrive while the
// ring is loading).
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
// 3-D TMA tile load into this CTA's shared memory that completes on a barrier
// of the pair's first CTA (no multicast).
__device__ __forceinline__ void tma_load_3d_pair(void *smem_dst, const void *tmap, uint32_t bar,
                                                 int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(smem_dst)),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
// The tile into L2 only: safe before the previous kernel of the stream is
// done, whose writes go through L2 as well.
__device__ __forceinline__ void tma_prefetch_3d(const void *tmap, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(tmap),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ float4 peer_ld4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

}  // namespace dev
}  // namespace fp8bq
