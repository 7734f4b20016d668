// The fifth-generation tensor cores of sm_103a as inline PTX: tensor-memory
// allocation and loads, matrix multiply-accumulate with both operands in
// shared memory, its completion barriers, two-dimensional tensor copies and
// cluster addressing.  Barriers and bounded waits come from mhc_bulk.cuh.
//
// CG is the CTA group: 1, or 2 for a pair of CTAs that compute one tile
// together (each holds half of both operands and half of the accumulators).
#pragma once

#include "mhc_bulk.cuh"

namespace mhc {
namespace umma {

// --------------------------------------------------------------------------
// descriptors
// --------------------------------------------------------------------------

// An operand tile in shared memory, 128-byte swizzled as the tensor copies
// write it (1024-byte aligned):
//  * K-major: rows of 128 bytes of K; groups of 8 rows 1024 bytes apart;
//  * MN-major (2-byte types): panels of 64 M or N values, `panel` bytes apart,
//    each with one 128-byte row per K; groups of 8 K 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t panel) {
    return uint64_t((addr >> 4) & 0x3FFFu) | uint64_t((panel >> 4) & 0x3FFFu) << 16 | uint64_t(1024 >> 4) << 32 |
           uint64_t(1) << 46 | uint64_t(2) << 61;
}

// Instruction descriptor: FP32 accumulators; operand format (kind::f16: 0
// binary16, 1 BF16; kind::f8f6f4: 0 E4M3); M (of the group) and N.
constexpr uint32_t instr_desc(uint32_t format, bool a_mn, bool b_mn, uint32_t M, uint32_t N) {
    return 1u << 4 | format << 7 | format << 10 | uint32_t(a_mn) << 15 | uint32_t(b_mn) << 16 | (N >> 3) << 17 |
           (M >> 4) << 24;
}

// --------------------------------------------------------------------------
// tensor memory
// --------------------------------------------------------------------------

// Whole warp; columns a power of two of at least 32.  With CG = 2 the same
// warp of both CTAs.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :
                     : "r"(smem_addr(dst)), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :
                     : "r"(smem_addr(dst)), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" : : "r"(addr), "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" : : "r"(addr), "r"(columns));
}

// 8 consecutive columns of the thread's lane (a warp reads and writes the
// lanes 32 * (warp % 4) ..); loaded values are valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[8]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st(uint32_t addr, const float (&v)[8]) {
    const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 :
                 : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// After the wait for every load before it; the values pass through it, so that no use of them is moved before it.
__device__ __forceinline__ void tmem_wait_ld(float (&v)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
                 :
                 : "memory");
}

__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// --------------------------------------------------------------------------
// multiply-accumulate (one thread; with CG = 2 of the group's first CTA)
// --------------------------------------------------------------------------

template <int CG, bool FP8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    const uint32_t acc = accumulate ? 1 : 0;
#define MHC_UMMA(GROUP, KIND)                                                       \
    asm volatile(                                                                   \
        "{\n\t"                                                                     \
        ".reg .pred p;\n\t"                                                         \
        "setp.ne.u32 p, %4, 0;\n\t"                                                 \
        "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t"  \
        "}"                                                                         \
        :                                                                           \
        : "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)                              \
        : "memory")
    if constexpr (CG == 1 && !FP8) MHC_UMMA("1", "f16");
    if constexpr (CG == 1 && FP8) MHC_UMMA("1", "f8f6f4");
    if constexpr (CG == 2 && !FP8) MHC_UMMA("2", "f16");
    if constexpr (CG == 2 && FP8) MHC_UMMA("2", "f8f6f4");
#undef MHC_UMMA
}

// Arrives on `bar` (with CG = 2 on that barrier of both CTAs) once every MMA
// this thread has issued is complete.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     :
                     : "r"(bar)
                     : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            :
            : "r"(bar), "h"(uint16_t(3))
            : "memory");
}

// mbar_wait of mhc_bulk.cuh without a call (a kernel whose sums stay in
// registers across a wait would spill them around one), and without a look at
// the timer, which takes longer than most waits, in the first polls.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
    if (try_wait(bar, parity)) return true;
#pragma unroll 1
    for (int i = 0; i < 1024; ++i)
        if (try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    do {
        if (try_wait(bar, parity)) return true;
    } while (global_ns() - t0 < kWaitLimitNs);
    return false;
}

__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" : : "r"(bar), "r"(bytes) : "memory");
}

// One lane of a converged warp.  The loops around copies and multiplications
// run in the whole warp and only these instructions in one lane: their
// operands then stay in the registers that a warp's lanes share, which such
// instructions read (in a loop of one lane each is moved there first, at
// twice the time).
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "}"
        : "=r"(one));
    return one != 0;
}

// A ring of stages: one that a thread is at, and the parity of its round.
struct Ring {
    uint32_t stage = 0, parity = 0;
    __device__ __forceinline__ void next(uint32_t stages) {
        if (++stage == stages) stage = 0, parity ^= 1;
    }
};

// --------------------------------------------------------------------------
// copies and clusters
// --------------------------------------------------------------------------

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" : : "l"(map) : "memory");
}

// The box at element coordinates {c0, c1} of a 2-D tensor map; elements past
// the tensor's end read as zero, and the whole box counts on barrier `bar`
// (a shared::cluster address; with CG = 2 it may be the other CTA's).
template <int CG>
__device__ __forceinline__ void tensor_copy_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
            "[%4];"
            :
            : "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
            "{%2, %3}], [%4];"
            :
            : "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" : : "l"(p)); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// The shared::cluster address of `addr` (a shared address of this CTA) in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Signals without waiting for this thread's stores to global memory (a
// release would: 10% of a product with 8 blocks of K): what it hands over, tensor
// memory, fence_before_sync orders.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" : : "r"(bar) : "memory");
}

// Every thread of every CTA of the cluster.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

}  // namespace umma
}  // namespace mhc
