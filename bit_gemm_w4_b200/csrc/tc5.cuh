// Tensor memory and block-scaled tensor-core MMAs (tcgen05) for the 4-bit
// float products. kGroup is the CTA group: 1, or 2 for a pair of CTAs that
// work on one tile.
#pragma once

#include "common.cuh"

namespace mq {
namespace tc5 {

template <int kCtas>
__device__ __forceinline__ void alloc(uint32_t *slot, uint32_t ncols) {
    if constexpr (kCtas == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}

template <int kCtas>
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t ncols) {
    if constexpr (kCtas == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// One lane of a converged warp. The instructions below take their operands
// from registers that a warp shares: a loop that the whole warp runs, with
// their issue alone under elect(), lets the compiler keep descriptors and
// addresses there.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Shared-memory matrix descriptors (version 1). Operands: K-major rows of 128
// bytes, 128-byte swizzle, groups of 8 rows 1024 bytes apart. Scales: units of
// 32 rows x 16 bytes, no swizzle, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(128 >> 4) << 32) |
           (1ull << 46);
}

// Instruction descriptor of the block-scaled 4-bit kinds: E2M1 operands, both
// K-major, dense, K = 64; scale type e4m3 (0) or e8m0 (1); the byte of a
// scale cell where A's and B's scales start (0 or 2).
__device__ __forceinline__ uint32_t idesc(uint32_t m, uint32_t n, bool e8m0) {
    return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) | ((m >> 7) << 27);
}
__device__ __forceinline__ uint32_t idesc_scale_byte(uint32_t byte) { return (byte << 4) | (byte << 29); }

// D[tmem] (+)= (A * scales) (B * scales)^T over 64 columns; A, B in shared
// memory, scales in tensor memory.
template <int kCtas, bool NV>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t sa, uint32_t sb,
                                    uint32_t accumulate) {
#define MQ_TC5_MMA(GROUP, KIND, VEC)                                                                     \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                       \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND ".block_scale.scale_vec::" VEC           \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                      \
                 "l"(a), "l"(b), "r"(desc), "r"(sa), "r"(sb), "r"(accumulate)                            \
                 : "memory")
    if constexpr (kCtas == 2) {
        if constexpr (NV)
            MQ_TC5_MMA("2", "mxf4nvf4", "4X");
        else
            MQ_TC5_MMA("2", "mxf4", "2X");
    } else {
        if constexpr (NV)
            MQ_TC5_MMA("1", "mxf4nvf4", "4X");
        else
            MQ_TC5_MMA("1", "mxf4", "2X");
    }
#undef MQ_TC5_MMA
}

// One unit of scales (128 rows x 4 bytes, 512 bytes) from shared memory to
// four columns of tensor memory, repeated in each quarter of the lanes.
template <int kCtas>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (kCtas == 2)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Arrives on `bar` when every MMA and copy this thread issued is done.
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// The same for a pair, on the barrier at this offset in both CTAs.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<unsigned short>(3))
        : "memory");
}

// 32 lanes x 16 columns of 32-bit values: thread i gets lane (base + i). The
// values are there after load_wait.
__device__ __forceinline__ void load16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

}  // namespace tc5
}  // namespace mq
