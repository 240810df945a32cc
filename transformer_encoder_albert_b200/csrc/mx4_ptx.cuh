// mx4_ptx.cuh -- inline-PTX wrappers of the block-scaled E2M1 products (tcgen05.mma
// kind::mxf4 / mxf4nvf4, tcgen05.cp of their scales).  Written from the public PTX ISA.
#pragma once
#include "sm100_ptx.cuh"

namespace albert {

// Products of microscaled E2M1 operands, K = 64 per instruction (32 bytes of a
// K-major row): every block of A and B is multiplied by its scale, read from
// tensor memory.  NV: blocks of 16 with E4M3 scales, four per row and instruction;
// else blocks of 32 with E8M0 scales, two (the descriptor's scale ids pick the
// lower or the upper two bytes of a scale word).
//
// These forms are executed by a whole warp in step and take effect in the one lane
// whose `leader` (from elect_leader) is set: outside a divergent branch the operands
// stay in uniform registers.  Issued by one lane inside a branch, a scale copy cost
// its thread about 60 cycles and a product about 106.
__device__ __forceinline__ uint32_t elect_leader() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
template <bool NV, bool PAIR>
__device__ __forceinline__ void umma_mx4(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
#define ALBERT_UMMA_MX4(group, kind)                                                                      \
    asm volatile(                                                                                         \
        "{\n\t.reg .pred p, q;\n\t"                                                                       \
        "setp.ne.b32 p, %6, 0;\n\t"                                                                       \
        "setp.ne.b32 q, %7, 0;\n\t"                                                                       \
        "@q tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"        \
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate), \
          "r"(leader) : "memory")
    if constexpr (NV && PAIR) ALBERT_UMMA_MX4("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (NV) ALBERT_UMMA_MX4("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (PAIR) ALBERT_UMMA_MX4("2", "mxf4.block_scale.scale_vec::2X");
    else ALBERT_UMMA_MX4("1", "mxf4.block_scale.scale_vec::2X");
#undef ALBERT_UMMA_MX4
}

// Copies one 512-byte scale tile (32 rows of 16 bytes) from shared memory to four
// tensor-memory columns, repeated in the four 32-lane quadrants; pair form: each
// CTA's tile at this offset to its own tensor memory.  Products of another thread that read
// these columns wait for a commit behind it.
template <bool PAIR>
__device__ __forceinline__ void tmem_cp_scales(uint32_t leader, uint32_t taddr, uint64_t s_desc) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                     "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(s_desc), "r"(leader) : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                     "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(s_desc), "r"(leader) : "memory");
}

// umma_commit / umma_commit_pair (sm100_ptx.cuh) of the elected lane.
template <bool PAIR>
__device__ __forceinline__ void umma_commit_elected(uint32_t leader, uint32_t bar, uint16_t cta_mask) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                     "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
                     ::"r"(bar), "h"(cta_mask), "r"(leader) : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                     "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                     ::"r"(bar), "r"(leader) : "memory");
}

// tma_load_2d / tma_load_2d_pair (sm100_ptx.cuh) of the elected lane.
template <bool PAIR>
__device__ __forceinline__ void tma_load_elected(uint32_t leader, uint32_t dst, const void *tmap, uint32_t bar, int x, int y) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                     "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4}], [%2];\n\t}"
                     ::"r"(dst), "l"(tmap), "r"(bar), "r"(x), "r"(y), "r"(leader) : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                     "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4}], [%2];\n\t}"
                     ::"r"(dst), "l"(tmap), "r"(bar), "r"(x), "r"(y), "r"(leader) : "memory");
}

// Shared-memory descriptor of a scale tile: rows of 16 bytes, no swizzle, 8-row
// groups 128 bytes apart (fields as in sw128_kmajor_desc).
__device__ __forceinline__ uint64_t scale_tile_desc(uint32_t smem_addr) {
    return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(128u >> 4) << 32) |
           ((uint64_t)1u << 46);
}

// Instruction descriptor of the block-scaled E2M1 products: A and B E2M1 (format 1
// in bits 7-9 and 10-11), K-major, N >> 3 at bits 17-22, scale type at bit 23 (1 =
// E8M0, 0 = E4M3), M >> 7 at bits 27-28; which bytes of a scale word apply: bits 4-5
// (B) and 29-30 (A).
template <bool NV>
__host__ __device__ constexpr uint32_t idesc_mx4(int M, int N, int sf_id) {
    return ((uint32_t)sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((NV ? 0u : 1u) << 23) |
           ((uint32_t)(M >> 7) << 27) | ((uint32_t)sf_id << 29);
}

}  // namespace albert
