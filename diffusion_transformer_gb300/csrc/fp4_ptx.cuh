// Inline-PTX building blocks of the 4-bit product beside those of ptx.cuh: clusters, the block-scaled
// tcgen05 MMA with its scales, packed fp32 products. Written from the public PTX ISA description.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace dit {

// TMA box of a 3-D map whose completion is counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Every thread of the cluster arrives and waits: what the CTAs did before is visible to one another,
// and none is past it while another is not yet there.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_shared_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// 32 TMEM lanes x 16 consecutive columns (see tmem_ld32).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// d = a * b, lane by lane, each product rounded by itself.
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// ------------------------------------------------------------------------------------------
// Block-scaled MMA of e2m1 operands: D += sum over blocks of sa sb (codes_a . codes_b), K = 64 per
// instruction, operands packed two codes per byte. The scales are read from tensor memory: a 512-byte
// chunk (32 rows of 16 bytes, row r holding the four consecutive scale bytes of operand rows r, r + 32,
// r + 64 and r + 96) is copied by tcgen05.cp to four columns, once per 32-lane quadrant. Issued by one
// thread, tcgen05.cp and tcgen05.mma run in issue order.
// ------------------------------------------------------------------------------------------
template <bool PAIR>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (PAIR)  // each CTA of the pair copies from its own shared memory to its own tensor memory
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
#define DIT_UMMA_FP4(GROUP, KIND)                                                              \
  asm volatile(                                                                                \
      "{\n"                                                                                    \
      ".reg .pred P;\n"                                                                        \
      "setp.ne.b32 P, %4, 0;\n"                                                                \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%5], [%6], P;\n"      \
      "}\n" ::"r"(d_tmem),                                                                     \
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)      \
      : "memory")
// NV: four e4m3 scales per row and instruction; otherwise two e8m0 scales (the instruction
// descriptor's scale ids say which half of the four bytes).
template <bool NV, bool PAIR>
__device__ __forceinline__ void umma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  if constexpr (NV && PAIR) DIT_UMMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
  else if constexpr (NV) DIT_UMMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
  else if constexpr (PAIR) DIT_UMMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
  else DIT_UMMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
}
#undef DIT_UMMA_FP4

// Instruction descriptor of the block-scaled 4-bit kinds: bits 4-5 B scale id, 7-9 / 10-12 A / B format
// (1 = e2m1), 17-22 N >> 3, 23 scale type (0 = e4m3, 1 = e8m0), 24-28 M >> 4, 29-30 A scale id.
__host__ __device__ constexpr uint32_t idesc_fp4(bool nv, int M, int N, uint32_t scale_id) {
  return (scale_id << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (nv ? 0u : 1u << 23) |
         (uint32_t(M >> 4) << 24) | (scale_id << 29);
}

// Shared-memory descriptor of a scale chunk: no swizzle, 8-row groups of 16-byte rows 128 bytes apart
// (one such group wide, so the leading byte offset is unused).
__device__ __forceinline__ uint64_t scale_chunk_desc(uint32_t saddr) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
}

}  // namespace dit
