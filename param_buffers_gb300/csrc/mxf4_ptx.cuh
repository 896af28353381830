// What the MXFP4 products need of PTX beyond sm100_ptx.cuh: the kind::mxf4 MMA of a CTA pair, its
// instruction descriptor, and a 3-D tensor copy.
#pragma once
#include "sm100_ptx.cuh"

namespace gtp {
namespace ptx {

// The cluster's barrier without the release of its arrival, which waits for a memory fence (about 600 cycles even when
// nothing is outstanding).  It orders execution alone: barrier inits have their own fence (fence_barrier_init), and
// whoever uses it at the end of a kernel has seen every remote operation complete by other means.
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// tma_load_2d_pair of a 3-D tensor.
__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap *map, uint32_t bar_cluster_addr, void *dst,
                                                 int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// D[tmem] (+)= (A * 2^sA) (B * 2^sB)^T, packed E2M1 x E2M1, one E8M0 scale per 32 K elements: two
// bytes per row and instruction (K = 64), bytes 0-1 or 2-3 of each 32-bit scale word by sf_id.
__device__ __forceinline__ void mma_mxf4_block_scale_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                          uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::mxf4: as idesc_nvf4_e2m1 with E8M0 scales (bit 23) and the
// first of the instruction's two scale bytes (0 or 2) in both scale-byte fields.
__host__ __device__ constexpr uint32_t idesc_mxf4_e2m1(int M, int N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (1u << 23) | (uint32_t(M >> 4) << 24) |
         (sf_id << 29);
}

}  // namespace ptx
}  // namespace gtp
