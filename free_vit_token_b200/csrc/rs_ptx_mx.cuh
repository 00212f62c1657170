// rs_ptx_mx.cuh -- inline-PTX wrappers of the 8-bit product beside those of rs_ptx.cuh: the
// block-scaled tcgen05.mma, scale tiles to TMEM, their descriptors, and issue by one elected
// lane of a converged warp.
#pragma once

#include <cstdint>

#include "rs_ptx.cuh"

namespace rs {

// True in one lane of a converged warp, the same one every time. Code that the whole warp runs,
// with only the tcgen05 and TMA instructions under this predicate, keeps their operands in
// uniform registers; under `lane == 0` each of them is assembled lane by lane.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}
// wait_bounded by every lane of a converged warp, with one answer for all of them.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& w,
                                          bool honor_abort = true, bool cluster = false) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, w, honor_abort, cluster)) != 0;
}

// 3-D tiled load of a CTA pair (see tma_load_2d_pair).
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t x, int32_t y,
                                                 int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Block-scaled form (kind::mxf8f6f4, one E8M0 scale per row and 32 K elements): D (+)= A B^T
// with the scale bytes of A's rows at `sa` and of B's rows at `sb` in TMEM, the byte of each
// 32-bit word chosen by the instruction descriptor. One thread issues.
__device__ __forceinline__ void umma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_mx_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t sa, uint32_t sb,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
// A scale tile (32 rows of 16 bytes in shared memory) into 4 TMEM columns, repeated in each
// quarter of the lanes; ordered before the MMAs that this thread issues after it. The pair
// form copies each CTA's own tile (same shared-memory offset) into its own TMEM.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// Shared-memory matrix descriptor of a scale tile: 32 rows of 16 bytes without a swizzle,
// 8-row groups 128 bytes apart (the only stride this shape has).
__device__ __forceinline__ uint64_t scale_tile_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}

// Instruction descriptor of kind::mxf8f6f4: e4m3 A and B (0), both K-major, E8M0 scales
// (bit 23), N>>3 at 17-22, M>>4 at 24-28; the scale byte of each 32-bit word at 29-30 (A)
// and 4-5 (B).
__host__ __device__ constexpr uint32_t idesc_mx_e4m3(int m, int n) {
  return (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_mx_byte(uint32_t idesc, uint32_t b) {
  return idesc | (b << 29) | (b << 4);
}

}  // namespace rs
