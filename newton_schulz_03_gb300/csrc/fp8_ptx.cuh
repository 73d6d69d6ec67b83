// fp8_ptx.cuh -- inline-PTX wrappers of the FP8 products, beside those of
// sm103_ptx.cuh: block-scaled MMA, scales to tensor memory, lane election,
// arrivals without a cluster-wide release, stores with a cache policy.
#pragma once

#include <cstdint>

#include "sm103_ptx.cuh"

namespace muon {
namespace ptx {

// True in one lane of a converged warp, the same one at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Arrive on either CTA's barrier without ordering this thread's memory accesses:
// for arrivals that only say that tensor memory has been read (a release at
// cluster scope takes some 1400 cycles while stores are in flight).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// L2 policy: first to be evicted (data that nothing reads again soon).
__device__ __forceinline__ uint64_t l2_evict_first() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}

__device__ __forceinline__ void tma_store_3d_hint(const void* tmap, const void* smem_src, int32_t x,
                                                  int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint"
      " [%0, {%2, %3, %4}], [%1], %5;" ::"l"(reinterpret_cast<uint64_t>(tmap)),
      "r"(smem_addr(smem_src)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// D[tmem] (+)= (A * 2^sa) * (B * 2^sb) for a CTA pair: 8-bit floats, one E8M0
// scale per row of A (column of B) and 32 K values, scales in TMEM.
__device__ __forceinline__ void tc_mma_mxf8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t sa_tmem,
                                                 uint32_t sb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
      : "memory");
}

// 32 rows x 16 bytes from shared memory (each CTA's own) to four TMEM columns
// of both CTAs of the pair, repeated in every 32-lane quarter: the layout of
// 128 rows' scales.  Executes in order with this thread's MMAs.
__device__ __forceinline__ void tc_copy_scales_pair(uint32_t taddr, uint64_t s_desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(s_desc)
               : "memory");
}

// TMA store of a 3-D FP32 box that adds to what is there.
__device__ __forceinline__ void tma_reduce_add_3d(const void* tmap, const void* smem_src,
                                                  int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}],"
      " [%1];" ::"l"(reinterpret_cast<uint64_t>(tmap)),
      "r"(smem_addr(smem_src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Shared-memory descriptor of 8-row x 16-byte core matrices without swizzle,
// 128 bytes from one to the next (the scales' layout).
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (8ull << 32) | (1ull << 46);
}

// Instruction descriptor for kind::mxf8f6f4 with e4m3 A and B (both K-major),
// E8M0 scales, scale byte 0 of each 32-bit TMEM cell; and with byte `b`.
__host__ __device__ constexpr uint32_t idesc_mxf8(uint32_t M, uint32_t N) {
  return ((N >> 3) << 17)     // N / 8
         | (1u << 23)         // scale type: E8M0
         | ((M >> 4) << 24);  // M / 16
}
__host__ __device__ constexpr uint32_t idesc_mxf8_byte(uint32_t idesc, uint32_t b) {
  return idesc | (b << 4) | (b << 29);
}

}  // namespace ptx
}  // namespace muon
