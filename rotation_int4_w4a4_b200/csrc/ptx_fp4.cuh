// Instructions of the 4-bit floating-point product beside those of ptx.cuh (sm_100a): block-scaled products, copies of their
// scales into tensor memory, tiled stores.
#pragma once

#include "ptx.cuh"

namespace pq {
namespace ptx {

// Instruction descriptor for block-scaled E2M1 operands (kind::mxf4nvf4, kind::mxf4), both K-major, float32 accumulator: A/B
// formats bits 7-9 / 10-11 (1 = E2M1), scale type bit 23 (0 = E4M3, 1 = E8M0), N/8 at bit 17, M/128 at bit 27, and which
// bytes of a scale word the instruction takes (sf: 0, or 2 for the second pair of two) at bits 4-5 (B) and 29-30 (A).
__host__ __device__ constexpr uint32_t idesc_e2m1(bool e8m0, int M, int N, int sf) {
  return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) |
         ((uint32_t)(M >> 7) << 27) | ((uint32_t)sf << 29);
}

// D (+)= (A * scale_A) (B * scale_B)^T on E2M1 operands, 64 codes along K; a_scale, b_scale: tensor-memory columns of
// scale words (rows = lanes, 32 rows a column, in all four lane quarters).  NV: a word holds four E4M3 scales of 16 codes;
// otherwise two pairs of E8M0 scales of 32 codes.  PAIR: M = 256 over a CTA pair.
template <bool NV, bool PAIR>
__device__ __forceinline__ void umma_e2m1(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t a_scale,
                                          uint32_t b_scale, uint32_t accumulate) {
#define PQ_UMMA_E2M1(GROUP, KIND)                                                            \
  asm volatile(                                                                              \
      "{\n\t.reg .pred p;\n\t"                                                               \
      "setp.ne.b32 p, %6, 0;\n\t"                                                            \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem), \
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)      \
      : "memory")
  if constexpr (NV && PAIR) PQ_UMMA_E2M1("2", "mxf4nvf4.block_scale.scale_vec::4X");
  else if constexpr (NV) PQ_UMMA_E2M1("1", "mxf4nvf4.block_scale.scale_vec::4X");
  else if constexpr (PAIR) PQ_UMMA_E2M1("2", "mxf4.block_scale.scale_vec::2X");
  else PQ_UMMA_E2M1("1", "mxf4.block_scale.scale_vec::2X");
#undef PQ_UMMA_E2M1
}

// 512 bytes of shared memory, 32 rows of 16, to 4 columns of tensor memory, the same in all four lane quarters (PAIR: in
// both CTAs of the pair, each from its own shared memory at the same offset).
template <bool PAIR>
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Rows of 16 bytes one after the other, without a swizzle: groups of 8 rows 128 bytes apart (stride offset).
__device__ __forceinline__ uint64_t smem_desc_rows16(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(128 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// 2-D tiled store of this CTA's shared memory (written through the async proxy's fence); x innermost, nothing outside the
// tensor is written.  bulk_commit closes the thread's group of stores, bulk_wait_read waits until the groups' shared memory
// may be written again, bulk_wait until they are complete.
__device__ __forceinline__ void tma_store_2d(const void* tmap, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(tmap), "r"(x), "r"(y),
               "r"(smem_addr(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void sts_v4(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

}  // namespace ptx
}  // namespace pq
