// attn_tc.cuh -- tensor-core pieces of the attention kernels beside tc.cuh: tiles brought in by
// TMA with the 128-byte swizzle, their matrix descriptors, MMAs whose A operand lies in tensor
// memory, and TMEM moves of packed bf16.
//
// A tile of R rows x D columns (bf16) is D / 64 slabs of R rows x 128 bytes, each on a 1024-byte
// boundary, as TMA's SWIZZLE_128B writes them: 16-byte piece c of row r at r * 128 + ((c ^ (r & 7))
// << 4).  Read along the columns (K-major) an MMA's 16 columns are 32 bytes of a slab; read along
// the rows (MN-major, M or N = the tile's columns) its 16 rows are two 8-row groups of 1024 bytes.
#pragma once

#include <cuda.h>

#include "tc.cuh"

namespace gdn {
namespace tc {

constexpr uint64_t kDescSwizzle128 = (uint64_t)2 << 61;

// K-major: M or N = rows; 8-row groups 1024 bytes apart (the leading offset is not used)
__device__ __forceinline__ uint64_t desc_k_sw128(uint32_t saddr) {
  return make_desc(saddr, 16, 1024) | kDescSwizzle128;
}
// MN-major: M or N = columns; slabs of 64 columns `slab` bytes apart, 8-row groups 1024
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t slab) {
  return make_desc(saddr, slab, 1024) | kDescSwizzle128;
}

// D (+)= A B^T with A [128 x 16 K] packed bf16 pairs in TMEM
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D = A B^T over D columns, A and B row tiles (K-major); RA, RB rows
template <int COLS, int RA, int RB>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < COLS / 16; ++kk)
    mma_bf16(d, desc_k_sw128(a + (kk / 4) * RA * 128 + (kk % 4) * 32),
             desc_k_sw128(b + (kk / 4) * RB * 128 + (kk % 4) * 32), idesc, kk > 0);
}
// D (+)= P B, P [128 x RB] in TMEM, B a tile of RB rows (K) read MN-major
template <int RB>
__device__ __forceinline__ void mma_ts_cols(uint32_t d, uint32_t p, uint32_t b, uint32_t idesc, bool accumulate) {
#pragma unroll
  for (int kk = 0; kk < RB / 16; ++kk)
    mma_bf16_ts(d, p + kk * 8, desc_mn_sw128(b + kk * 2048, RB * 128), idesc, (accumulate || kk > 0) ? 1u : 0u);
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Box of a [T, H, D] tensor map: 64 columns from `col`, one head, the map's rows from `row`.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int col, int head, int row,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(col), "r"(head), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

// Warp: 16 packed words into 16 consecutive columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Warpgroup: registers per thread from here on (the groups' shares add up to at most the launch's)
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}

}  // namespace tc

// Host: tensor map of a packed [T, H, d] bf16 tensor whose boxes are 64 columns x one head x
// `rows` rows in the 128-byte swizzle; rows past T read as zeros.  False if it cannot be made.
bool make_rows_map(CUtensorMap* map, const void* base, int T, int H, int d, int rows);

}  // namespace gdn
