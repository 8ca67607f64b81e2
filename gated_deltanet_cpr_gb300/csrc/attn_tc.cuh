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

// The products of the attention kernels.  Operands come as the descriptor of their tile's start; a
// step along K adds a constant to it (the address field counts 16 bytes and does not overflow), so
// that the one issuing thread spends two instructions per MMA on its operands.  Forming every
// descriptor from an address made that thread the bottleneck.
//
// D = A B^T over COLS columns, A and B row tiles of RA and RB rows (K-major)
template <int COLS, int RA, int RB>
__device__ __forceinline__ void mma_rows(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < COLS / 16; ++kk)
    mma_bf16(d, a + ((kk / 4) * RA * 128 + (kk % 4) * 32) / 16, b + ((kk / 4) * RB * 128 + (kk % 4) * 32) / 16, idesc,
             kk > 0);
}
// D (+)= P B, P [128 x RB] in TMEM, B a tile of RB rows (K) read MN-major
template <int RB>
__device__ __forceinline__ void mma_ts_cols(uint32_t d, uint32_t p, uint64_t b, uint32_t idesc, bool accumulate) {
  mma_bf16_ts(d, p, b, idesc, accumulate ? 1u : 0u);
#pragma unroll
  for (int kk = 1; kk < RB / 16; ++kk) mma_bf16_ts(d, p + kk * 8, b + kk * 2048 / 16, idesc, 1u);
}

// One lane of a converged warp (the same one each time).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// A wait of the whole converged warp, whose result (and what follows) is uniform.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}
// After a wait gave up, before memory is given back: the copies announced on a barrier, in whichever
// phase they are, and (whole warp) the MMAs that this warp has issued; each with a limit of its own.
__device__ __forceinline__ void settle(uint64_t* bar) {
  mbar_wait(bar, 0, 1u << 10);
  mbar_wait(bar, 1, 1u << 10);
}
__device__ __forceinline__ void settle_mma(uint64_t* unused) {
  __syncwarp();
  if (elect_one()) mma_commit(unused);
  mbar_wait(unused, 0, 1u << 12);
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

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

// Test hook, all threads of a CTA: the warp with `load` starts the copy of the map's first box, of
// `bytes`, on `full`, and all wait for a phase of `unused` that nothing completes.  False: they gave up.
__device__ __forceinline__ bool wait_for_nothing(const CUtensorMap* map, void* box, uint32_t bytes, uint64_t* full,
                                                 uint64_t* unused, bool load) {
  if (load && elect_one()) {
    mbar_expect_tx(full, bytes);
    tma_load_3d(box, map, 0, 0, 0, full);
  }
  return mbar_wait(unused, 0, 1u << 10);
}

// Warp: 128 consecutive fp32 columns of this thread's TMEM lane in one load, waited for
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float* v) {
  uint32_t r[128];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]),"=r"(r[1]),"=r"(r[2]),"=r"(r[3]),"=r"(r[4]),"=r"(r[5]),"=r"(r[6]),"=r"(r[7]),
        "=r"(r[8]),"=r"(r[9]),"=r"(r[10]),"=r"(r[11]),"=r"(r[12]),"=r"(r[13]),"=r"(r[14]),"=r"(r[15]),
        "=r"(r[16]),"=r"(r[17]),"=r"(r[18]),"=r"(r[19]),"=r"(r[20]),"=r"(r[21]),"=r"(r[22]),"=r"(r[23]),
        "=r"(r[24]),"=r"(r[25]),"=r"(r[26]),"=r"(r[27]),"=r"(r[28]),"=r"(r[29]),"=r"(r[30]),"=r"(r[31]),
        "=r"(r[32]),"=r"(r[33]),"=r"(r[34]),"=r"(r[35]),"=r"(r[36]),"=r"(r[37]),"=r"(r[38]),"=r"(r[39]),
        "=r"(r[40]),"=r"(r[41]),"=r"(r[42]),"=r"(r[43]),"=r"(r[44]),"=r"(r[45]),"=r"(r[46]),"=r"(r[47]),
        "=r"(r[48]),"=r"(r[49]),"=r"(r[50]),"=r"(r[51]),"=r"(r[52]),"=r"(r[53]),"=r"(r[54]),"=r"(r[55]),
        "=r"(r[56]),"=r"(r[57]),"=r"(r[58]),"=r"(r[59]),"=r"(r[60]),"=r"(r[61]),"=r"(r[62]),"=r"(r[63]),
        "=r"(r[64]),"=r"(r[65]),"=r"(r[66]),"=r"(r[67]),"=r"(r[68]),"=r"(r[69]),"=r"(r[70]),"=r"(r[71]),
        "=r"(r[72]),"=r"(r[73]),"=r"(r[74]),"=r"(r[75]),"=r"(r[76]),"=r"(r[77]),"=r"(r[78]),"=r"(r[79]),
        "=r"(r[80]),"=r"(r[81]),"=r"(r[82]),"=r"(r[83]),"=r"(r[84]),"=r"(r[85]),"=r"(r[86]),"=r"(r[87]),
        "=r"(r[88]),"=r"(r[89]),"=r"(r[90]),"=r"(r[91]),"=r"(r[92]),"=r"(r[93]),"=r"(r[94]),"=r"(r[95]),
        "=r"(r[96]),"=r"(r[97]),"=r"(r[98]),"=r"(r[99]),"=r"(r[100]),"=r"(r[101]),"=r"(r[102]),"=r"(r[103]),
        "=r"(r[104]),"=r"(r[105]),"=r"(r[106]),"=r"(r[107]),"=r"(r[108]),"=r"(r[109]),"=r"(r[110]),"=r"(r[111]),
        "=r"(r[112]),"=r"(r[113]),"=r"(r[114]),"=r"(r[115]),"=r"(r[116]),"=r"(r[117]),"=r"(r[118]),"=r"(r[119]),
        "=r"(r[120]),"=r"(r[121]),"=r"(r[122]),"=r"(r[123]),"=r"(r[124]),"=r"(r[125]),"=r"(r[126]),"=r"(r[127])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(r[i]);
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
// `rows` rows in the 128-byte swizzle; rows past T read as zeros.  False if it cannot be made.  An
// empty tensor, of which nothing is ever loaded, gets a map of one row of `any`.
bool make_rows_map(CUtensorMap* map, const void* base, int T, int H, int d, int rows, const void* any);

}  // namespace gdn
