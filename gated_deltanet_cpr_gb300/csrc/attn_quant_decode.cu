// attn_quant_decode.cu -- attention of one new token per request over the 8-bit cache.
//
// The formulas are those of attn_decode.cu, with k = c s and v = c s where a block is held in codes c with a
// scale s, and the rows as they came in the tail.  Everything is counted in granules of 16 consecutive keys: a
// granule's rows are contiguous in its page and share their scales.
//
// One warp takes a run of granules of one key head for up to 16 query heads.  The products run on warp-level MMAs
// in f16 with the keys as rows (scores^T = K q^T, out^T += V^T P^T), so that up to 8 heads cost one column tile and nothing
// is computed for heads that are not there.  Codes are exact in f16: int8 as 1024 + (c + 128), less 1152;
// e4m3 by conversion.  q is scaled by a power of two so that its largest entry lies in [2^14, 2^15), P by 2^14, so that f16
// holds them with 11 bits down to 2^-28 of the largest; fp32 calls split both into two f16, 22 bits.  P's 2^14 is in the
// operand alone and goes with the codes or their scale: put into what is taken off a score, it would be lost where
// fp32 has no such bits (scores of 2^25 and more), and leave rounding of its own in any other.  Scales multiply the
// scores, and the sums of one granule's 16 values, in fp32.
//
// Half the bytes of a bf16 cache leave half the time for the same products, so that instructions bound this kernel
// where DRAM bounds attn_decode.cu: widening a code to f16 is 2.5 of them a pair of codes in int8 (1 to 1.5 in e4m3) and a
// third of all.  256 requests of about 2112 tokens, 32 / 8 heads, d = 128: 194 us in int8, 191 in e4m3, where the bytes take 167
// and 169 at a copy's rate (bf16 pages: 325).  Scores as rows of the MMA (16 heads, of which 4 are there) took 220.  Few
// requests are bound by the chain of one run, launch and join: 4 of about 700 tokens take 10.3 us.
#include <cuda_fp16.h>

#include "attn_decode.cuh"
#include "attn_quant.h"

namespace gdn {

namespace {

constexpr float kUpP = 0x1p14f, kDownP = 0x1p-14f;  // probabilities are p 2^14 in f16
constexpr float kLowest = -3.402823466e38f;         // the maximum before any score: no score is less, and taken off it stays finite

// Sums of p v are held times 2^-s, 2^s being above twice the request's length: they and their runs' cannot overflow, whatever
// the values are (a mean of finite values is finite, their sum need not be).  Scales carry it, so that it costs a product a
// granule; it is exact for values of 2^-100, the least that a block holds as more than zeros, up to 262144 tokens.
__device__ __forceinline__ float sums_down(int len) { return __uint_as_float((uint32_t)(127 - (33 - __clz(len))) << 23); }

// What a warp needs to know of a request.
struct QuantRequest {
  int len;         // tokens (0 if the length is not valid)
  int n;           // granules with visible keys
  int head, skip;  // granule of number u: u < head ? u : u + skip
  bool bad;
  __device__ __forceinline__ QuantRequest(const QuantDecode& a, int length) {
    len = length;
    bad = len < 0 || len > a.max_len;
    if (bad) len = 0;
    n = (int)(((uint32_t)len + kGranule - 1) >> kGranuleShift);
    head = skip = 0;
    if (a.window > 0 && len > a.window) {
      const int first = (len - a.window) >> kGranuleShift;
      head = min((min(a.sinks, len) + kGranule - 1) >> kGranuleShift, first);
      skip = first - head;
      n -= skip;
    }
  }
  __device__ __forceinline__ int granule(int u) const { return u < head ? u : u + skip; }
  __device__ __forceinline__ int runs(const QuantDecode& a) const { return quant_split(n, a.hkv).runs; }
};

// A run as the computing side needs it; bad: a page or the slot is outside the cache.
struct QuantRun {
  int i, y, run, runs, len, slot, bad;
};

struct Quant {
  using Kind = Quant;
  using Args = QuantDecode;
  using Request = QuantRequest;
  using Run = QuantRun;
  // a page of the request's visible whole blocks, or its tail's slot, is outside the cache
  __device__ __forceinline__ static int check(const QuantDecode& a, const QuantRequest& rq, int i, int tid, int threads) {
    if (!rq.n) return 0;
    int wrong = 0;
    const int held = (rq.len >> a.c.block_shift) << a.c.block_shift;  // keys in pages
    if (tid == 0 && held < rq.len) {  // the last key is always visible
      const int slot = a.slot ? a.slot[i] : i;
      if (slot < 0 || slot >= a.c.slots) wrong = GDN_DEVERR_SLOT;
    }
    if (held) {
      const int last = (held - 1) >> a.page_shift;  // pages [0, head) and [first, last]
      const int first = (rq.granule(rq.head) << kGranuleShift) >> a.page_shift;
      const int head = rq.head ? min((((rq.head << kGranuleShift) - 1) >> a.page_shift), last) + 1 : 0;
      const int count = head + max(0, last - first + 1);
      for (int b = tid; b < count; b += threads) {
        const int p = b < head ? b : first + b - head;
        const int page = p < a.max_blocks ? a.block_table[(int64_t)i * a.max_blocks + p] : -1;
        if (page < 0 || page >= a.c.num_pages) wrong = GDN_DEVERR_PAGES;
      }
    }
    return wrong;
  }
  // what the sums of p v are divided by
  __device__ __forceinline__ static float divisor(const QuantRequest& rq, float l) { return __fmul_rn(l, sums_down(rq.len)); }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same with nothing to add to
__device__ __forceinline__ void mma_f16_from0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// an 8 x 8 matrix of pairs, transposed over the warp
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// four 8 x 8 matrices at addr + OFF
template <bool TRANS, int OFF>
__device__ __forceinline__ void load_matrices(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFF)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFF)
                 : "memory");
}
// 16 bytes at gmem + G to smem + S
template <int S, int G>
__device__ __forceinline__ void copy16(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(smem), "l"(gmem), "n"(S), "n"(G) : "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 x = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}
// the part of (lo, hi) that pack_f16 lost
__device__ __forceinline__ uint32_t pack_f16_rest(float lo, float hi, uint32_t packed) {
  const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&packed));
  return pack_f16(__fsub_rn(lo, p.x), __fsub_rn(hi, p.y));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}
// 2^e
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// For values of largest magnitude m: e so that they times 2^-e stay below 2^15 and the largest reaches 2^14 (unless
// it is below 2^-110).
__device__ __forceinline__ int f16_exponent(float m) { return max((int)(__float_as_uint(m) >> 23) - 127, -110) - 14; }

// Two pairs of f16 from four codes: of keys' codes (0, 1) and (2, 3), or of VALUES' (0, 2) and (1, 3).  Values in int8 come
// times 2^-14, which is exact: as 2^-4 + (c + 128) 2^-14, less 2^-4 + 2^-7.
template <bool E4M3, bool VALUES>
__device__ __forceinline__ void widen16(uint32_t four, uint32_t& first, uint32_t& second) {
  if constexpr (E4M3) {
    if constexpr (VALUES) four = __byte_perm(four, 0u, 0x3120);
    asm("{.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(first), "=r"(second)
        : "r"(four));
  } else {
    const uint32_t u = four ^ 0x80808080u;
    const uint32_t high = VALUES ? 0x2c2c2c2cu : 0x64646464u;
    const uint32_t a = __byte_perm(u, high, VALUES ? 0x4240 : 0x4140);
    const uint32_t b = __byte_perm(u, high, VALUES ? 0x4341 : 0x4342);
    const float off = VALUES ? 1152.f * kDownP : 1152.f;
    const __half2 bias = __floats2half2_rn(off, off);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias), y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    first = *reinterpret_cast<const uint32_t*>(&x);
    second = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// ------------------------------------------------------------------------- engine ----
// A tile is up to T granules of the pages, or up to TAIL_ROWS rows of a granule of the tail.  NH column tiles of 8 heads.
// Lane (g, t) = (lane / 4, lane % 4) holds of scores^T keys g, g + 8 of a granule for heads 2 t, 2 t + 1, of out^T columns
// 16 j + 2 g, + 1 for them.  The MMAs' inner order is free as long as both operands agree: k-steps of 16 take columns 16 s +
// 4 t .. + 3 of lane t, so that a lane's four codes of a row are one register of a matrix load.
template <int D, typename T_, int NH, bool E4M3>
struct QuantEngine : Quant {
  using Elem = T_;
  static constexpr int DIM = D, ROWB = D, TAILB = D * (int)sizeof(Elem);  // bytes of a row
  static constexpr bool SPLIT = sizeof(Elem) == 4;                        // two f16 for q, P and the tail's rows
  static constexpr int T = 256 / D;
  static constexpr int SIDE = T * kGranule * ROWB;  // bytes of a tile's keys, or of its values
  static constexpr int TAIL_ROWS = SIDE / TAILB < kGranule ? SIDE / TAILB : kGranule;
  static constexpr int STAGE = 2 * SIDE + 128, EXTRA = 0;
  // of a tile, behind its rows
  struct Meta {
    float ks[T], vs[T];  // scales of its granules
    alignas(16) int key; // first key of its first granule, or of its rows in the tail
    int what;            // granules in the pages, 0: rows of the tail; + kLast, + kEdge
    int skip;            // granules whose number is skip_from or more lie `skip` keys further on
    int skip_from;
  };
  static_assert(sizeof(Meta) <= 128 && (2 * SIDE) % 128 == 0 && STAGE % 128 == 0, "key is stored with the three behind it, 16 bytes");
  static constexpr int kLast = 64, kEdge = 128;  // the run's last tile; some keys may not be visible
  // Granules are gone through one by one: the instructions of two at a time (197 us for 256 requests of about 2112 tokens
  // against 194, fp32 window case 32.1 against 26.7) overflow the nearest cache.  Two column tiles need more registers than 12
  // warps leave, and go in pairs: with d = 64 these 256 requests take 111.5 us with 12 heads a key head, one by one 115.6 (e4m3
  // 106.3 and 110.8); with d = 128, where a pair is a whole tile, 33 requests of 500 to 15619 take 49.2 either way, but 256 of
  // about 2112 with 16 heads a key head 165.7 against 152.7.  12 warps with a tile on its way take the first 256 requests in
  // 194 us, 8 with two 207, 16 with tiles of one granule 209 (of 193 then).
  static constexpr bool PAIRS = NH == 2 && !SPLIT;
  static constexpr int MOST_WARPS = NH == 2 ? 8 : 12, RING = NH == 2 ? 3 : 2;
  static_assert(RING <= 3, "the queue holds four runs: the computed one, those of RING - 1 tiles ahead and the next");
  static constexpr int KS = D / 16, P = 1 + SPLIT;  // steps, parts of a split value

  uint32_t q[P][KS][NH][2];
  float qs[NH][2];  // scale of the scores
  float m[NH][2], l[NH][2], o[KS][NH][4];
  float down;  // o is held times this

  // place of 16-byte piece c of row r: 8 rows of a matrix load lie in 8 bank groups
  __device__ __forceinline__ static uint32_t place(int r, int c) {
    constexpr int PER = 128 / ROWB;  // rows in 128 bytes
    return r * ROWB + ((c ^ ((r / PER) & (ROWB / 16 - 1))) << 4);
  }
  __device__ __forceinline__ static uint32_t place_tail(int r, int c) {
    constexpr int PIECES = TAILB / 16, PER = TAILB < 128 ? 128 / TAILB : 1, MASK = PIECES < 8 ? PIECES - 1 : 7;
    return r * TAILB + ((c ^ ((r / PER) & MASK)) << 4);
  }

  __device__ __forceinline__ void start(const QuantDecode& a, int64_t row, int heads, int len, int lane) {
    down = sums_down(len);
    const int g = lane >> 2, t = lane & 3;
    const float scale = __fmul_rn(a.scale, kLog2e);
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      float x[KS][4], mx = 0.f;
      bool odd = false;
      const Elem* src = static_cast<const Elem*>(a.q) + (row + g + 8 * h) * D + 4 * t;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const float4 v = g + 8 * h < heads ? load4(src + 16 * s) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[s][0] = v.x, x[s][1] = v.y, x[s][2] = v.z, x[s][3] = v.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mx = fmaxf(mx, fabsf(x[s][e]));
          odd |= !(fabsf(x[s][e]) < INFINITY);
        }
      }
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const uint32_t which = __ballot_sync(0xffffffffu, odd);
      const bool any = (which >> (4 * g)) & 15u;  // an infinity or a NaN in this head's row
      const int e = any ? 0 : f16_exponent(mx);
      const float by = pow2(-e), f = any ? __builtin_nanf("") : __fmul_rn(scale, pow2(e));
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float lo = any ? 0.f : __fmul_rn(x[s][2 * b], by), hi = any ? 0.f : __fmul_rn(x[s][2 * b + 1], by);
          q[0][s][h][b] = pack_f16(lo, hi);
          if constexpr (SPLIT) q[1][s][h][b] = pack_f16_rest(lo, hi, q[0][s][h][b]);
        }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        qs[h][b] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + b));
        m[h][b] = kLowest;
        l[h][b] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][h][e] = 0.f;
  }

  // Products of a granule's keys, whose scale is ks, to scores.
  __device__ __forceinline__ void scores(float ks, float (&x)[NH][4]) const {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const float f[2] = {__fmul_rn(ks, qs[h][0]), __fmul_rn(ks, qs[h][1])};
#pragma unroll
      for (int e = 0; e < 4; ++e) x[h][e] = __fmul_rn(x[h][e], f[e & 1]);
    }
  }
  // Scores x of G granules, the first `rows` of each from key[i] on, to probabilities, with the running maximum and sum.
  template <int G>
  __device__ __forceinline__ void softmax(const QuantDecode& a, bool full, const int (&key)[G], int rows, int len,
                                          float (&x)[G][NH][4], int lane) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (!full) {  // some may not be visible
        const int lo = a.window > 0 ? len - a.window : 0;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const int r = (lane >> 2) + 4 * e, k = key[i] + r;
          if (r < rows && k < len && (k >= lo || k < a.sinks)) continue;
#pragma unroll
          for (int h = 0; h < NH; ++h) x[i][h][e] = x[i][h][e + 1] = -INFINITY;
        }
      }
    }
    float mx[NH][2];
    bool more = false;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[h][e] = fmaxf(x[0][h][e], x[0][h][e + 2]);
#pragma unroll
        for (int i = 1; i < G; ++i) mx[h][e] = fmaxf(mx[h][e], fmaxf(x[i][h][e], x[i][h][e + 2]));
        more |= mx[h][e] > m[h][e];
      }
    if (__any_sync(0xffffffffu, more)) {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = mx[h][e];
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, w));
          y = fmaxf(y, m[h][e]);
          f[e] = exp2_approx(__fsub_rn(m[h][e], y));
          m[h][e] = y;
          l[h][e] = __fmul_rn(l[h][e], f[e]);
        }
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][h][e] = __fmul_rn(o[j][h][e], f[e & 1]);
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
          x[i][h][e] = exp2_approx(__fsub_rn(x[i][h][e], m[h][e]));
          x[i][h][e + 2] = exp2_approx(__fsub_rn(x[i][h][e + 2], m[h][e]));
          l[h][e] = __fadd_rn(l[h][e], __fadd_rn(x[i][h][e], x[i][h][e + 2]));
        }
      }
  }
  // P^T 2^14 of a granule as the MMA's right operand: keys 2 t, 2 t + 1 (+ 8) of head g
  __device__ __forceinline__ static void operand(const float (&p)[4], uint32_t (&b)[P][2]) {
    const float2 up = make_float2(kUpP, kUpP), x = mul2(make_float2(p[0], p[1]), up), y = mul2(make_float2(p[2], p[3]), up);
    const uint32_t lo = pack_f16(x.x, x.y), hi = pack_f16(y.x, y.y);
    b[0][0] = transposed(lo);
    b[0][1] = transposed(hi);
    if constexpr (SPLIT) {
      b[P - 1][0] = transposed(pack_f16_rest(x.x, x.y, lo));
      b[P - 1][1] = transposed(pack_f16_rest(y.x, y.y, hi));
    }
  }
  __device__ __forceinline__ void add(int j, int h, const float (&c)[4], float scale) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][h][e] = __fmaf_rn(c[e], scale, o[j][h][e]);
  }

  // Granules i .. i + G - 1 of the tile, in the pages.
  template <int G>
  __device__ __forceinline__ void granules(const QuantDecode& a, const unsigned char* stage, int i, bool full, int len, int lane) {
    const Meta& meta = *reinterpret_cast<const Meta*>(stage + 2 * SIDE);
    // this lane's row for matrix loads (keys 0 .. 7 and 8 .. 15) and, s steps on, its piece (0 and 1 of a pair): the
    // swizzle turns bits, and a stage begins at a multiple of 128 bytes
    const uint32_t at = tc::smem_u32(stage) + i * (kGranule * ROWB) + place((lane & 7) + (lane & 8), lane >> 4);
    uint32_t r[G][KS / 2][4];
    // sums of even and odd steps; of fp32 queries' upper and lower parts: the products' own sums are cut, not rounded, so only
    // those of the lower part, 2^-11 of the other's size, run through all steps
    float x[G][NH][4], y[G][NH][4];
    load_all<G, false, 0>(at, r);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int b = 0; b < G; ++b) {
        uint32_t k[4];
        widen16<E4M3, false>(r[b][s / 2][2 * (s & 1)], k[0], k[2]);
        widen16<E4M3, false>(r[b][s / 2][2 * (s & 1) + 1], k[1], k[3]);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          if constexpr (SPLIT) {
            add_step(x[b][h], y[b][h], s, k, h);
          } else {
            float(&c)[4] = s & 1 ? y[b][h] : x[b][h];
            if (s < 2) mma_f16_from0(c, k, q[0][s][h][0], q[0][s][h][1]);
            else mma_f16(c, k, q[0][s][h][0], q[0][s][h][1]);
          }
        }
      }
    load_all<G, true, SIDE>(at, r);
    float vs[G];
    int key[G];
#pragma unroll
    for (int b = 0; b < G; ++b) {
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[b][h][e] = __fadd_rn(x[b][h][e], y[b][h][e]);
      scores(meta.ks[i + b], x[b]);
      vs[b] = __fmul_rn(meta.vs[i + b], E4M3 ? __fmul_rn(down, kDownP) : down);
      key[b] = meta.key + ((i + b) << kGranuleShift) + (i + b >= meta.skip_from ? meta.skip : 0);
    }
    softmax<G>(a, full, key, kGranule, len, x, lane);
    uint32_t p[G][NH][P][2];
#pragma unroll
    for (int b = 0; b < G; ++b)
#pragma unroll
      for (int h = 0; h < NH; ++h) operand(x[b][h], p[b][h]);
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int b = 0; b < G; ++b) {
        uint32_t v[4];
        widen16<E4M3, true>(r[b][j / 2][2 * (j & 1)], v[0], v[1]);
        widen16<E4M3, true>(r[b][j / 2][2 * (j & 1) + 1], v[2], v[3]);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          float c[4];
          mma_f16_from0(c, v, p[b][h][0][0], p[b][h][0][1]);
          if constexpr (SPLIT) {
            float rest[4];
            mma_f16_from0(rest, v, p[b][h][P - 1][0], p[b][h][P - 1][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = __fadd_rn(c[e], rest[e]);
          }
          add(j, h, c, vs[b]);
        }
      }
  }
  // fp32 queries: step s of keys k for head tile h, upper part to x, lower part to y
  __device__ __forceinline__ void add_step(float (&x)[4], float (&y)[4], int s, const uint32_t (&k)[4], int h) const {
    float c[4];
    mma_f16_from0(c, k, q[0][s][h][0], q[0][s][h][1]);
    if (s == 0) mma_f16_from0(y, k, q[P - 1][s][h][0], q[P - 1][s][h][1]);
    else mma_f16(y, k, q[P - 1][s][h][0], q[P - 1][s][h][1]);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = s == 0 ? c[e] : __fadd_rn(x[e], c[e]);
  }
  template <int G, bool TRANS, int OFF>
  __device__ __forceinline__ static void load_all(uint32_t at, uint32_t (&r)[G][KS / 2][4]) {
#pragma unroll
    for (int s = 0; s < KS / 2; ++s) {
      load_matrices<TRANS, OFF>(at ^ (uint32_t)(s << 5), r[0][s]);
      if constexpr (G == 2) load_matrices<TRANS, OFF + kGranule * ROWB>(at ^ (uint32_t)(s << 5), r[1][s]);
    }
  }

  // Keys key .. key + TAIL_ROWS - 1 of the tail.  bf16 rows are operands as they are, with the rows of q (read again: scaled
  // to f16's range they would overflow with keys of 2^106) and with P as the sum of two bf16.
  __device__ __forceinline__ void tail_bf16(const QuantDecode& a, const unsigned char* stage, int key, int len, int64_t row,
                                            int heads, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const float scale = __fmul_rn(a.scale, kLog2e);
    float xs[1][NH][4];
    float(&x)[NH][4] = xs[0];
    const Elem* src = static_cast<const Elem*>(a.q) + (row + g) * D + 4 * t;
    uint32_t odd = 0;  // an exponent of ones in either half carries into its upper bit
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint32_t k[4] = {0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < TAIL_ROWS / 8; ++r) {
        const int at = (16 * s + 4 * t) * 2;
        const uint2 u = *reinterpret_cast<const uint2*>(stage + place_tail(g + 8 * r, at >> 4) + (at & 15));
        k[r] = u.x;
        k[r + 2] = u.y;
        odd |= ((u.x & 0x7fff7fffu) + 0x00800080u) | ((u.y & 0x7fff7fffu) + 0x00800080u);
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        uint2 u = make_uint2(0u, 0u);
        if (g + 8 * h < heads) u = *reinterpret_cast<const uint2*>(src + (8 * h) * D + 16 * s);
        if (s == 0) x[h][0] = x[h][1] = x[h][2] = x[h][3] = 0.f;
        tc::mma16816(x[h], k, u.x, u.y);
      }
    }
    // a key that is not finite gives NaN, not a weight of 0, and so does a query
    const float by = __any_sync(0xffffffffu, odd & 0x80008000u) ? __builtin_nanf("") : scale;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[h][e] = __fmul_rn(x[h][e], qs[h][e & 1] == qs[h][e & 1] ? by : qs[h][e & 1]);
    softmax<1>(a, false, {key}, TAIL_ROWS, len, xs, lane);
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[h][e] = __fmul_rn(x[h][e], down);
    uint32_t b[NH][2][2];
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t hi = pack_bf16(x[h][2 * r], x[h][2 * r + 1]);
        b[h][0][r] = transposed(hi);
        b[h][1][r] = transposed(pack_bf16(__fsub_rn(x[h][2 * r], __uint_as_float(hi << 16)),
                                          __fsub_rn(x[h][2 * r + 1], __uint_as_float(hi & 0xffff0000u))));
      }
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      uint32_t v[4] = {0, 0, 0, 0};
      const int at = (16 * j + 2 * g) * 2;
#pragma unroll
      for (int r = 0; r < TAIL_ROWS / 8; ++r) {  // keys 2 t, 2 t + 1 and those + 8
        const unsigned char* src = stage + SIDE + (at & 15);
        const uint32_t k0 = *reinterpret_cast<const uint32_t*>(src + place_tail(8 * r + 2 * t, at >> 4));
        const uint32_t k1 = *reinterpret_cast<const uint32_t*>(src + place_tail(8 * r + 2 * t + 1, at >> 4));
        v[2 * r] = __byte_perm(k0, k1, 0x5410);
        v[2 * r + 1] = __byte_perm(k0, k1, 0x7632);
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        tc::mma16816(o[j][h], v, b[h][0][0], b[h][0][1]);
        tc::mma16816(o[j][h], v, b[h][1][0], b[h][1][1]);
      }
    }
  }

  // f16_exponent of a row of A, from the bits of its four lanes' largest magnitudes.
  __device__ __forceinline__ static int row_exponent(uint32_t m) {
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return f16_exponent(__uint_as_float(m));
  }
  __device__ __forceinline__ static uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

  // The same of fp32 rows, as sums of two f16: a key's row is scaled by a power of two of its own, and so is a column of the
  // values, so that small ones beside large ones keep their bits.  An infinity's second part is NaN, so that all that it
  // would reach is.
  __device__ __forceinline__ void tail_f32(const QuantDecode& a, const unsigned char* stage, int key, int len, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float xs[1][NH][4], ys[NH][4], kd[2], ks[2];
    float(&x)[NH][4] = xs[0];
    auto row_of = [&](int r, int s) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (g + 8 * r < TAIL_ROWS) v = *reinterpret_cast<const float4*>(stage + place_tail(g + 8 * r, 4 * s + t));
      return v;
    };
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t most = 0;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const float4 v = row_of(r, s);
        most = max(max(max(most, magnitude(v.x)), max(magnitude(v.y), magnitude(v.z))), magnitude(v.w));
      }
      const int e = row_exponent(most);
      kd[r] = pow2(-e);
      ks[r] = pow2(e);
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint32_t k[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float4 v = row_of(r, s);
        const float y[4] = {__fmul_rn(v.x, kd[r]), __fmul_rn(v.y, kd[r]), __fmul_rn(v.z, kd[r]), __fmul_rn(v.w, kd[r])};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          k[0][r + 2 * b] = pack_f16(y[2 * b], y[2 * b + 1]);
          k[1][r + 2 * b] = pack_f16_rest(y[2 * b], y[2 * b + 1], k[0][r + 2 * b]);
        }
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        add_step(x[h], ys[h], s, k[0], h);
        mma_f16(ys[h], k[1], q[0][s][h][0], q[0][s][h][1]);
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[h][e] = __fmul_rn(__fadd_rn(x[h][e], ys[h][e]), __fmul_rn(ks[e >> 1], qs[h][e & 1]));
    softmax<1>(a, false, {key}, TAIL_ROWS, len, xs, lane);
    uint32_t b[NH][P][2];
#pragma unroll
    for (int h = 0; h < NH; ++h) operand(x[h], b[h]);
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      uint32_t v[2][4];
      const int at = (16 * j + 2 * g) * 4;
      float2 y[2][2];  // keys 2 t, 2 t + 1 and those + 8, of two columns
      uint32_t most[2] = {0, 0};
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int row = 8 * r + 2 * t + w;
          y[r][w] = make_float2(0.f, 0.f);
          if (row < TAIL_ROWS) y[r][w] = *reinterpret_cast<const float2*>(stage + SIDE + place_tail(row, at >> 4) + (at & 15));
          most[0] = max(most[0], magnitude(y[r][w].x));
          most[1] = max(most[1], magnitude(y[r][w].y));
        }
      float vd[2], vs[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int e = row_exponent(most[c]);
        vd[c] = pow2(-e);
        vs[c] = __fmul_rn(pow2(e), down);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 lo = make_float2(__fmul_rn(y[r][0].x, vd[0]), __fmul_rn(y[r][1].x, vd[0]));
        const float2 hi = make_float2(__fmul_rn(y[r][0].y, vd[1]), __fmul_rn(y[r][1].y, vd[1]));
        v[0][2 * r] = pack_f16(lo.x, lo.y);
        v[0][2 * r + 1] = pack_f16(hi.x, hi.y);
        v[1][2 * r] = pack_f16_rest(lo.x, lo.y, v[0][2 * r]);
        v[1][2 * r + 1] = pack_f16_rest(hi.x, hi.y, v[0][2 * r + 1]);
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float c[4], rest[4];
        mma_f16_from0(c, v[0], b[h][0][0], b[h][0][1]);
        mma_f16_from0(rest, v[0], b[h][P - 1][0], b[h][P - 1][1]);
        mma_f16(rest, v[1], b[h][0][0], b[h][0][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[j][h][e] = __fmaf_rn(__fmul_rn(__fadd_rn(c[e], rest[e]), kDownP), vs[e >> 1], o[j][h][e]);
      }
    }
  }

  __device__ __forceinline__ void finish(const Sink& k, bool bad, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = l[h][e];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, w));
        if (bad) s = __builtin_nanf("");
        const int head = 8 * h + 2 * t + e;
        if (head >= k.heads) continue;
        if (g == 0) k.stats(head, m[h][e], s);
        if (k.acc) {
          float* to = k.acc + head * k.acc_step + 2 * g;
#pragma unroll
          for (int j = 0; j < KS; ++j) *reinterpret_cast<float2*>(to + 16 * j) = make_float2(o[j][h][e], o[j][h][2 + e]);
        } else {
          Elem* to = static_cast<Elem*>(k.out) + head * D + 2 * g;
          const float f = __fdiv_rn(1.f, __fmul_rn(s, down));
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            const float y0 = __fmul_rn(o[j][h][e], f), y1 = __fmul_rn(o[j][h][2 + e], f);
            if constexpr (SPLIT) *reinterpret_cast<float2*>(to + 16 * j) = make_float2(y0, y1);
            else *reinterpret_cast<uint32_t*>(to + 16 * j) = pack_bf16(y0, y1);
          }
        }
      }
  }
};

// --------------------------------------------------------------------------- walk ----
// The fetching side of a warp: which run it takes, which tile comes next, and where its rows lie.  It leaves what the computing
// side needs to know beside the rows, so that only one of them walks, and keeps few values, as registers are short (38 instead of 19:
// 10% more instructions).
template <typename E>
struct QuantWalk {
  // (run, request, part) slots are numbered with the run slowest and dealt out in chunks of `chunk` <= 32 consecutive ones,
  // one per lane: the first by the warp's number, further ones from a counter, as runs differ in length and many slots
  // of short requests are empty.  A further chunk is asked for when the present run comes to its end, so that a warp on a
  // long one does not keep it from others, in two steps a tile apart (a number from the counter, then its requests' lengths).
  uint32_t total, chunk;
  int32_t* counter;
  enum { kNone, kAsked, kKnown } more;
  uint32_t slot_no;  // this lane's of the chunk (total or more: none), or lane 0's number from the counter
  int len, slot;     // its request's length and tail
  uint32_t left;     // lanes of the chunk whose runs are still to come
  // the run being fetched: granules [u, end), those from `tail` on in its tail; only granules edge - 1 and edge of the others
  // can hold keys that are not visible; granule number x lies `skip` further on from `head` on; of key head h
  bool live;
  uint32_t u, end, tail, edge;
  int head, skip, h;
  uint32_t first;  // pages are looked up for 32 granules at once, one a lane: those from this one on
  int page;        // this lane's
  int sub;         // rows of the tail's granule that earlier tiles took

  __device__ __forceinline__ int granule(uint32_t x) const { return (int)x < head ? (int)x : (int)x + skip; }

  __device__ __forceinline__ void look_ahead(const QuantDecode& a, int parts, uint32_t base, int lane) {
    slot_no = lane < (int)chunk ? base + (uint32_t)lane : total;
    more = kKnown;
    if (slot_no >= total) return;
    const uint32_t ny = (uint32_t)(a.hkv * parts);
    const int i = (int)(slot_no % ((uint32_t)a.N * ny) / ny);
    len = a.seq_lens[i];
    slot = a.slot ? a.slot[i] : i;
  }
  __device__ __forceinline__ void prepare(const QuantDecode& a, int parts, int lane) {
    if (more == kNone) {
      if (counter && lane == 0) slot_no = (uint32_t)atomicAdd(counter, 1);
      more = kAsked;
    } else if (more == kAsked) {
      const uint32_t n = __shfl_sync(0xffffffffu, slot_no, 0);
      look_ahead(a, parts, counter ? (gridDim.x * DecodeSmem<E>::WARPS + n) * chunk : total, lane);
    }
  }
  __device__ __forceinline__ void look_up(const QuantDecode& a, int lane, const QuantRun& r) {
    first = u;
    page = 0;
    if (u + lane >= min(end, tail)) return;
    const int b = (int)(((uint32_t)granule(u + lane) << kGranuleShift) >> a.page_shift);
    page = b < a.max_blocks ? a.block_table[(int64_t)r.i * a.max_blocks + b] : -1;
  }
  // The first run, or the next one: to the queue, which holds at most the computed one, those of RING - 1 tiles ahead and
  // this.  Requests without keys have their rows written here.
  __device__ void next_run(const QuantDecode& a, int parts, int lane, QuantRun* queue, int& put) {
    live = false;
    const uint32_t ny = (uint32_t)(a.hkv * parts), rows = (uint32_t)a.N * ny;
    while (!left) {
      while (more != kKnown) prepare(a, parts, lane);
      if (__shfl_sync(0xffffffffu, slot_no, 0) >= total) return;
      bool have = false;
      if (slot_no < total) {
        const QuantRequest rq(a, len);
        const int run = (int)(slot_no / rows), runs = rq.runs(a);
        have = run < runs;
        if (runs == 0 && run == 0) write_empty(a, (int)(slot_no % rows / ny), (int)(slot_no % ny), parts, rq.bad);
      }
      left = __ballot_sync(0xffffffffu, have);
      more = kNone;
    }
    const int src = __ffs(left) - 1;
    left &= left - 1;
    const uint32_t w = __shfl_sync(0xffffffffu, slot_no, src);
    QuantRun r;
    r.run = (int)(w / rows);
    r.i = (int)(w % rows / ny);
    r.y = (int)(w % ny);
    r.len = __shfl_sync(0xffffffffu, len, src);
    r.slot = __shfl_sync(0xffffffffu, slot, src);
    r.bad = 0;
    const QuantRequest rq(a, r.len);
    const Split s = quant_split(rq.n, a.hkv);
    r.runs = s.runs;
    live = true;
    u = (uint32_t)r.run * (uint32_t)s.keys;
    end = min((uint32_t)rq.n, u + (uint32_t)s.keys);
    head = rq.head;
    skip = rq.skip;
    edge = a.window > 0 && r.len > a.window ? (uint32_t)head : 1u << 30;
    const int g = (r.len >> a.c.block_shift) << (a.c.block_shift - kGranuleShift);  // first granule of the tail
    tail = (uint32_t)(g <= head ? g : max(head, g - skip));
    h = r.y / parts;
    sub = 0;
    if (lane == 0) queue[put & 3] = r;
    ++put;
    look_up(a, lane, r);
    const int group = a.hq / a.hkv, g0 = (r.y % parts) * kHeadsPerRun, heads = min(kHeadsPerRun, group - g0);
    constexpr int ROW = E::DIM * (int)sizeof(typename E::Elem);
    const char* q = static_cast<const char*>(a.q) + ((int64_t)r.i * a.hq + h * group + g0) * ROW;
    for (int e = lane * 128; e < heads * ROW; e += 32 * 128) tc::prefetch_l2(q + e);
    __syncwarp();
  }
  // zeros for a request without keys, NaN for a length that is not valid; one lane
  __device__ static void write_empty(const QuantDecode& a, int i, int y, int parts, bool bad) {
    const int group = a.hq / a.hkv, g0 = (y % parts) * kHeadsPerRun, heads = min(kHeadsPerRun, group - g0);
    const int64_t row = (int64_t)i * a.hq + (y / parts) * group + g0;
    const float x = bad ? __builtin_nanf("") : 0.f;
    for (int e = 0; e < heads * E::DIM; e += 4)
      store4(static_cast<typename E::Elem*>(a.out) + row * E::DIM + e, make_float4(x, x, x, x));
    if (a.lse)
      for (int k = 0; k < heads; ++k) a.lse[row + k] = bad ? x : -INFINITY;
  }

  // The current tile into `stage`, then on to the next one.
  __device__ __forceinline__ void fetch(const QuantDecode& a, int parts, unsigned char* stage, int lane, QuantRun* queue, int& put) {
    if (live) {
      if (!left && end - u <= 3 * E::T) prepare(a, parts, lane);
      const uint32_t st = tc::smem_u32(stage);
      int key = granule(u) << kGranuleShift, what, skip_from = E::T;
      if (u < tail) {
        const uint32_t stop = min(end, tail);
        const int n = (int)min((uint32_t)E::T, stop - u);
        if (u - first + n > 32) look_up(a, lane, queue[(put - 1) & 3]);
        const bool lost = (uint32_t)page >= (uint32_t)a.c.num_pages && first + lane < stop;
        if (!__any_sync(0xffffffffu, lost)) {
          constexpr int PIECES = E::ROWB / 16;
          // where this lane's first piece of a granule goes; its next ones are 512 bytes on, in the same piece of rows 4
          // (d = 128: the swizzle's upper bit turns) or more further on
          const uint32_t dst = st + E::place(lane / PIECES, lane % PIECES);
          const uint32_t mask = (1u << a.page_shift) - 1u;
          uint32_t rows = 0;  // lane i: row of granule i in the pages
#pragma unroll
          for (int i = 0; i < E::T; ++i) {
            if (i >= n) break;
            const uint32_t at = (uint32_t)__shfl_sync(0xffffffffu, page, u - first + i) * (uint32_t)a.hkv + (uint32_t)h;
            const uint32_t row = (at << a.page_shift) + (((uint32_t)granule(u + i) << kGranuleShift) & mask);
            rows = lane % E::T == i ? row : rows;
            const int64_t off = (int64_t)row * E::ROWB + 16 * lane;
            const uint8_t *kp = a.c.k_pages + off, *vp = a.c.v_pages + off;
            const uint32_t to = dst + i * (kGranule * E::ROWB);
            copy16<0, 0>(to, kp);
            copy16<E::SIDE, 0>(to, vp);
            if constexpr (E::ROWB >= 64) {
              const uint32_t odd = E::ROWB == 128 ? to ^ 64u : to;
              copy16<512, 512>(odd, kp);
              copy16<E::SIDE + 512, 512>(odd, vp);
              if constexpr (E::ROWB == 128) {
                copy16<1024, 1024>(to, kp);
                copy16<E::SIDE + 1024, 1024>(to, vp);
                copy16<1536, 1536>(odd, kp);
                copy16<E::SIDE + 1536, 1536>(odd, vp);
              }
            }
          }
          // scales: lanes 0 .. T - 1 those of keys, T .. 2 T - 1 of values
          if (lane < 2 * E::T && lane % E::T < n)
            copy4(st + 2 * E::SIDE + 4 * lane, (lane < E::T ? a.c.k_scale : a.c.v_scale) + (rows >> a.c.block_shift));
        } else if (lane == 0) {
          queue[(put - 1) & 3].bad = 1;  // the tile holds what it held: the run's results are NaN
        }
        what = n + (u + (uint32_t)n - edge <= (uint32_t)n ? E::kEdge : 0);  // it holds granule edge - 1 or edge
        if (u < (uint32_t)head) skip_from = min(E::T, head - (int)u);
        u += n;
      } else {
        // only rows that are visible: what else the tail holds is nobody's
        const QuantRun& r = queue[(put - 1) & 3];
        const int n = r.len, B = 1 << a.c.block_shift, lo = a.window > 0 ? n - a.window : 0;
        const bool lost = r.slot < 0 || r.slot >= a.c.slots;
        key += sub;
        const int64_t off = lost ? 0 : (((int64_t)r.slot * a.hkv + h) * B + (key & (B - 1))) * E::TAILB;
        constexpr int PIECES = E::TAIL_ROWS * E::TAILB / 16, PER = E::TAILB / 16;
#pragma unroll 4
        for (int p = lane; p < PIECES; p += 32) {
          const int k = key + p / PER;
          const bool load = !lost && k < n && (k >= lo || k < a.sinks);
          const uint32_t dst = st + E::place_tail(p / PER, p % PER);
          const int64_t from = load ? off + 16 * p : 0;
          cp_async16_or_zero(dst, static_cast<const char*>(a.c.k_tail) + from, load);
          cp_async16_or_zero(dst + E::SIDE, static_cast<const char*>(a.c.v_tail) + from, load);
        }
        if (lost && lane == 0) queue[(put - 1) & 3].bad = 1;
        what = 0;
        sub += E::TAIL_ROWS;
        if (sub == kGranule || key + E::TAIL_ROWS >= n) sub = 0, ++u;
      }
      if (lane == 0) {
        typename E::Meta& meta = *reinterpret_cast<typename E::Meta*>(stage + 2 * E::SIDE);
        *reinterpret_cast<int4*>(&meta.key) =
            make_int4(key, what + (u >= end ? E::kLast : 0), skip << kGranuleShift, skip_from);
      }
      if (u >= end) next_run(a, parts, lane, queue, put);
    }
    tc::cp_async_commit();
  }
  __device__ __forceinline__ static void copy4(uint32_t smem, const void* gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem), "l"(gmem) : "memory");
  }
};

template <typename E>
__global__ void __launch_bounds__(32 * DecodeSmem<E>::WARPS, 1) k_quant_decode(const QuantDecode a, const int parts, const uint32_t chunk, int32_t* counter) {
  using L = DecodeSmem<E>;
  extern __shared__ __align__(128) unsigned char all[];
  unsigned char* sh = all + (threadIdx.x >> 5) * L::WARP;
  asm volatile("griddepcontrol.launch_dependents;");  // the join kernel may get ready
  const int lane = threadIdx.x & 31, group = a.hq / a.hkv;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->err = 0;  // set by the join kernel
  QuantRun* queue = reinterpret_cast<QuantRun*>(sh + L::QUEUE);
  QuantWalk<E> f;
  f.total = (uint32_t)(a.N * a.hkv * parts * a.max_splits);
  f.chunk = chunk;
  f.counter = counter;
  f.left = 0;
  int head = 0, tail = 0, put = 0, get = 0;
  f.look_ahead(a, parts, ((threadIdx.x >> 5) * gridDim.x + blockIdx.x) * chunk, lane);
  if (counter) asm volatile("griddepcontrol.wait;" ::: "memory");  // it has been cleared
  f.next_run(a, parts, lane, queue, tail);
#pragma unroll 1
  for (int s = 0; s < E::RING - 1; ++s) {
    f.fetch(a, parts, sh + put * L::STAGE, lane, queue, tail);
    put = put + 1 == E::RING ? 0 : put + 1;
  }
  E eng;
  while (head != tail) {
    __syncwarp();
    const QuantRun& r = queue[head & 3];
    const int len = r.len;
    {
      const int g0 = (r.y % parts) * kHeadsPerRun;
      eng.start(a, (int64_t)r.i * a.hq + (r.y / parts) * group + g0, min(kHeadsPerRun, group - g0), len, lane);
    }
    int what;
    do {
      // the next tile on its way first, into the place that every lane has read
      f.fetch(a, parts, sh + put * L::STAGE, lane, queue, tail);
      put = put + 1 == E::RING ? 0 : put + 1;
      asm volatile("cp.async.wait_group %0;" ::"n"(E::RING - 1) : "memory");
      __syncwarp();
      const unsigned char* stage = sh + get * L::STAGE;
      const typename E::Meta& meta = *reinterpret_cast<const typename E::Meta*>(stage + 2 * E::SIDE);
      what = meta.what;
      const int n = what & (E::kLast - 1);
      if (n) {
        const bool full = !(what & E::kEdge);
        int i = 0;
        if constexpr (E::PAIRS) {
#pragma unroll 1
          for (; i + 2 <= n; i += 2) eng.template granules<2>(a, stage, i, full, len, lane);
          if (i < n) eng.template granules<1>(a, stage, i, full, len, lane);
        } else {
#pragma unroll 1
          for (; i < n; ++i) eng.template granules<1>(a, stage, i, full, len, lane);
        }
      } else {
        if constexpr (E::SPLIT) eng.tail_f32(a, stage, meta.key, len, lane);
        else {
          const int g0 = (r.y % parts) * kHeadsPerRun;
          eng.tail_bf16(a, stage, meta.key, len, (int64_t)r.i * a.hq + (r.y / parts) * group + g0, min(kHeadsPerRun, group - g0), lane);
        }
      }
      get = get + 1 == E::RING ? 0 : get + 1;
      __syncwarp();
    } while (!(what & E::kLast));
    const int g0 = (r.y % parts) * kHeadsPerRun, heads = min(kHeadsPerRun, group - g0);
    eng.finish(Sink(a, r, (r.y / parts) * group + g0, heads, sizeof(typename E::Elem)), r.bad != 0, lane);
    ++head;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, typename T, int NH>
int decode_h(const QuantDecode& a, cudaStream_t st) {
  using I = QuantEngine<D, T, NH, false>;
  using F = QuantEngine<D, T, NH, true>;
  return a.c.e4m3 ? launch_decode<F>(k_quant_decode<F>, a, st) : launch_decode<I>(k_quant_decode<I>, a, st);
}

template <int D, typename T>
int decode_t(const QuantDecode& a, cudaStream_t st) {
  return a.hq / a.hkv <= 8 ? decode_h<D, T, 1>(a, st) : decode_h<D, T, 2>(a, st);
}

template <typename T>
int decode(const QuantDecode& a, cudaStream_t st) {
  if (a.d == 32) return decode_t<32, T>(a, st);
  if (a.d == 64) return decode_t<64, T>(a, st);
  return decode_t<128, T>(a, st);
}

}  // namespace

// A bound on the runs of any request of that many granules or fewer: quant_target grows with them between the counts
// where quant_shift changes, and a request has at most quant_target runs.
int quant_max_splits(int64_t granules, int hkv) {
  int best = 1;
  for (int s = kQuantMinShift; s <= kQuantMaxShift; ++s) {
    const int64_t last = s < kQuantMaxShift ? (((int64_t)kQuantRuns << (s + 1)) - 1) / hkv : granules;
    const int n = (int)(last < granules ? last : granules);
    if (n > 0 && quant_target(n, hkv) > best) best = quant_target(n, hkv);
  }
  return best;
}

int launch_quant_decode(const QuantDecode& a, bool bf16, cudaStream_t st) {
  return bf16 ? decode<__nv_bfloat16>(a, st) : decode<float>(a, st);
}

}  // namespace gdn
