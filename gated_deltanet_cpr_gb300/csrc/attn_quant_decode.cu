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
// holds them with 11 bits down to 2^-28 of the largest; fp32 calls split both into two f16, 22 bits.  Scales multiply the
// scores, and the sums of one granule's 16 values, in fp32.
#include <cuda_fp16.h>

#include "attn_decode.cuh"
#include "attn_quant.h"

namespace gdn {

namespace {

constexpr int kShiftP = 14;  // probabilities are held as p 2^14

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
  __device__ __forceinline__ Split split(const QuantDecode& a) const {
    const uint32_t keys = (uint32_t)n << kGranuleShift;
    return split_of(keys > 0x7fffffffu ? 0x7fffffff : (int)keys, a.hkv);
  }
  __device__ __forceinline__ int runs(const QuantDecode& a) const { return split(a).runs; }
};

struct QuantAhead {
  int len, slot;
  __device__ __forceinline__ void load(const QuantDecode& a, int i) {
    len = a.seq_lens[i];
    slot = a.slot ? a.slot[i] : i;
  }
};

// Granules [u, end) of request i, those from `tail` on in its tail; bad: a page or the slot is outside the cache.
struct QuantRun {
  int i, y, run, runs;
  uint32_t u, end, tail;
  int head, skip, len, slot, bad;
  __device__ __forceinline__ int granule(uint32_t x) const { return (int)x < head ? (int)x : (int)x + skip; }
  __device__ __forceinline__ void set(const QuantDecode& a, const QuantRequest& rq, const QuantAhead& ahead) {
    const Split s = rq.split(a);
    runs = s.runs;
    u = (uint32_t)run * (uint32_t)(s.keys >> kGranuleShift);
    end = min((uint32_t)rq.n, u + (uint32_t)(s.keys >> kGranuleShift));
    head = rq.head;
    skip = rq.skip;
    len = rq.len;
    slot = ahead.slot;
    const int g = (rq.len >> a.c.block_shift) << (a.c.block_shift - kGranuleShift);  // first granule of the tail
    tail = (uint32_t)(g <= head ? g : max(head, g - skip));
  }
  __device__ __forceinline__ void from(const QuantRun& o, int lane) {
    i = __shfl_sync(0xffffffffu, o.i, lane);
    y = __shfl_sync(0xffffffffu, o.y, lane);
    run = __shfl_sync(0xffffffffu, o.run, lane);
    runs = __shfl_sync(0xffffffffu, o.runs, lane);
    u = __shfl_sync(0xffffffffu, o.u, lane);
    end = __shfl_sync(0xffffffffu, o.end, lane);
    tail = __shfl_sync(0xffffffffu, o.tail, lane);
    head = __shfl_sync(0xffffffffu, o.head, lane);
    skip = __shfl_sync(0xffffffffu, o.skip, lane);
    len = __shfl_sync(0xffffffffu, o.len, lane);
    slot = __shfl_sync(0xffffffffu, o.slot, lane);
  }
};

struct Quant {
  using Kind = Quant;
  using Args = QuantDecode;
  using Request = QuantRequest;
  using Ahead = QuantAhead;
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
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of pairs, transposed over the warp
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
// 2^e
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// For values of largest magnitude m: e so that they times 2^-e stay below 2^15 and the largest reaches 2^14 (unless
// it is below 2^-110).
__device__ __forceinline__ int f16_exponent(float m) { return max((int)(__float_as_uint(m) >> 23) - 127, -110) - 14; }

// Two pairs of f16 from four codes: of codes (0, 1) and (2, 3), or, APART, of (0, 2) and (1, 3).
template <bool E4M3, bool APART>
__device__ __forceinline__ void widen16(uint32_t four, uint32_t& first, uint32_t& second) {
  if constexpr (E4M3) {
    if constexpr (APART) four = __byte_perm(four, 0u, 0x3120);
    asm("{.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(first), "=r"(second)
        : "r"(four));
  } else {
    const uint32_t u = four ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, APART ? 0x4240 : 0x4140);
    const uint32_t b = __byte_perm(u, 0x64646464u, APART ? 0x4341 : 0x4342);
    const __half2 bias = __floats2half2_rn(1152.f, 1152.f);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias), y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    first = *reinterpret_cast<const uint32_t*>(&x);
    second = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// ------------------------------------------------------------------------- engine ----
// A tile is up to T granules of the pages, or one of the tail.  NH column tiles of 8 heads.  Lane (g, t) = (lane / 4,
// lane % 4) holds of scores^T keys g, g + 8 of a granule for heads 2 t, 2 t + 1, of out^T columns 16 j + 2 g, + 1 for them.
// The MMAs' inner order is free as long as both operands agree: k-steps of 16 take columns 16 s + 4 t .. + 3 of lane t, so
// that a lane's four codes of a row are one register of a matrix load.
template <int D, typename T_, int NH, bool E4M3>
struct QuantEngine : Quant {
  using Elem = T_;
  static constexpr int DIM = D, ROWB = D, TAILB = D * (int)sizeof(Elem);  // bytes of a row
  static constexpr bool SPLIT = sizeof(Elem) == 4;                        // two f16 for q, P and the tail's rows
  static constexpr int T = D == 128 && !SPLIT ? 2 : 4;
  static constexpr int ROWS = T * kGranule, SIDE = ROWS * ROWB;  // keys of a tile and the bytes of them, or of their values
  static constexpr int META = 2 * SIDE, STAGE = META + 128, RING = 2, EXTRA = 0;
  static constexpr bool MANY_REGS = SPLIT && NH == 2;
  static_assert(kGranule * TAILB <= SIDE, "a granule of the tail fits a tile");
  // of a tile: granules, whether it is of the tail, first keys, scales
  struct Meta {
    int count, tail;
    int key[T];
    float ks[T], vs[T];
  };
  static_assert(sizeof(Meta) <= 128, "");
  static constexpr int KS = D / 16, P = 1 + SPLIT;  // steps, parts of a split value

  uint32_t q[P][KS][NH][2];
  float qs[NH][2];  // scale of the scores
  float m[NH][2], l[NH][2], o[D / 16][NH][4];

  // place of 16-byte piece c of row r: 8 rows of a matrix load lie in 8 bank groups
  __device__ __forceinline__ static uint32_t place(int r, int c) {
    constexpr int PER = 128 / ROWB;  // rows in 128 bytes
    return r * ROWB + ((c ^ ((r / PER) & (ROWB / 16 - 1))) << 4);
  }
  __device__ __forceinline__ static uint32_t place_tail(int r, int c) {
    constexpr int PIECES = TAILB / 16, PER = TAILB < 128 ? 128 / TAILB : 1, MASK = PIECES < 8 ? PIECES - 1 : 7;
    return r * TAILB + ((c ^ ((r / PER) & MASK)) << 4);
  }

  __device__ __forceinline__ void start(const QuantDecode& a, int64_t row, int heads, int lane) {
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
      const float down = pow2(-e), f = any ? __builtin_nanf("") : __fmul_rn(scale, pow2(e));
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float lo = any ? 0.f : __fmul_rn(x[s][2 * b], down), hi = any ? 0.f : __fmul_rn(x[s][2 * b + 1], down);
          q[0][s][h][b] = pack_f16(lo, hi);
          if constexpr (SPLIT) q[1][s][h][b] = pack_f16_rest(lo, hi, q[0][s][h][b]);
        }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        qs[h][b] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + b));
        m[h][b] = -INFINITY;
        l[h][b] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][h][e] = 0.f;
  }

  // Scores of G granules (of which `count` are there) to probabilities p 2^14, with the running maximum and sum.
  // x: products; on return the probabilities.
  template <int G>
  __device__ __forceinline__ void softmax(const QuantDecode& a, const Meta& meta, int count, int len, float (&x)[G][NH][4], int lane) {
    float mx[NH][2];
#pragma unroll
    for (int h = 0; h < NH; ++h) mx[h][0] = mx[h][1] = -INFINITY;
    const int lo = a.window > 0 ? len - a.window : 0;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int key = meta.key[i];
      const float ks = meta.ks[i];
      // all keys of the granule visible, as in all but a few
      const bool full = i < count && key + (kGranule - 1) < len && (key >= lo || key + kGranule <= a.sinks);
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[i][h][e] = __fmul_rn(x[i][h][e], __fmul_rn(ks, qs[h][e & 1]));
          if (!full) {
            const int k = key + (lane >> 2) + 8 * (e >> 1);
            if (i >= count || k >= len || (k < lo && k >= a.sinks)) x[i][h][e] = -INFINITY;
          }
          mx[h][e & 1] = fmaxf(mx[h][e & 1], x[i][h][e]);
        }
    }
    bool more = false;
#pragma unroll
    for (int h = 0; h < NH; ++h) more |= mx[h][0] > m[h][0] || mx[h][1] > m[h][1];
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
          f[e] = m[h][e] == -INFINITY ? 0.f : exp2_approx(__fsub_rn(m[h][e], y));
          m[h][e] = y;
          l[h][e] = __fmul_rn(l[h][e], f[e]);
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][h][e] = __fmul_rn(o[j][h][e], f[e & 1]);
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float base = m[h][e] == -INFINITY ? 0.f : __fsub_rn(m[h][e], (float)kShiftP);
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
          for (int b = e; b < 4; b += 2) {
            x[i][h][b] = exp2_approx(__fsub_rn(x[i][h][b], base));
            l[h][e] = __fadd_rn(l[h][e], x[i][h][b]);
          }
      }
  }
  // P^T of a granule as the MMA's right operand: keys 2 t, 2 t + 1 (+ 8) of head g
  __device__ __forceinline__ static void operand(const float (&p)[4], uint32_t (&b)[P][2]) {
    const uint32_t lo = pack_f16(p[0], p[1]), hi = pack_f16(p[2], p[3]);
    b[0][0] = transposed(lo);
    b[0][1] = transposed(hi);
    if constexpr (SPLIT) {
      b[1][0] = transposed(pack_f16_rest(p[0], p[1], lo));
      b[1][1] = transposed(pack_f16_rest(p[2], p[3], hi));
    }
  }
  __device__ __forceinline__ void add(int j, int h, const float (&c)[4], float scale) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][h][e] = __fmaf_rn(c[e], scale, o[j][h][e]);
  }

  __device__ __forceinline__ void tile(const QuantDecode& a, const unsigned char* stage, int len, int lane) {
    const Meta& meta = *reinterpret_cast<const Meta*>(stage + META);
    const int count = meta.count;
    const uint32_t st = tc::smem_u32(stage);
    // matrix-load addresses: keys 0 .. 7 and 8 .. 15 of a granule, piece 0 and 1 of a pair
    const int kr = (lane & 7) + (lane & 8), kc = lane >> 4;
    float x[T][NH][4];
#pragma unroll
    for (int i = 0; i < T; ++i) {
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][h][e] = 0.f;
      if (i >= count) continue;
#pragma unroll
      for (int s = 0; s < KS; s += 2) {
        uint32_t r[4];
        tc::ldsm_x4(st + place(kGranule * i + kr, s + kc), r);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t k[4];
          widen16<E4M3, false>(r[2 * w], k[0], k[2]);
          widen16<E4M3, false>(r[2 * w + 1], k[1], k[3]);
#pragma unroll
          for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int p = 0; p < P; ++p) mma_f16(x[i][h], k, q[p][s + w][h][0], q[p][s + w][h][1]);
        }
      }
    }
    softmax<T>(a, meta, count, len, x, lane);
#pragma unroll
    for (int i = 0; i < T; ++i) {
      if (i >= count) continue;
      uint32_t b[NH][P][2];
#pragma unroll
      for (int h = 0; h < NH; ++h) operand(x[i][h], b[h]);
      const float vs = meta.vs[i];
#pragma unroll
      for (int j = 0; j < KS; j += 2) {
        uint32_t r[4];
        tc::ldsm_x4_trans(st + SIDE + place(kGranule * i + kr, j + kc), r);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t v[4];
          widen16<E4M3, true>(r[2 * w], v[0], v[1]);
          widen16<E4M3, true>(r[2 * w + 1], v[2], v[3]);
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < P; ++p) mma_f16(c, v, b[h][p][0], b[h][p][1]);
            add(j + w, h, c, vs);
          }
        }
      }
    }
  }

  // Largest magnitude of a granule of the tail: NaN where one of them is not finite.
  __device__ __forceinline__ static float tail_max(const unsigned char* side, int lane) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kGranule * TAILB / 512; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(side + 512 * i + 16 * lane);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m = max(m, SPLIT ? w[e] & 0x7fffffffu : max((w[e] << 16) & 0x7fffffffu, w[e] & 0x7fff0000u));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    return m >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float(m);
  }

  // The same over one granule of the tail, whose keys and values are scaled by powers of two to f16.
  __device__ __forceinline__ void tail(const QuantDecode& a, unsigned char* stage, int len, int lane) {
    Meta& meta = *reinterpret_cast<Meta*>(stage + META);
    const int g = lane >> 2, t = lane & 3;
    const float km = tail_max(stage, lane), vm = tail_max(stage + SIDE, lane);
    const int ke = f16_exponent(km), ve = f16_exponent(vm);
    const float kd = km == km ? pow2(-ke) : 0.f, vd = vm == vm ? pow2(-ve) : 0.f;
    if (lane == 0) {
      meta.ks[0] = km == km ? pow2(ke) : km;
      meta.vs[0] = vm == vm ? pow2(ve) : vm;
    }
    __syncwarp();
    float x[1][NH][4];
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[0][h][e] = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint32_t k[P][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        constexpr int BYTES = 4 * (int)sizeof(Elem);
        const int at = (16 * s + 4 * t) * (int)sizeof(Elem);
        const float4 v =
            load4(reinterpret_cast<const Elem*>(stage + place_tail(g + 8 * r, at >> 4) + (BYTES < 16 ? at & 15 : 0)));
        const float y[4] = {scaled(v.x, kd), scaled(v.y, kd), scaled(v.z, kd), scaled(v.w, kd)};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          k[0][r + 2 * b] = pack_f16(y[2 * b], y[2 * b + 1]);
          if constexpr (SPLIT) k[P - 1][r + 2 * b] = pack_f16_rest(y[2 * b], y[2 * b + 1], k[0][r + 2 * b]);
        }
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        mma_f16(x[0][h], k[0], q[0][s][h][0], q[0][s][h][1]);
        if constexpr (SPLIT) {
          mma_f16(x[0][h], k[0], q[P - 1][s][h][0], q[P - 1][s][h][1]);
          mma_f16(x[0][h], k[P - 1], q[0][s][h][0], q[0][s][h][1]);
        }
      }
    }
    softmax<1>(a, meta, 1, len, x, lane);
    const float vs = meta.vs[0];
    uint32_t b[NH][P][2];
#pragma unroll
    for (int h = 0; h < NH; ++h) operand(x[0][h], b[h]);
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      uint32_t v[P][4];
      const int at = (16 * j + 2 * g) * (int)sizeof(Elem);
#pragma unroll
      for (int r = 0; r < 2; ++r) {  // keys 2 t, 2 t + 1 and those + 8
        float y[2][2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const Elem* src = reinterpret_cast<const Elem*>(stage + SIDE + place_tail(8 * r + 2 * t + w, at >> 4) + (at & 15));
          y[w][0] = scaled(to_f32(src[0]), vd);
          y[w][1] = scaled(to_f32(src[1]), vd);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          v[0][2 * r + c] = pack_f16(y[0][c], y[1][c]);
          if constexpr (SPLIT) v[P - 1][2 * r + c] = pack_f16_rest(y[0][c], y[1][c], v[0][2 * r + c]);
        }
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(c, v[0], b[h][0][0], b[h][0][1]);
        if constexpr (SPLIT) {
          mma_f16(c, v[0], b[h][P - 1][0], b[h][P - 1][1]);
          mma_f16(c, v[P - 1], b[h][0][0], b[h][0][1]);
        }
        add(j, h, c, vs);
      }
    }
  }
  // 0 where the granule is not finite: its scale says so
  __device__ __forceinline__ static float scaled(float x, float down) { return down == 0.f ? 0.f : __fmul_rn(x, down); }

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
        if (g == 0) k.stats(head, __fsub_rn(m[h][e], (float)kShiftP), s);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const int c = 16 * j + 2 * g;
          const float y0 = o[j][h][e], y1 = o[j][h][2 + e];
          if (k.acc) {
            *reinterpret_cast<float2*>(k.acc + head * k.acc_step + c) = make_float2(y0, y1);
          } else if constexpr (SPLIT) {
            *reinterpret_cast<float2*>(static_cast<float*>(k.out) + head * D + c) = make_float2(__fdiv_rn(y0, s), __fdiv_rn(y1, s));
          } else {
            *reinterpret_cast<__nv_bfloat162*>(static_cast<Elem*>(k.out) + head * D + c) =
                __floats2bfloat162_rn(__fdiv_rn(y0, s), __fdiv_rn(y1, s));
          }
        }
      }
  }
};

// --------------------------------------------------------------------------- walk ----
// The fetching side of a warp: which tile comes next, and where its rows lie.
template <typename E>
struct QuantWalk : Dealer<E> {
  using Dealer<E>::r;
  using Dealer<E>::live;
  using Dealer<E>::seek;
  using Dealer<E>::push;
  int page;  // lane < T: page of granule r.u + lane, on its way during the tile before

  __device__ __forceinline__ bool in_pages(int lane) const { return lane < E::T && r.u + lane < min(r.end, r.tail); }

  __device__ __forceinline__ void look_up(const QuantDecode& a, int lane) {
    page = -1;
    if (!live || !in_pages(lane)) return;
    const int b = (int)(((uint32_t)r.granule(r.u + lane) << kGranuleShift) >> a.page_shift);
    if (b < a.max_blocks) page = a.block_table[(int64_t)r.i * a.max_blocks + b];
  }

  // The current tile into `stage`, then on to the next one (its pages are looked up meanwhile).
  __device__ __forceinline__ void fetch(const QuantDecode& a, int parts, unsigned char* stage, int lane, QuantRun* queue, int& tail) {
    if (live) {
      const uint32_t st = tc::smem_u32(stage);
      typename E::Meta& meta = *reinterpret_cast<typename E::Meta*>(stage + E::META);
      const int h = r.y / parts;
      const bool waits = r.u >= r.tail;
      const int count = waits ? 1 : (int)min((uint32_t)E::T, min(r.end, r.tail) - r.u);
      const int key = r.granule(r.u + min(lane, count - 1)) << kGranuleShift;  // of this lane's granule
      if (lane < E::T) meta.key[lane] = key;
      if (lane == 0) meta.count = count, meta.tail = waits;
      bool lost = false;
      if (!waits) {
        uint32_t row = ~0u;  // of this lane's granule in the pages: none, or its page is outside the cache
        lost = lane < count && (page < 0 || page >= a.c.num_pages);
        if (lane < count && !lost)
          row = (uint32_t)((((int64_t)page * a.hkv + h) << a.page_shift) + (key & ((1 << a.page_shift) - 1)));
        if (lane < count) {
          if (lost) {
            meta.ks[lane] = meta.vs[lane] = 0.f;
          } else {
            tc::cp_async4(&meta.ks[lane], a.c.k_scale + (row >> a.c.block_shift));
            tc::cp_async4(&meta.vs[lane], a.c.v_scale + (row >> a.c.block_shift));
          }
        }
        constexpr int PIECES = kGranule * E::ROWB / 16;  // of a granule
#pragma unroll
        for (int i = 0; i < E::T; ++i) {
          if (i >= count) break;
          const uint32_t at = __shfl_sync(0xffffffffu, row, i);
          const bool load = at != ~0u;
          const int64_t off = load ? (int64_t)at * E::ROWB : 0;
#pragma unroll
          for (int p = lane; p < PIECES; p += 32) {
            const uint32_t dst = st + E::place(kGranule * i + p / (E::ROWB / 16), p % (E::ROWB / 16));
            cp_async16_or_zero(dst, a.c.k_pages + off + 16 * p, load);
            cp_async16_or_zero(dst + E::SIDE, a.c.v_pages + off + 16 * p, load);
          }
        }
      } else {
        // only rows that are visible: what else the tail holds is nobody's
        lost = r.slot < 0 || r.slot >= a.c.slots;
        const int B = 1 << a.c.block_shift, lo = a.window > 0 ? r.len - a.window : 0;
        const int64_t off = lost ? 0 : (((int64_t)r.slot * a.hkv + h) * B + (key & (B - 1))) * E::TAILB;
        constexpr int PIECES = kGranule * E::TAILB / 16, PER = E::TAILB / 16;
#pragma unroll
        for (int p = lane; p < PIECES; p += 32) {
          const int k = key + p / PER;
          const bool load = !lost && k < r.len && (k >= lo || k < a.sinks);
          const uint32_t dst = st + E::place_tail(p / PER, p % PER);
          const int64_t from = load ? off + 16 * p : 0;
          cp_async16_or_zero(dst, static_cast<const char*>(a.c.k_tail) + from, load);
          cp_async16_or_zero(dst + E::SIDE, static_cast<const char*>(a.c.v_tail) + from, load);
        }
      }
      if (__any_sync(0xffffffffu, lost) && lane == 0) queue[(tail - 1) & 3].bad = 1;
      r.u += count;
      if (r.u >= r.end) {
        seek(a, parts, lane);
        if (live) push(a, parts, queue, tail, lane);
      }
      look_up(a, lane);
    }
    tc::cp_async_commit();
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
  f.base = ((threadIdx.x >> 5) * gridDim.x + blockIdx.x) * chunk;
  f.left = 0;
  int head = 0, tail = 0, put = 0, get = 0;
  f.look_ahead(a, parts, lane);
  if (counter) asm volatile("griddepcontrol.wait;" ::: "memory");  // it has been cleared
  f.seek(a, parts, lane);
  if (f.live) f.push(a, parts, queue, tail, lane);
  f.look_up(a, lane);
#pragma unroll
  for (int s = 0; s < E::RING - 1; ++s) {
    f.fetch(a, parts, sh + put * L::STAGE, lane, queue, tail);
    put = put + 1 == E::RING ? 0 : put + 1;
  }
  E eng;
  while (head != tail) {
    __syncwarp();
    QuantRun r = queue[head & 3];
    const int g0 = (r.y % parts) * kHeadsPerRun, heads = min(kHeadsPerRun, group - g0);
    const int h0 = (r.y / parts) * group + g0;
    eng.start(a, (int64_t)r.i * a.hq + h0, heads, lane);
    while (r.u < r.end) {
      // the next tile on its way first, into the place that every lane has read
      f.fetch(a, parts, sh + put * L::STAGE, lane, queue, tail);
      put = put + 1 == E::RING ? 0 : put + 1;
      asm volatile("cp.async.wait_group %0;" ::"n"(E::RING - 1) : "memory");
      __syncwarp();
      unsigned char* stage = sh + get * L::STAGE;
      const typename E::Meta& meta = *reinterpret_cast<const typename E::Meta*>(stage + E::META);
      r.u += meta.count;
      if (meta.tail) eng.tail(a, stage, r.len, lane);
      else eng.tile(a, stage, r.len, lane);
      get = get + 1 == E::RING ? 0 : get + 1;
      __syncwarp();
    }
    __syncwarp();
    eng.finish(Sink(a, r, h0, heads, sizeof(typename E::Elem)), queue[head & 3].bad != 0, lane);
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

int launch_quant_decode(const QuantDecode& a, bool bf16, cudaStream_t st) {
  return bf16 ? decode<__nv_bfloat16>(a, st) : decode<float>(a, st);
}

}  // namespace gdn
