// attn_quant_rows.cu -- the 8-bit cache's rows: rounding new keys and values to codes and scales as they are
// written, and reading cached ones back into packed rows.
//
// Both kernels move every byte once.  Reading is bound by DRAM: 282 thousand rows of 4 heads, d = 128, 869 MB, in 133 us, 6.5 TB/s
// (98% of a copy's rate).  Writing is bound by instructions, about 580 for the 2048 values of a block, and by the chain of dependent loads
// that a warp makes for one unit (offsets, lengths, rows): 16384 tokens of 8 heads, 101 MB, in 20 us, 5.1 TB/s.
// A warp that took several units after one search was slower (more registers, fewer warps).  Short calls are
// launch and that chain: 256 single tokens 4.7 us, 23 chunks 4.9.  The position-aligned pieces of the requests are numbered so
// that a warp finds its request with one search of the offsets, 32 of them at a time.
#include <algorithm>

#include "attn_quant.h"

namespace gdn {

namespace {

// Threads of a CTA.  Four warps start and end sooner than eight (256 rows read 3.4 against 3.7 us, 10 thousand granules 6.6
// against 6.9; long reads the same); a block of 128 tokens takes eight.
constexpr int kThreads = 128, kMostThreads = 256, kMostWarps = kMostThreads / 32;

// The last n < N with (cu[n] >> shift) + gap n <= w: the request that piece w belongs to.  All lanes take part.
__device__ __forceinline__ int request_of(const int32_t* cu, int N, int shift, int gap, uint32_t w, int lane) {
  int lo = 0, n = N;
  while (n > 1) {
    const int step = (n + 31) >> 5, i = lo + lane * step;
    const bool at = lane * step < n && (uint32_t)(cu[i] >> shift) + (uint32_t)(gap * i) <= w;
    const uint32_t m = __ballot_sync(0xffffffffu, at) | 1u;
    const int k = (31 - __clz(m)) * step;
    lo += k;
    n = min(step, n - k);
  }
  return lo;
}

// A piece of a request: `1 << shift` positions from `first` on.
struct Piece {
  int n, j;             // request, number of the piece in it
  uint32_t first;       // position
  uint32_t begin, len;  // the request's positions [begin, len) have rows; len 0: its length is not valid
  int cu0;              // row of position `begin`
  bool on;
};
__device__ __forceinline__ Piece piece_of(const QuantRows& a, int shift, uint32_t w, int lane) {
  Piece p;
  const int s = a.by_token ? 0 : shift, gap = a.by_token ? 0 : 2;
  int c0 = -1, c1 = -1;
  p.n = 0;
  if (a.by_token && a.T == a.N) {  // a row each, as in a decode step: no search, if that is so
    p.n = (int)w;
    c0 = a.cu[p.n];
    c1 = a.cu[p.n + 1];
  }
  if (c0 != (int)w || c1 != (int)w + 1) {
    p.n = request_of(a.cu, a.N, s, gap, w, lane);
    c0 = a.cu[p.n];
    c1 = a.cu[p.n + 1];
  }
  const int len = a.seq_lens[p.n], rows = c1 - c0;
  const bool fits = len >= rows;
  p.cu0 = c0;
  p.begin = fits ? (uint32_t)(len - rows) : 0u;  // if not, numbered as if its rows began at position 0
  const uint32_t end = fits ? (uint32_t)len : (uint32_t)rows;
  p.on = c0 >= 0 && c1 > c0 && c1 <= a.T;
  const int at = (int)(w - ((uint32_t)(c0 >> s) + (uint32_t)(gap * p.n)));  // row or piece of the request; both are below 2^31
  const uint32_t mask = (1u << shift) - 1u;
  if (a.by_token) {
    const uint32_t pos = p.begin + (uint32_t)at;
    p.on = p.on && at >= 0 && at < rows && (at == 0 || (pos & mask) == 0u);
    p.first = pos & ~mask;
  } else {
    p.first = ((p.begin >> shift) + (uint32_t)at) << shift;
    p.on = p.on && at >= 0 && p.first < end;
  }
  p.j = (int)((p.first >> shift) - (p.begin >> shift));
  p.len = fits ? end : 0u;
  return p;
}

__device__ __forceinline__ void report(WsHeader* h, int code) {
  if (!h) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the word has been cleared
  set_error(h, code);
}

// What is wrong with offsets, lengths and slots; one block.  APPEND: a slot is needed whatever the length.
template <bool APPEND>
__device__ void check_requests(const QuantRows& a) {
  int bad = 0;
  for (int n = threadIdx.x; n < a.N; n += blockDim.x) {
    const int c0 = a.cu[n], c1 = a.cu[n + 1];
    const int first = n == 0 ? 0 : c0, last = n == a.N - 1 ? a.T : c1;
    if (c0 != first || c1 != last || c0 < 0 || c1 < c0 || c1 > a.T) {
      bad |= 1;
      continue;
    }
    if (c1 == c0) continue;
    const int len = a.seq_lens[n], slot = a.slot ? a.slot[n] : n;
    if (len < c1 - c0) bad |= 2;
    else if ((slot < 0 || slot >= a.c.slots) && (APPEND || (len & ((1 << a.c.block_shift) - 1)))) bad |= 4;
  }
  bad = (__syncthreads_or(bad & 1) ? 1 : 0) | (__syncthreads_or(bad & 2) ? 2 : 0) | (__syncthreads_or(bad & 4) ? 4 : 0);
  if (threadIdx.x == 0 && bad)
    report(a.hdr, bad & 1 ? GDN_DEVERR_CU_SEQLENS : bad & 2 ? GDN_DEVERR_POS : GDN_DEVERR_SLOT);
}

// ------------------------------------------------------------------------- rounding ----
// Codes of an int8 block: the quotient 127 x / m is rounded as it is in exact arithmetic.  inv is 127 / m rounded up, so that x
// inv is the quotient or up to 2^-23 of it more (in magnitude), and one fma rounds it to a whole number.  In bf16 that is right
// as it stands, in three cases, with X and M the 8-bit significands of x and m.  A quotient that is no half lies 2^-16 of
// itself or more away from one, 254 X 2^t and odd M 2^u being whole numbers of 16 bits.  One that is a half, 254 x = odd m, has
// a 127 in odd or in M: 63.5 goes up to 64, which is even; M = 254 makes 127 / m a power of two, and a half goes to even by
// itself.  In fp32 one that rounds up from next to a half can be wrong: there the sign of 254 x - (2 k + 1) m decides, which
// the two products and what their rounding lost give exactly.
struct Rounder {
  float inv, m, scale;  // scale: what the block stores; m == 0: its codes are zeros
  float down;           // keeps the products of the exact comparison finite
  __device__ __forceinline__ Rounder(uint32_t amax_bits, bool e4m3) {
    m = __uint_as_float(amax_bits);
    inv = 0.f;
    down = 1.f;
    if (amax_bits >= 0x7f800000u) {
      scale = __builtin_nanf("");
      m = 0.f;
    } else if (m < 0x1p-100f) {
      scale = 0.f;
      m = 0.f;
    } else if (e4m3) {
      // 448 = 1.75 2^8: the exponent of m less 8, one more where its significand is above 1.75
      const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
      scale = __uint_as_float((uint32_t)e << 23);
      inv = __uint_as_float((uint32_t)(254 - e) << 23);
    } else {
      scale = __fdiv_rn(m, 127.f);
      inv = __fdiv_ru(127.f, m);
      if (m > 0x1p100f) down = 0x1p-20f;
    }
  }
  static constexpr float kMagic = 12582912.f;  // 1.5 2^23: the sum's last bits are a whole number, ties to even
  static constexpr float kNear = 0.5f - 0x1p-14f;
  // y = x inv + kMagic rounded to a whole number r, and d what that took off: if x inv lies next to a half, the whole number on
  // the right side of it, as x 127 / m has it.
  __device__ __forceinline__ static float settle(float x, float y, float d, float m, float down) {
    const float r = __fsub_rn(y, kMagic), s = d < 0.f ? -1.f : 1.f, odd = __fmaf_rn(2.f, r, s);  // the half is odd / 2
    const float a = __fmul_rn(x, down), b = __fmul_rn(m, down);
    const float q = __fmul_rn(254.f, a), f = __fmaf_rn(254.f, a, -q), p = __fmul_rn(odd, b), e = __fmaf_rn(odd, b, -p);
    const float diff = __fmul_rn(__fadd_rn(__fsub_rn(q, p), __fsub_rn(f, e)), s);  // > 0: past the half
    return fabsf(d) > kNear && (diff > 0.f || (diff == 0.f && ((int)r & 1))) ? __fadd_rn(y, s) : y;
  }
  // codes of 4 values, pairs (x0, x1) and (x2, x3)
  template <bool E4M3, bool BF16>
  __device__ __forceinline__ uint32_t four(const float2 (&x)[2]) const {
    const float2 i2 = make_float2(inv, inv);
    if constexpr (E4M3) {
      uint16_t lo, hi;
      const float2 a = mul2(x[0], i2), b = mul2(x[1], i2);
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
      return (uint32_t)lo | ((uint32_t)hi << 16);
    } else {
      const float2 up = make_float2(kMagic, kMagic), one = make_float2(1.f, 1.f);
      const float2 y[2] = {fma2(x[0], i2, up), fma2(x[1], i2, up)};
      if constexpr (!BF16) {
        float2 d[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 r = fma2(y[i], one, make_float2(-kMagic, -kMagic));
          d[i] = fma2(x[i], i2, make_float2(-r.x, -r.y));  // what the rounding took off
        }
        if (fmaxf(fmaxf(fabsf(d[0].x), fabsf(d[0].y)), fmaxf(fabsf(d[1].x), fabsf(d[1].y))) > kNear)
          return settled(make_float4(x[0].x, x[0].y, x[1].x, x[1].y), make_float4(d[0].x, d[0].y, d[1].x, d[1].y),
                         make_float4(y[0].x, y[0].y, y[1].x, y[1].y), m, down);
      }
      return bytes(y[0].x, y[0].y, y[1].x, y[1].y);
    }
  }
  // the last bytes of four sums with kMagic
  __device__ __forceinline__ static uint32_t bytes(float y0, float y1, float y2, float y3) {
    const uint32_t a = __byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(y2), __float_as_uint(y3), 0x0040);
    return __byte_perm(a, b, 0x5410);
  }
  // a call of its own: in place it would fill the instruction cache
  __device__ __noinline__ static uint32_t settled(float4 x, float4 d, float4 y, float m, float down) {
    return bytes(settle(x.x, y.x, d.x, m, down), settle(x.y, y.y, d.y, m, down), settle(x.z, y.z, d.z, m, down),
                 settle(x.w, y.w, d.w, m, down));
  }
};

// a lane's 16 bytes of a row
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ __forceinline__ static uint32_t amax(const uint4& u, uint32_t m) {  // of pairs
    m = __vmaxu2(m, u.x & 0x7fff7fffu);
    m = __vmaxu2(m, u.y & 0x7fff7fffu);
    m = __vmaxu2(m, u.z & 0x7fff7fffu);
    return __vmaxu2(m, u.w & 0x7fff7fffu);
  }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
  __device__ __forceinline__ static float2 pair(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  template <bool E4M3>
  __device__ __forceinline__ static void store(const Rounder& r, const uint4& u, uint8_t* to) {
    uint2 o;
    o.x = r.four<E4M3, true>({pair(u.x), pair(u.y)});
    o.y = r.four<E4M3, true>({pair(u.z), pair(u.w)});
    *reinterpret_cast<uint2*>(to) = o;
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ __forceinline__ static uint32_t amax(const uint4& u, uint32_t m) {
    return max(max(max(m, u.x & 0x7fffffffu), max(u.y & 0x7fffffffu, u.z & 0x7fffffffu)), u.w & 0x7fffffffu);
  }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return m; }
  template <bool E4M3>
  __device__ __forceinline__ static void store(const Rounder& r, const uint4& u, uint8_t* to) {
    *reinterpret_cast<uint32_t*>(to) =
        r.four<E4M3, false>({make_float2(__uint_as_float(u.x), __uint_as_float(u.y)),
                             make_float2(__uint_as_float(u.z), __uint_as_float(u.w))});
  }
};

// --------------------------------------------------------------------------- append ----
// A unit is one block of one head of k or v; a warp takes 16 of its rows, block / 16 warps a unit, whose largest values
// meet in shared memory.  The request's first block also takes care of its tail: a first block that is completed has the tail's
// rows in registers before the rows of a later, unfinished one replace them.
template <int D, typename T>
__global__ void __launch_bounds__(kMostThreads) k_quant_append(const QuantRows a) {
  constexpr int VEC = Vec<T>::N, LPR = D / VEC, RPP = 32 / LPR, PASSES = kGranule / RPP;
  __shared__ uint32_t most[kMostWarps];
  if (blockIdx.x == 0) {
    if (a.hdr) check_requests<true>(a);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const QuantCache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, B = 1 << c.block_shift;
  const int each_shift = c.block_shift - kGranuleShift, each = 1 << each_shift;  // warps of a unit
  const int part = warp & (each - 1);                                            // this one's rows of it
  const uint32_t pieces = a.by_token ? (uint32_t)a.T : (uint32_t)(a.T >> c.block_shift) + 2u * (uint32_t)a.N;
  const uint32_t all = 2u * (uint32_t)c.hkv, unit = quant_unit(blockIdx.x - 1, (int)blockDim.x, warp, each_shift);
  const uint32_t w = divide(unit, a.heads), rest = unit - w * all;
  const int h = (int)(rest >> 1);
  const bool is_v = rest & 1;
  Piece p{};
  if (w < pieces) p = piece_of(a, c.block_shift, w, lane);
  int slot = 0, page = -1;
  if (p.on) {
    slot = a.slot ? a.slot[p.n] : p.n;
    p.on = p.len != 0 && slot >= 0 && slot < c.slots;  // if not, reported by block 0
  }
  const bool whole = p.on && p.first + (uint32_t)B <= p.len;
  if (whole) {
    const uint32_t b = p.first >> c.page_shift;
    page = b < (uint32_t)a.max_blocks ? a.block_table[(int64_t)p.n * a.max_blocks + b] : -1;
  }
  const int r0 = part * kGranule + lane / LPR, col = lane % LPR * VEC;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const T* src = static_cast<const T*>(is_v ? a.v_in : a.k_in) + h * D + col;
  T* tail = static_cast<T*>(is_v ? c.v_tail : c.k_tail) + (((int64_t)slot * c.hkv + h) * B + r0) * D + col;
  // rows [0, PASSES) of this lane of the block at `first`: new tokens' rows from src, earlier ones' from the tail
  uint4 x[PASSES];
  auto load = [&](uint32_t first, bool from_tail) {
    const T* s = src + (int64_t)(p.cu0 + (int)(first + (uint32_t)r0 - p.begin)) * stride;  // of a row that may not be there
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const uint32_t pos = first + (uint32_t)(r0 + i * RPP);
      x[i] = make_uint4(0, 0, 0, 0);
      if (pos < p.len && pos >= p.begin) x[i] = *reinterpret_cast<const uint4*>(s + i * RPP * stride);
      else if (pos < p.begin && from_tail) x[i] = *reinterpret_cast<const uint4*>(tail + i * RPP * D);
    }
  };
  uint32_t m = 0;
  if (whole && p.first >= p.begin) {  // all of it new, as in a prefill
    const T* s = src + (int64_t)(p.cu0 + (int)(p.first + (uint32_t)r0 - p.begin)) * stride;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) x[i] = *reinterpret_cast<const uint4*>(s + i * RPP * stride);
  } else if (whole || (p.on && p.j == 0)) {  // an unfinished block that is not the first is the first one's unit's to write, below
    load(p.first, whole);
  }
  if (whole) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) m = Vec<T>::amax(x[i], m);
    m = __reduce_max_sync(0xffffffffu, Vec<T>::bits(m));
  }
  if (each > 1) {
    if (lane == 0) most[warp] = m;
    __syncthreads();  // the tail's rows are in registers, too
    for (int i = 0; i < each; ++i) m = max(m, most[warp - part + i]);
  }
  if (whole) {
    if (page < 0 || page >= c.num_pages) {
      if (lane == 0) report(a.hdr, GDN_DEVERR_PAGES);
    } else {
      const Rounder round(m, c.e4m3);
      const int64_t row = (((int64_t)page * c.hkv + h) << c.page_shift) + (p.first & ((1u << c.page_shift) - 1u));
      uint8_t* to = (is_v ? c.v_pages : c.k_pages) + (row + r0) * D + col;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        if (round.m == 0.f) x[i] = make_uint4(0, 0, 0, 0);
      }
      if (c.e4m3) {
#pragma unroll
        for (int i = 0; i < PASSES; ++i) Vec<T>::template store<true>(round, x[i], to + i * RPP * D);
      } else {
#pragma unroll
        for (int i = 0; i < PASSES; ++i) Vec<T>::template store<false>(round, x[i], to + i * RPP * D);
      }
      if (part == 0 && lane == 0) (is_v ? c.v_scale : c.k_scale)[row >> c.block_shift] = round.scale;
    }
  }
  const uint32_t last = p.len & ~(uint32_t)(B - 1);  // where the request's unfinished block begins
  if (p.on && p.j == 0 && last < p.len) {
    if (whole) load(last, false);  // after the first one, whose rows the tail held
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const uint32_t pos = last + (uint32_t)(r0 + i * RPP);
      if (pos < p.len && pos >= p.begin) *reinterpret_cast<uint4*>(tail + i * RPP * D) = x[i];
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // so that the word is cleared before the next kernel begins
}

// ----------------------------------------------------------------------------- read ----
__device__ __forceinline__ void widen(uint32_t four, bool e4m3, float scale, float (&y)[4]) {
  if (e4m3) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(four & 0xffffu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(four >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    y[0] = a.x, y[1] = a.y, y[2] = b.x, y[3] = b.y;
  } else {
    // 2^23 + (c + 128), less 2^23 + 128
    const uint32_t u = four ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __fsub_rn(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)), 8388736.f);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(y[i], scale);
}

// One granule of one head of k or v a warp: 16 rows, contiguous in the page.
template <int D, typename T, typename TO>
__global__ void __launch_bounds__(kThreads) k_quant_read(const QuantRows a) {
  constexpr int LPR = D / 8, RPP = 32 / LPR, PASSES = kGranule / RPP;
  if (blockIdx.x == 0) {
    if (a.hdr) check_requests<false>(a);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const QuantCache& c = a.c;
  const int lane = threadIdx.x & 31;
  const uint32_t units = (a.by_token ? (uint32_t)a.T : (uint32_t)(a.T / kGranule) + 2u * (uint32_t)a.N) * 2u * (uint32_t)c.hkv;
  const uint32_t unit = quant_unit(blockIdx.x - 1, kThreads, (int)(threadIdx.x >> 5), 0);
  if (unit < units) {
    const uint32_t w = divide(unit, a.heads), rest = unit - w * 2u * (uint32_t)c.hkv;
    const int h = (int)(rest >> 1);
    const bool is_v = rest & 1;
    const Piece p = piece_of(a, kGranuleShift, w, lane);
    if (p.on) {
      const int B = 1 << c.block_shift, r0 = lane / LPR, col = lane % LPR * 8;
      const bool valid = p.len != 0;
      const int rows = a.cu[p.n + 1] - p.cu0;
      const uint32_t end = valid ? p.len : (uint32_t)rows, waits = p.len & ~(uint32_t)(B - 1);
      TO* out = static_cast<TO*>(is_v ? a.v_out : a.k_out) + ((int64_t)p.cu0 * c.hkv + h) * D + col;
      auto put = [&](uint32_t pos, const float (&y)[8]) {
        TO* to = out + (int64_t)(pos - p.begin) * c.hkv * D;
        if constexpr (sizeof(TO) == 2) {
          uint4 u;
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
            v[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          u = make_uint4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<uint4*>(to) = u;
        } else {
          store4(reinterpret_cast<float*>(to), make_float4(y[0], y[1], y[2], y[3]));
          store4(reinterpret_cast<float*>(to) + 4, make_float4(y[4], y[5], y[6], y[7]));
        }
      };
      bool lost = !valid;
      if (valid && p.first < waits) {
        const uint32_t b = p.first >> c.page_shift;
        const int page = b < (uint32_t)a.max_blocks ? a.block_table[(int64_t)p.n * a.max_blocks + b] : -1;
        if (page < 0 || page >= c.num_pages) {
          lost = true;
          if (lane == 0) report(a.hdr, GDN_DEVERR_PAGES);
        } else {
          const int64_t row = (((int64_t)page * c.hkv + h) << c.page_shift) + (p.first & ((1u << c.page_shift) - 1u));
          const uint8_t* from = (is_v ? c.v_pages : c.k_pages) + (row + r0) * D + col;
          uint2 x[PASSES];
#pragma unroll
          for (int i = 0; i < PASSES; ++i) x[i] = *reinterpret_cast<const uint2*>(from + i * RPP * D);
          const float scale = (is_v ? c.v_scale : c.k_scale)[row >> c.block_shift];
#pragma unroll
          for (int i = 0; i < PASSES; ++i) {
            const uint32_t pos = p.first + (uint32_t)(r0 + i * RPP);
            float lo[4], hi[4];
            widen(x[i].x, c.e4m3, scale, lo);
            widen(x[i].y, c.e4m3, scale, hi);
            if (pos >= p.begin && pos < end) put(pos, {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
          }
        }
      } else if (valid) {
        const int slot = a.slot ? a.slot[p.n] : p.n;
        lost = slot < 0 || slot >= c.slots;  // reported by block 0
        const T* tail = static_cast<const T*>(is_v ? c.v_tail : c.k_tail) + ((int64_t)slot * c.hkv + h) * B * D + col;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const uint32_t pos = p.first + (uint32_t)(r0 + i * RPP);
          if (lost || pos < p.begin || pos >= end) continue;
          float y[8];
          load8(tail + (int64_t)(pos - waits) * D, y);
          put(pos, y);
        }
      }
      if (lost) {
        const float x = __builtin_nanf("");
        for (int i = 0; i < PASSES; ++i) {
          const uint32_t pos = p.first + (uint32_t)(r0 + i * RPP);
          if (pos >= p.begin && pos < end) put(pos, {x, x, x, x, x, x, x, x});
        }
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The error word of a call; the rows' kernel starts beside this and waits for it where it has something to report.
__global__ void k_quant_clear(WsHeader* hdr) {
  asm volatile("griddepcontrol.launch_dependents;");
  hdr->err = 0;
}

template <typename K>
int launch(K* kernel, const QuantRows& a, int64_t units, int each, int threads, cudaStream_t st) {
  if (a.hdr) k_quant_clear<<<1, 1, 0, st>>>(a.hdr);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.stream = st;
  c.attrs = &attr;
  c.numAttrs = a.hdr ? 1 : 0;
  c.gridDim = dim3((unsigned)quant_blocks(units, each, threads));
  c.blockDim = dim3(threads);
  cudaLaunchKernelEx(&c, kernel, a);
  return a.hdr ? 2 : 1;
}

template <int D, typename T>
int append_t(QuantRows a, cudaStream_t st) {
  const int each = (1 << a.c.block_shift) / kGranule;  // warps of a unit
  a.by_token = quant_by_token(a.N, a.T, a.c.block_shift);
  a.heads = divide_by(2u * (uint32_t)a.c.hkv);
  const int64_t units = quant_units(a.N, a.T, a.c.block_shift, a.c.hkv);
  return launch(k_quant_append<D, T>, a, units, each, std::max(kThreads, 32 * each), st);
}

template <int D, typename T, typename TO>
int read_t(QuantRows a, cudaStream_t st) {
  a.by_token = quant_by_token(a.N, a.T, kGranuleShift);
  a.heads = divide_by(2u * (uint32_t)a.c.hkv);
  const int64_t units = quant_units(a.N, a.T, kGranuleShift, a.c.hkv);
  return launch(k_quant_read<D, T, TO>, a, units, 1, kThreads, st);
}

template <int D>
int read_d(const QuantRows& a, bool bf16, bool out_bf16, cudaStream_t st) {
  using H = __nv_bfloat16;
  if (bf16) return out_bf16 ? read_t<D, H, H>(a, st) : read_t<D, H, float>(a, st);
  return out_bf16 ? read_t<D, float, H>(a, st) : read_t<D, float, float>(a, st);
}

}  // namespace

int launch_quant_append(const QuantRows& a, int d, bool bf16, cudaStream_t st) {
  using H = __nv_bfloat16;
  if (d == 32) return bf16 ? append_t<32, H>(a, st) : append_t<32, float>(a, st);
  if (d == 64) return bf16 ? append_t<64, H>(a, st) : append_t<64, float>(a, st);
  return bf16 ? append_t<128, H>(a, st) : append_t<128, float>(a, st);
}

int launch_quant_read(const QuantRows& a, int d, bool bf16, bool out_bf16, cudaStream_t st) {
  if (d == 32) return read_d<32>(a, bf16, out_bf16, st);
  if (d == 64) return read_d<64>(a, bf16, out_bf16, st);
  return read_d<128>(a, bf16, out_bf16, st);
}

}  // namespace gdn
