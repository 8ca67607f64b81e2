// attn_quant.h -- internal interface of the 8-bit cache: the C-ABI host code (attn_host.cu) checks arguments and
// calls these launchers.
#pragma once

#include "attn.h"

namespace gdn {

// Keys of one granule.  Blocks are multiples of it and begin at multiples of it, so the rows of a granule lie in
// one page, share their scales, and are all in the pages or all in the tail.
constexpr int kGranuleShift = 4, kGranule = 1 << kGranuleShift;

struct QuantCache {
  uint8_t *k_pages, *v_pages;  // [num_pages, hkv, page, d]
  float *k_scale, *v_scale;    // [num_pages, hkv, page / block]
  void *k_tail, *v_tail;       // [slots, hkv, block, d]
  int num_pages, page_shift, block_shift, slots, hkv;
  bool e4m3;
};

// n / d for n below 2^31 by a product (d >= 2): with 2^(l-1) < d <= 2^l, mul = floor(2^(31+l) / d) + 1 fits 32 bits, and
// n mul / 2^(31+l) exceeds n / d by less than 1 / d.
struct Divide {
  uint32_t mul, shift;
};
inline Divide divide_by(uint32_t d) {
  uint32_t l = 1;
  while ((uint64_t)1 << l < d) ++l;
  return {(uint32_t)(((uint64_t)1 << (31 + l)) / d + 1), l - 1};
}
__host__ __device__ inline uint32_t divide(uint32_t n, Divide d) {
#ifdef __CUDA_ARCH__
  return __umulhi(n, d.mul) >> d.shift;
#else
  return (uint32_t)((uint64_t)n * d.mul >> 32) >> d.shift;
#endif
}

// What append and read share: request n has rows cu[n] .. cu[n + 1] of the packed tensors, which are the last
// ones of its seq_lens[n] positions.
struct QuantRows {
  QuantCache c;
  int N, T, max_blocks;
  const int32_t *cu, *seq_lens, *block_table, *slot;
  WsHeader* hdr;            // or NULL: what is wrong is not reported
  Divide heads;             // by 2 hkv, the units of a piece
  bool by_token;            // pieces are numbered by the first of their rows, not as below
  const void *k_in, *v_in;  // append
  int64_t k_stride, v_stride;
  void *k_out, *v_out;  // read
};
// Pieces of `1 << shift` positions that hold rows: numbered with a request's first at cu[n] / piece + 2 n, which
// leaves every request enough numbers without a sum over the others.
inline int64_t quant_pieces(int N, int T, int shift) { return (int64_t)(T >> shift) + 2 * (int64_t)N; }
// With few rows a request it is fewer to number every row, and to leave out those that do not begin a piece.
inline bool quant_by_token(int N, int T, int shift) { return T < quant_pieces(N, T, shift); }
// A unit is a piece of one head of k or v, one warp's or, in append, block / 16 warps'; units are numbered in 31 bits, a piece's
// side by side.  Calls of more are refused.
inline bool quant_units_fit(int N, int T, int shift, int hkv) { return quant_pieces(N, T, shift) * 2 * hkv < (int64_t)1 << 31; }
inline int64_t quant_units(int N, int T, int shift, int hkv) {
  return (quant_by_token(N, T, shift) ? T : quant_pieces(N, T, shift)) * 2 * hkv;
}
// CTAs of `threads` for them, where a unit takes `each` warps, and one before them that checks the call
inline int64_t quant_blocks(int64_t units, int each, int threads) { return 1 + (units * each + threads / 32 - 1) / (threads / 32); }
// the unit that a warp of CTA `block` (not counting the first) takes; units and more of them behind the last have no piece
__host__ __device__ inline uint32_t quant_unit(uint32_t block, int threads, int warp, int each_shift) {
  return block * (uint32_t)(threads >> (5 + each_shift)) + (uint32_t)(warp >> each_shift);
}

// Decode attention: a request's visible keys are counted in granules that hold any.
struct QuantDecode : PagedDecode {
  QuantCache c;
  const int32_t* slot;
};
// At most that many granules of a request of `len` keys hold visible ones.
inline int64_t quant_granules(int64_t len, int window, int sinks) {
  const int64_t all = (len + kGranule - 1) / kGranule;
  if (window <= 0 || len <= window) return all;
  const int64_t some = ((int64_t)sinks + kGranule - 1) / kGranule + ((int64_t)window + 2 * kGranule - 2) / kGranule;
  return some < all ? some : all;
}
// Granules of a run (Split::keys) and runs of a request, from the request's granules and the number of key heads alone, so
// that a request's result does not depend on the batch: kQuantRuns to twice as many runs over all of a request's key heads,
// of 4 to 32 granules, evened out; fewer where these would be shorter, more where they would be longer (21597 tokens of 4 key
// heads: 41 runs a head).  With at most 16 granules a run, 7 requests of 4 to 22 thousand tokens take 20.4 us instead of 22.7, 33
// of 500 to 15619 with 16 heads a key head 48.5 instead of 49.2, but 256 of about 2112 with 8 key heads 199.5 instead of 194; with
// at most 8 granules these three take 24.3, 55.6 and 261.
constexpr int kQuantRuns = 32, kQuantMinShift = 2, kQuantMaxShift = 5;
__host__ __device__ inline int quant_shift(int n, int hkv) {
  const int64_t x = (int64_t)n * hkv;
  int s = kQuantMinShift;
  while (s < kQuantMaxShift && x >= (int64_t)kQuantRuns << (s + 1)) ++s;
  return s;
}
__host__ __device__ inline int quant_target(int n, int hkv) {
  const int s = quant_shift(n, hkv), r = (n + (1 << s >> 1)) >> s;
  return r < 1 ? 1 : r;
}
__host__ __device__ inline Split quant_split(int n, int hkv) {
  const int r = quant_target(n, hkv);
  Split s;
  s.keys = (n + r - 1) / r;
  s.runs = n == 0 ? 0 : (n + s.keys - 1) / s.keys;
  return s;
}
int quant_max_splits(int64_t granules, int hkv);
int launch_quant_decode(const QuantDecode& a, bool bf16, cudaStream_t st);

int launch_quant_append(const QuantRows& a, int d, bool bf16, cudaStream_t st);
int launch_quant_read(const QuantRows& a, int d, bool bf16, bool out_bf16, cudaStream_t st);

}  // namespace gdn
