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

// What append and read share: request n has rows cu[n] .. cu[n + 1] of the packed tensors, which are the last
// ones of its seq_lens[n] positions.
struct QuantRows {
  QuantCache c;
  int N, T, max_blocks;
  const int32_t *cu, *seq_lens, *block_table, *slot;
  WsHeader* hdr;
  const void *k_in, *v_in;  // append
  int64_t k_stride, v_stride;
  void *k_out, *v_out;  // read
};
// Pieces of `1 << shift` positions that hold rows: numbered with a request's first at cu[n] / piece + 2 n, which
// leaves every request enough numbers without a sum over the others.
inline int64_t quant_pieces(int N, int T, int shift) { return (int64_t)(T >> shift) + 2 * (int64_t)N; }

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
int launch_quant_decode(const QuantDecode& a, bool bf16, cudaStream_t st);

int launch_quant_append(const QuantRows& a, int d, bool bf16, cudaStream_t st);
int launch_quant_read(const QuantRows& a, int d, bool bf16, bool out_bf16, cudaStream_t st);

}  // namespace gdn
