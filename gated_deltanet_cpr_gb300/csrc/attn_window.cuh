// attn_window.cuh -- what the sliding-window attention kernels share: which sequence and rows a
// CTA works on, and which keys those rows see.
//
// A query at position p (its row plus Lk - Lq) sees key j iff j <= p and (no window, or
// p - j < window, or j < sinks).  For a block of query rows the visible keys lie in
// [0, min(sinks, ...)) and [lo, hi); for a block of keys the queries that see any of them lie
// in one range, which for a block that holds first keys runs to the end of the sequence.
#pragma once

#include "attn.h"

namespace gdn {
namespace win {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sequence and block of work item `item`, without a work list: block b of sequence s is item
// floor(cu[s] / rows) + s + b.  These never collide (floor(x) + ceil(y) <= floor(x + y) + 1), at
// most one item per sequence stays empty, and floor(total / rows) + N items hold them all.
__host__ __device__ inline int64_t item_count(int total, int rows, int N) { return (int64_t)total / rows + N; }

struct Seq {
  int s, q0, Lq, k0, Lk;
  bool ok;
};

__device__ __forceinline__ bool valid_range(const int32_t* cu, int s, int total) {
  const int a = cu[s], b = cu[s + 1];
  return 0 <= a && a <= b && b <= total;
}

// `over_keys`: items are blocks of keys instead of queries.  The block's first row goes to row0;
// ok is false for an empty item or a table that is not valid there.
__device__ __forceinline__ Seq find_seq(const WindowAttn& a, int64_t item, int rows, bool over_keys, int& row0) {
  const int32_t* cu = over_keys ? a.cu_k : a.cu_q;
  int lo = 0, hi = a.N;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (cu[m] / rows + m <= item) lo = m; else hi = m;
  }
  Seq q;
  q.s = lo;
  q.ok = valid_range(a.cu_q, lo, a.Tq) && valid_range(a.cu_k, lo, a.Tk);
  q.q0 = a.cu_q[lo];
  q.Lq = a.cu_q[lo + 1] - q.q0;
  q.k0 = a.cu_k[lo];
  q.Lk = a.cu_k[lo + 1] - q.k0;
  const int64_t b = item - (cu[lo] / rows + lo);
  row0 = (int)(b * rows);
  q.ok = q.ok && b >= 0 && row0 < (over_keys ? q.Lk : q.Lq);
  return q;
}

// Thread block 0 sets the call's error word from both tables; all its threads call this.
__device__ __forceinline__ void check_tables(const WindowAttn& a) {
  bool bad = false;
  for (int s = threadIdx.x; s < a.N; s += blockDim.x)
    bad |= !valid_range(a.cu_q, s, a.Tq) || !valid_range(a.cu_k, s, a.Tk);
  if (threadIdx.x == 0)
    bad |= a.cu_q[0] != 0 || a.cu_k[0] != 0 || a.cu_q[a.N] != a.Tq || a.cu_k[a.N] != a.Tk;
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) a.hdr->err = any ? GDN_DEVERR_CU_SEQLENS : 0;
}

__device__ __forceinline__ bool visible(int p, int j, int window, int sinks) {
  return j <= p && (window <= 0 || p - j < window || j < sinks);
}

// Key blocks (of `bk` keys) that query positions [p0, p1] need: [0, head) and [from, to).
struct KeyBlocks {
  int head, from, to;
  __device__ __forceinline__ KeyBlocks(int p0, int p1, int Lk, int window, int sinks, int bk) {
    to = p1 < 0 ? 0 : (min(p1, Lk - 1) + bk) / bk;
    from = window > 0 ? max(0, p0 - window + 1) / bk : 0;
    from = min(from, to);
    // first keys that the window of some row no longer shows: those below p1 - window + 1
    head = window > 0 && p1 - window + 1 > 0 ? (min(sinks, p1 - window + 1) + bk - 1) / bk : 0;
    head = min(head, from);
  }
  __device__ __forceinline__ int count() const { return head + to - from; }
  __device__ __forceinline__ int block(int i) const { return i < head ? i : from + (i - head); }
};

// Query rows [q_lo, q_hi) of the sequence that see any key of [j0, j1).
struct QueryRange {
  int lo, hi;
  __device__ __forceinline__ QueryRange(const Seq& q, int j0, int j1, int window, int sinks) {
    const int off = q.Lk - q.Lq;
    lo = max(0, j0 - off);
    hi = window > 0 && j0 >= sinks ? min(q.Lq, j1 - 1 + window - off) : q.Lq;
    hi = max(hi, lo);
  }
};

}  // namespace win
}  // namespace gdn
