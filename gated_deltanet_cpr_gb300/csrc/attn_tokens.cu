// attn_tokens.cu -- the attention layer's per-token operators: norms of queries and keys with
// the rotation in the same pass (and its gradient), and the paged cache's bookkeeping.
#include "attn.h"

namespace gdn {

namespace {

// =====================================================================================
// Norm and rotation.  One row is one head of one token; LPR = D / 4 lanes hold 4 consecutive
// entries each, a warp holds 32 / LPR rows at a time and U of these at once (their loads are
// issued together).  A work item is one token and a run of U * 32 / LPR of its rows, so that
// the few rows of a decode step spread over warps.
// =====================================================================================
constexpr int kNormThreads = 256;

template <int D>
struct RowLanes {
  static constexpr int LPR = D / 4, GPW = 32 / LPR;
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return __fmaf_rn(a.w, b.w, __fmaf_rn(a.z, b.z, __fmaf_rn(a.y, b.y, __fmul_rn(a.x, b.x))));
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  return make_float4(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y), __fmul_rn(a.z, b.z), __fmul_rn(a.w, b.w));
}
__device__ __forceinline__ float4 scale4(float4 a, float b) { return mul4(a, make_float4(b, b, b, b)); }

// 1 / sqrt of the norm's sum of squares (plus eps); 1 without a norm.  The square root and the
// reciprocal are the correctly rounded ones: they run once per row.
__device__ __forceinline__ float inverse_norm(int norm, float sumsq, float inv_d, float eps) {
  if (norm == GDN_NORM_NONE) return 1.f;
  const float m = norm == GDN_NORM_RMS ? __fmul_rn(sumsq, inv_d) : sumsq;
  return __frcp_rn(__fsqrt_rn(__fadd_rn(m, eps)));
}

// The angles that a lane's 4 entries use, and where its partners are.
struct Turn {
  float4 c, s;   // half: of entries i .. i + 3; interleaved: (c0, c0, c1, c1)
  int src;       // half: the lane that holds the partners
  bool on, low;  // whether these entries turn; half: whether they are the first of their pairs
};

template <int LPR>
__device__ __forceinline__ Turn turn_of(const NormRope& a, int64_t p, int lane, float sign) {
  Turn t;
  const int i = 4 * (lane % LPR), half = a.rot / 2;
  t.on = i < a.rot;
  t.low = i < half;
  t.src = t.on && a.layout == GDN_ROPE_HALF ? (t.low ? lane + a.rot / 8 : lane - a.rot / 8) : lane;
  t.c = make_float4(1.f, 1.f, 1.f, 1.f);
  t.s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (t.on) {
    if (a.layout == GDN_ROPE_HALF) {
      const int64_t at = p * half + (t.low ? i : i - half);
      t.c = *reinterpret_cast<const float4*>(a.cos + at);
      t.s = *reinterpret_cast<const float4*>(a.sin + at);
    } else {
      const float2 c = *reinterpret_cast<const float2*>(a.cos + p * half + i / 2);
      const float2 s = *reinterpret_cast<const float2*>(a.sin + p * half + i / 2);
      t.c = make_float4(c.x, c.x, c.y, c.y);
      t.s = make_float4(s.x, s.x, s.y, s.y);
    }
    t.s = scale4(t.s, sign);
  }
  return t;
}

// x c + (partner) s with the sign of the pair's place: the first takes -s, the second +s.
// All lanes of the warp call it together.
__device__ __forceinline__ float4 turn(const Turn& t, int layout, float4 x) {
  float4 y;
  if (layout == GDN_ROPE_HALF) {
    y.x = __shfl_sync(0xffffffffu, x.x, t.src);
    y.y = __shfl_sync(0xffffffffu, x.y, t.src);
    y.z = __shfl_sync(0xffffffffu, x.z, t.src);
    y.w = __shfl_sync(0xffffffffu, x.w, t.src);
    if (t.low) y = make_float4(-y.x, -y.y, -y.z, -y.w);
  } else {
    y = make_float4(-x.y, x.x, -x.w, x.z);
  }
  if (!t.on) return x;
  return make_float4(__fmaf_rn(y.x, t.s.x, __fmul_rn(x.x, t.c.x)), __fmaf_rn(y.y, t.s.y, __fmul_rn(x.y, t.c.y)),
                     __fmaf_rn(y.z, t.s.z, __fmul_rn(x.z, t.c.z)), __fmaf_rn(y.w, t.s.w, __fmul_rn(x.w, t.c.w)));
}

constexpr float kNan = __builtin_nanf("");

template <int D, typename TI, typename TO, int U>
__global__ void __launch_bounds__(kNormThreads) k_norm_rope(const NormRope a) {
  constexpr int LPR = RowLanes<D>::LPR, GPW = RowLanes<D>::GPW;
  const int lane = threadIdx.x & 31, i = 4 * (lane % LPR), grp = lane / LPR;
  const int rows = a.hq + a.hk + (a.v_pages ? a.hk : 0);
  const int per = (rows + U * GPW - 1) / (U * GPW);
  const int64_t item = (int64_t)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
  if (item >= (int64_t)a.T * per) return;
  const int64_t t = item / per;
  const int row0 = (int)(item % per) * U * GPW + grp;

  float4 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = row0 + u * GPW;
    x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < a.hq)
      x[u] = load4(static_cast<const TI*>(a.q) + t * a.q_stride + (int64_t)r * D + i);
    else if (r < a.hq + a.hk)
      x[u] = load4(static_cast<const TI*>(a.k) + t * a.k_stride + (int64_t)(r - a.hq) * D + i);
    else if (r < rows)
      x[u] = load4(static_cast<const TI*>(a.v) + t * a.v_stride + (int64_t)(r - a.hq - a.hk) * D + i);
  }
  const int64_t p = a.rot ? a.pos[t] : 0;
  const bool bad = a.rot && (p < 0 || p >= a.table_rows);
  const Turn tn = turn_of<LPR>(a, bad ? 0 : p, lane, 1.f);
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
  const float4 wq = a.wq ? load4(a.wq + i) : one, wk = a.wk ? load4(a.wk + i) : one;
  const int64_t slot = a.slot_map ? a.slot_map[t] : -1;
  const bool keep = slot >= 0 && slot < a.slots;
  const int64_t ps = (int64_t)1 << a.page_shift, page = slot >> a.page_shift, off = slot & (ps - 1);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = row0 + u * GPW;
    const float ss = row_sum<LPR>(dot4(x[u], x[u]));
    const float4 w = r < a.hq ? wq : wk;
    float4 y = turn(tn, a.layout, mul4(scale4(x[u], inverse_norm(a.norm, ss, 1.f / D, a.eps)), w));
    if (bad) y = make_float4(kNan, kNan, kNan, kNan);
    if (r < a.hq) {
      if (a.q_out) store4(static_cast<TO*>(a.q_out) + (t * a.hq + r) * D + i, y);
    } else if (r < a.hq + a.hk) {
      const int h = r - a.hq;
      if (a.k_out) store4(static_cast<TO*>(a.k_out) + (t * a.hk + h) * D + i, y);
      if (keep) store4(static_cast<TO*>(a.k_pages) + ((page * a.hk + h) * ps + off) * D + i, y);
    } else if (r < rows && keep) {
      const int h = r - a.hq - a.hk;
      store4(static_cast<TO*>(a.v_pages) + ((page * a.hk + h) * ps + off) * D + i, x[u]);
    }
  }
}

// Backward: dx per row, and with weights the sums of g x r over this block's items: each lane
// adds its 4 columns in the order of the items it meets, then the block's rows of lanes in
// ascending order; k_norm_rope_dw adds the blocks.
template <int D, typename TI, typename TG, int U>
__global__ void __launch_bounds__(kNormThreads) k_norm_rope_bwd(const NormRope a) {
  constexpr int LPR = RowLanes<D>::LPR, GPW = RowLanes<D>::GPW;
  const int lane = threadIdx.x & 31, i = 4 * (lane % LPR), grp = lane / LPR;
  const int rows = a.hq + a.hk, per = (rows + U * GPW - 1) / (U * GPW);
  const int64_t items = (int64_t)a.T * per, step = (int64_t)gridDim.x * (kNormThreads / 32);
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 wq = a.wq ? load4(a.wq + i) : one, wk = a.wk ? load4(a.wk + i) : one;
  const float cn = a.norm == GDN_NORM_RMS ? 1.f / D : a.norm == GDN_NORM_L2 ? 1.f : 0.f;
  float4 accq = zero, acck = zero;
  for (int64_t item = (int64_t)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5); item < items; item += step) {
    const int64_t t = item / per;
    const int row0 = (int)(item % per) * U * GPW + grp;
    float4 x[U], g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row0 + u * GPW;
      x[u] = g[u] = zero;
      if (r < a.hq) {
        x[u] = load4(static_cast<const TI*>(a.q) + t * a.q_stride + (int64_t)r * D + i);
        g[u] = load4(static_cast<const TG*>(a.gq) + (t * a.hq + r) * D + i);
      } else if (r < rows) {
        x[u] = load4(static_cast<const TI*>(a.k) + t * a.k_stride + (int64_t)(r - a.hq) * D + i);
        g[u] = load4(static_cast<const TG*>(a.gk) + (t * a.hk + (r - a.hq)) * D + i);
      }
    }
    const int64_t p = a.rot ? a.pos[t] : 0;
    const bool bad = a.rot && (p < 0 || p >= a.table_rows);
    const Turn tn = turn_of<LPR>(a, bad ? 0 : p, lane, -1.f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row0 + u * GPW;
      const float4 gr = turn(tn, a.layout, g[u]);
      const float4 gw = mul4(gr, r < a.hq ? wq : wk);
      const float rn = inverse_norm(a.norm, row_sum<LPR>(dot4(x[u], x[u])), 1.f / D, a.eps);
      const float xg = row_sum<LPR>(dot4(x[u], gw));
      const float f = -__fmul_rn(__fmul_rn(cn, __fmul_rn(rn, __fmul_rn(rn, rn))), xg);
      float4 dx = make_float4(__fmaf_rn(f, x[u].x, __fmul_rn(rn, gw.x)), __fmaf_rn(f, x[u].y, __fmul_rn(rn, gw.y)),
                              __fmaf_rn(f, x[u].z, __fmul_rn(rn, gw.z)), __fmaf_rn(f, x[u].w, __fmul_rn(rn, gw.w)));
      if (bad) dx = make_float4(kNan, kNan, kNan, kNan);
      if (r < a.hq)
        store4(static_cast<TI*>(a.dq) + (t * a.hq + r) * D + i, dx);
      else if (r < rows)
        store4(static_cast<TI*>(a.dk) + (t * a.hk + (r - a.hq)) * D + i, dx);
      if (a.partial && r < rows && !bad) {
        const float4 y = mul4(gr, scale4(x[u], rn));
        float4& acc = r < a.hq ? accq : acck;
        acc = make_float4(__fadd_rn(acc.x, y.x), __fadd_rn(acc.y, y.y), __fadd_rn(acc.z, y.z), __fadd_rn(acc.w, y.w));
      }
    }
  }
  if (!a.partial) return;
  constexpr int NR = kNormThreads / LPR;  // rows of lanes in the block
  __shared__ float sh[2][NR][D];
  const int rr = threadIdx.x / LPR;
  store4(&sh[0][rr][i], accq);
  store4(&sh[1][rr][i], acck);
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * D; e += kNormThreads) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r) s = __fadd_rn(s, sh[e / D][r][e % D]);
    a.partial[(int64_t)blockIdx.x * 2 * D + e] = s;
  }
}

// dw[e] = sum over blocks of partial[block][e], e < 2 D: 8 columns per CTA, 32 threads a column
// with ascending strided sums, then a fixed tree.
__global__ void __launch_bounds__(256) k_norm_rope_dw(const float* __restrict__ partial, int blocks, int D,
                                                      float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sh[8][33];
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3, e = blockIdx.x * 8 + c;
  float s = 0.f;
  for (int b = r; b < blocks; b += 32) s = __fadd_rn(s, partial[(int64_t)b * 2 * D + e]);
  sh[c][r] = s;
  __syncthreads();
  float x = sh[threadIdx.x >> 5][threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) {
    const int col = blockIdx.x * 8 + (threadIdx.x >> 5);
    (col < D ? dwq : dwk)[col % D] = x;
  }
}

template <int D, typename TI, typename TO>
void norm_rope_t(const NormRope& a, cudaStream_t st) {
  constexpr int U = 4, GPW = RowLanes<D>::GPW;
  const int rows = a.hq + a.hk + (a.v_pages ? a.hk : 0);
  const int64_t items = (int64_t)a.T * ((rows + U * GPW - 1) / (U * GPW));
  const int64_t blocks = (items + kNormThreads / 32 - 1) / (kNormThreads / 32);
  k_norm_rope<D, TI, TO, U><<<(unsigned)blocks, kNormThreads, 0, st>>>(a);
}

template <int D, typename TI, typename TG>
void norm_rope_bwd_t(const NormRope& a, cudaStream_t st) {
  constexpr int U = 4, GPW = RowLanes<D>::GPW;
  const int64_t items = (int64_t)a.T * ((a.hq + a.hk + U * GPW - 1) / (U * GPW));
  int64_t blocks = (items + kNormThreads / 32 - 1) / (kNormThreads / 32);
  if (a.partial && blocks > kNormBwdBlocks) blocks = kNormBwdBlocks;
  k_norm_rope_bwd<D, TI, TG, U><<<(unsigned)blocks, kNormThreads, 0, st>>>(a);
  if (a.partial) k_norm_rope_dw<<<2 * D / 8, 256, 0, st>>>(a.partial, (int)blocks, D, a.dwq, a.dwk);
}

#define GDN_BY_D(d, CALL)              \
  switch (d) {                         \
    case 32: CALL(32); break;          \
    case 64: CALL(64); break;          \
    default: CALL(128); break;         \
  }

// =====================================================================================
// Page tables.  Every CTA scans all the lengths (N <= 8192: a few microseconds, and no CTA has
// to wait for another), keeps the offsets in shared memory and then writes its share of the new
// table entries and tokens.
// =====================================================================================
constexpr int kMapThreads = 1024;

// exclusive block scan of (x, y); the totals in tx, ty
__device__ __forceinline__ void block_scan2(int64_t& x, int64_t& y, int64_t& tx, int64_t& ty) {
  __shared__ int64_t wx[32], wy[32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t x0 = x, y0 = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += u, y += v;
  }
  if (lane == 31) wx[w] = x, wy[w] = y;
  __syncthreads();
  if (w == 0) {
    int64_t u = wx[lane], v = wy[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t p = __shfl_up_sync(0xffffffffu, u, o), q = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) u += p, v += q;
    }
    wx[lane] = u;
    wy[lane] = v;
  }
  __syncthreads();
  tx = wx[31];
  ty = wy[31];
  x += (w ? wx[w - 1] : 0) - x0;
  y += (w ? wy[w - 1] : 0) - y0;
}

// the last n with off[n] <= t (off ascending, off[0] = 0 <= t < off[N])
__device__ __forceinline__ int find(const int32_t* off, int N, int t) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (off[m] <= t) lo = m; else hi = m;
  }
  return lo;
}

__device__ __forceinline__ bool page_ok(int page, int shift) {
  return page >= 0 && page <= (INT32_MAX >> shift);
}

__global__ void __launch_bounds__(kMapThreads) k_page_map(const PageMap a) {
  extern __shared__ int32_t sh[];
  int32_t* cu = sh;                 // [N + 1] offsets of the new tokens
  int32_t* first = sh + a.N + 1;    // [N + 1] offsets into the free list
  const int tid = threadIdx.x, ps1 = (1 << a.page_shift) - 1;
  const int per = (a.N + kMapThreads - 1) / kMapThreads, n0 = tid * per;
  // pass 1: sums of the thread's requests, and what is wrong with them
  int64_t tok = 0, pg = 0;
  bool bad_len = false, bad_row = false;
  for (int n = n0; n < n0 + per && n < a.N; ++n) {
    const int64_t l = a.lens[n], m = a.new_lens[n];
    const int64_t have = (l + ps1) >> a.page_shift, want = (l + m + ps1) >> a.page_shift;
    bad_len |= l < 0 || m < 0 || l + m > INT32_MAX;
    bad_row |= want > a.max_blocks;
    tok += m;
    pg += want - have;
  }
  int64_t tok0 = tok, pg0 = pg, tok_all, pg_all;
  block_scan2(tok0, pg0, tok_all, pg_all);
  const int any_len = __syncthreads_or(bad_len), any_row = __syncthreads_or(bad_row);
  const int err = any_len ? GDN_DEVERR_POS
                  : tok_all != a.T ? GDN_DEVERR_CU_SEQLENS
                  : (any_row || pg_all > a.num_free) ? GDN_DEVERR_PAGES : 0;
  const int64_t gtid = (int64_t)blockIdx.x * kMapThreads + tid, gsize = (int64_t)gridDim.x * kMapThreads;
  if (err) {
    for (int64_t t = gtid; t < a.T; t += gsize) a.positions[t] = a.slot_map[t] = -1;
    if (blockIdx.x == 0) {
      for (int n = tid; n < a.N; n += kMapThreads) a.seq_lens[n] = 0;
      for (int n = tid; n <= a.N; n += kMapThreads) a.cu[n] = 0;
      if (tid == 0) *a.pages_used = 0, a.hdr->err = err;
    }
    return;
  }
  // pass 2: the offsets
  int64_t c = tok0, f = pg0;
  for (int n = n0; n < n0 + per && n < a.N; ++n) {
    const int l = a.lens[n], m = a.new_lens[n];
    cu[n] = (int32_t)c;
    first[n] = (int32_t)f;
    if (blockIdx.x == 0) {
      a.seq_lens[n] = l + m;
      a.cu[n] = (int32_t)c;
    }
    c += m;
    f += (((int64_t)l + m + ps1) >> a.page_shift) - (((int64_t)l + ps1) >> a.page_shift);
  }
  if (tid == 0) {
    cu[a.N] = (int32_t)tok_all;
    first[a.N] = (int32_t)pg_all;
    if (blockIdx.x == 0) {
      a.cu[a.N] = (int32_t)tok_all;
      *a.pages_used = (int32_t)pg_all;
    }
  }
  __syncthreads();
  // the new pages' entries
  for (int64_t p = gtid; p < pg_all; p += gsize) {
    const int n = find(first, a.N, (int)p);
    const int have = (int)(((int64_t)a.lens[n] + ps1) >> a.page_shift);
    a.block_table[(int64_t)n * a.max_blocks + have + ((int)p - first[n])] = a.free_pages[p];
  }
  // the tokens, four in a row per thread
  for (int64_t t4 = gtid * 4; t4 < a.T; t4 += gsize * 4) {
    int n = find(cu, a.N, (int)t4);
    int32_t pos[4], slot[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = (int)t4 + e;
      pos[e] = slot[e] = -1;
      if (t < a.T) {
        while (cu[n + 1] <= t) ++n;
        const int l = a.lens[n], have = (int)(((int64_t)l + ps1) >> a.page_shift);
        pos[e] = l + (t - cu[n]);
        const int b = pos[e] >> a.page_shift;
        const int page = b < have ? a.block_table[(int64_t)n * a.max_blocks + b] : a.free_pages[first[n] + (b - have)];
        if (page_ok(page, a.page_shift)) slot[e] = (page << a.page_shift) + (pos[e] & ps1);
      }
    }
    if (t4 + 4 <= a.T) {
      *reinterpret_cast<int4*>(a.positions + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.slot_map + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
      for (int e = 0; t4 + e < a.T; ++e) {
        a.positions[t4 + e] = pos[e];
        a.slot_map[t4 + e] = slot[e];
      }
    }
  }
  // the error word: the pages that tokens of this step lie on
  if (blockIdx.x == 0) {
    bool bad = false;
    for (int64_t p = tid; p < pg_all; p += kMapThreads) bad |= !page_ok(a.free_pages[p], a.page_shift);
    for (int n = tid; n < a.N; n += kMapThreads) {
      const int l = a.lens[n];
      if ((l & ps1) && cu[n + 1] > cu[n])
        bad |= !page_ok(a.block_table[(int64_t)n * a.max_blocks + (l >> a.page_shift)], a.page_shift);
    }
    const int any = __syncthreads_or(bad);
    if (tid == 0) a.hdr->err = any ? GDN_DEVERR_PAGES : 0;
  }
}

}  // namespace

void launch_norm_rope(const NormRope& a, int d, bool in_bf16, bool out_bf16, cudaStream_t st) {
#define CALL(D)                                                                          \
  if (in_bf16 && out_bf16) norm_rope_t<D, __nv_bfloat16, __nv_bfloat16>(a, st);          \
  else if (in_bf16) norm_rope_t<D, __nv_bfloat16, float>(a, st);                         \
  else if (out_bf16) norm_rope_t<D, float, __nv_bfloat16>(a, st);                        \
  else norm_rope_t<D, float, float>(a, st)
  GDN_BY_D(d, CALL)
#undef CALL
}

int launch_norm_rope_bwd(const NormRope& a, int d, bool in_bf16, bool grad_bf16, cudaStream_t st) {
#define CALL(D)                                                                              \
  if (in_bf16 && grad_bf16) norm_rope_bwd_t<D, __nv_bfloat16, __nv_bfloat16>(a, st);         \
  else if (in_bf16) norm_rope_bwd_t<D, __nv_bfloat16, float>(a, st);                         \
  else if (grad_bf16) norm_rope_bwd_t<D, float, __nv_bfloat16>(a, st);                       \
  else norm_rope_bwd_t<D, float, float>(a, st)
  GDN_BY_D(d, CALL)
#undef CALL
  return a.partial ? 2 : 1;
}

void launch_page_map(const PageMap& a, cudaStream_t st) {
  const size_t smem = 2 * sizeof(int32_t) * ((size_t)a.N + 1);
  static std::atomic<uint64_t> ready{0};
  ensure_smem(k_page_map, 2 * (int)sizeof(int32_t) * (kPageMapMaxSeqs + 1), ready);
  int64_t blocks = ((int64_t)a.T + 4 * kMapThreads - 1) / (4 * kMapThreads);
  blocks = blocks < 1 ? 1 : blocks > 152 ? 152 : blocks;
  k_page_map<<<(unsigned)blocks, kMapThreads, smem, st>>>(a);
}

}  // namespace gdn
