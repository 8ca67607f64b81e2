// attn_tokens.cu -- the attention layer's per-token operators: norms of queries and keys with
// the rotation in the same pass (and its gradient), and the paged cache's bookkeeping.
#include "attn.h"

namespace gdn {

namespace {

// =====================================================================================
// Norm and rotation.  One row is one head of one token; LPR = D / 8 lanes hold two pieces of 4
// consecutive entries each, chosen so that the half layout's pairs (i, i + rot / 2) lie in one lane:
// a lane of the rotated part holds pieces at A and A + rot / 2, one of the rest at A and
// A + (D - rot) / 2.  The interleaved layout's pairs lie within a piece.  So the rotation needs no
// exchange, and the norm log2(LPR) shuffles.  A warp holds GPW = 32 / LPR rows at a time and U of
// these at once (their loads are issued together).  A warp takes one token's U * GPW heads of q, of
// k or of v, so that nothing inside depends on which it is, and the few rows of
// a decode step spread over warps.  With two pieces a lane the kernel issues half the instructions per row that one
// piece costs, and packed pairs halve the arithmetic again; before both it was bound by issue.
// 16384 tokens of 32 / 8 heads, d = 128, with the cache written: 202 us before, 85.5 now, 5.15 TB/s
// (77% of a copy's rate), bound by the bytes and what is left of their latency.
// =====================================================================================
constexpr int kNormThreads = 128;

template <int D>
struct RowLanes {
  static constexpr int LPR = D / 8, GPW = 32 / LPR;
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

struct Row8 {  // a lane's two pieces of a row: pairs 0, 1 of the first, 2, 3 of the second
  float2 p[4];
};
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ Row8 all8(float x) {
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = make_float2(x, x);
  return r;
}
__device__ __forceinline__ Row8 mul8(const Row8& x, const Row8& y) {
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = mul2(x.p[i], y.p[i]);
  return r;
}
__device__ __forceinline__ Row8 fma8(const Row8& x, const Row8& y, const Row8& z) {
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = fma2(x.p[i], y.p[i], z.p[i]);
  return r;
}
__device__ __forceinline__ float dot8(const Row8& x, const Row8& y) {
  const float2 s = add2(fma2(x.p[1], y.p[1], mul2(x.p[0], y.p[0])), fma2(x.p[3], y.p[3], mul2(x.p[2], y.p[2])));
  return __fadd_rn(s.x, s.y);
}
// the entries that a rotation adds to each: the other piece (half), the pair's other one (interleaved)
__device__ __forceinline__ Row8 partners(const Row8& x, bool half) {
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = half ? x.p[i ^ 2] : make_float2(x.p[i].y, x.p[i].x);
  return r;
}
__device__ __forceinline__ Row8 pick8(bool first, const Row8& x, const Row8& y) {
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.p[i] = make_float2(first ? x.p[i].x : y.p[i].x, first ? x.p[i].y : y.p[i].y);
  return r;
}
constexpr float kNan = __builtin_nanf("");
template <typename T>
__device__ __forceinline__ Row8 load8p(const T* p, int gap) {
  const float4 a = load4(p), b = load4(p + gap);
  Row8 r;
  r.p[0] = make_float2(a.x, a.y), r.p[1] = make_float2(a.z, a.w);
  r.p[2] = make_float2(b.x, b.y), r.p[3] = make_float2(b.z, b.w);
  return r;
}
template <typename T>
__device__ __forceinline__ void store8p(T* p, int gap, const Row8& x) {
  store4(p, make_float4(x.p[0].x, x.p[0].y, x.p[1].x, x.p[1].y));
  store4(p + gap, make_float4(x.p[2].x, x.p[2].y, x.p[3].x, x.p[3].y));
}

// 1 / sqrt of the norm's sum of squares (plus eps); 1 without a norm
__device__ __forceinline__ float inverse_norm(int norm, float sumsq, float inv_d, float eps) {
  if (norm == GDN_NORM_NONE) return 1.f;
  return rsqrtf(__fadd_rn(norm == GDN_NORM_RMS ? __fmul_rn(sumsq, inv_d) : sumsq, eps));
}

// Where a lane's pieces start, and whether they turn.
struct Pieces {
  int at, gap;  // at `at` and at + gap
  bool on;
};
template <int D>
__device__ __forceinline__ Pieces pieces_of(const NormRope& a, int lane) {
  const int l = lane % (D / 8);
  Pieces t;
  t.on = l < a.rot / 8;
  t.at = t.on ? 4 * l : a.rot + 4 * (l - a.rot / 8);
  t.gap = t.on ? a.rot / 2 : (D - a.rot) / 2;
  return t;
}
// cos, and sin with the sign of the entry's place in its pair (-, +) times `sign`; 1 and 0 where
// nothing turns
__device__ __forceinline__ void angles_of(const NormRope& a, int64_t row, float sign, const Pieces& t, bool half, Row8& c,
                                          Row8& s) {
  c = all8(1.f);
  s = all8(0.f);
  if (!t.on) return;
  const float *cp = a.cos + row * (a.rot / 2), *sp = a.sin + row * (a.rot / 2);
  if (half) {
    const float4 c4 = *reinterpret_cast<const float4*>(cp + t.at), s4 = *reinterpret_cast<const float4*>(sp + t.at);
    c.p[0] = c.p[2] = make_float2(c4.x, c4.y);
    c.p[1] = c.p[3] = make_float2(c4.z, c4.w);
    s.p[2] = make_float2(__fmul_rn(sign, s4.x), __fmul_rn(sign, s4.y));
    s.p[3] = make_float2(__fmul_rn(sign, s4.z), __fmul_rn(sign, s4.w));
    s.p[0] = make_float2(-s.p[2].x, -s.p[2].y);
    s.p[1] = make_float2(-s.p[3].x, -s.p[3].y);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 cc = *reinterpret_cast<const float2*>(cp + (t.at + i * t.gap) / 2);
      const float2 ss = *reinterpret_cast<const float2*>(sp + (t.at + i * t.gap) / 2);
      c.p[2 * i] = make_float2(cc.x, cc.x);
      c.p[2 * i + 1] = make_float2(cc.y, cc.y);
      s.p[2 * i] = make_float2(-__fmul_rn(sign, ss.x), __fmul_rn(sign, ss.x));
      s.p[2 * i + 1] = make_float2(-__fmul_rn(sign, ss.y), __fmul_rn(sign, ss.y));
    }
  }
}

// A run of RUN heads: which of q (0), k (1), v (2), and its first head.
struct HeadRun {
  int kind, h0, heads;
};
template <int RUN>
int head_runs(int hq, int hk, int hv) {
  return (hq + RUN - 1) / RUN + (hk + RUN - 1) / RUN + (hv + RUN - 1) / RUN;
}
template <int RUN>
__device__ __forceinline__ HeadRun head_run(const NormRope& a, int c) {
  const int nq = (a.hq + RUN - 1) / RUN, nk = (a.hk + RUN - 1) / RUN;
  HeadRun r;
  r.kind = c < nq ? 0 : c < nq + nk ? 1 : 2;
  r.h0 = (c - (r.kind == 0 ? 0 : r.kind == 1 ? nq : nq + nk)) * RUN;
  r.heads = r.kind == 0 ? a.hq : a.hk;
  return r;
}

// Eight blocks an SM (64 registers, which spill 80 to 92 bytes a thread where U = 4): with six, which do not, the
// prefill case took 92 us instead of 85.5, with nine, which spill more, 100.
template <int D, typename TI, typename TO, int U>
__global__ void __launch_bounds__(kNormThreads, U > 1 ? 8 : 1) k_norm_rope(const NormRope a, const int runs) {
  constexpr int LPR = RowLanes<D>::LPR, GPW = RowLanes<D>::GPW;
  const int lane = threadIdx.x & 31;
  // a token's runs of heads in neighbouring blocks: their rows are neighbours in memory
  const int64_t t = (int64_t)(blockIdx.x / runs) * (kNormThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const HeadRun it = head_run<U * GPW>(a, blockIdx.x % runs);
  const int h = it.h0 + lane / LPR;
  const Pieces pc = pieces_of<D>(a, lane);
  // what other loads wait for comes first
  const int64_t p = a.rot && it.kind < 2 ? a.pos[t] : 0;
  const int64_t slot = it.kind && a.slot_map ? a.slot_map[t] : -1;
  const TI* src = (it.kind == 0 ? static_cast<const TI*>(a.q) + t * a.q_stride
                   : it.kind == 1 ? static_cast<const TI*>(a.k) + t * a.k_stride
                                  : static_cast<const TI*>(a.v) + t * a.v_stride) + h * D + pc.at;
  Row8 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) x[u] = h + u * GPW < it.heads ? load8p(src + u * GPW * D, pc.gap) : all8(0.f);
  const bool bad = a.rot && (p < 0 || p >= a.table_rows), half = a.layout == GDN_ROPE_HALF;
  Row8 c, s;
  angles_of(a, bad ? 0 : p, 1.f, pc, half, c, s);
  // the cache's cell of head h
  TO* cell = nullptr;
  const int64_t ps = (int64_t)1 << a.page_shift;
  if (it.kind) {
    if (slot >= 0 && slot < a.slots)
      cell = static_cast<TO*>(it.kind == 1 ? a.k_pages : a.v_pages) +
             (((slot >> a.page_shift) * a.hk + h) * ps + (slot & (ps - 1))) * D + pc.at;
  }
  if (it.kind == 2) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (cell && h + u * GPW < it.heads) store8p(cell + u * GPW * ps * D, pc.gap, x[u]);
    return;
  }
  const float* wp = it.kind ? a.wk : a.wq;
  const Row8 w = wp ? load8p(wp + pc.at, pc.gap) : all8(1.f);
  // y = r (x (w c) + partner (w' s)), w' the partner's weight
  c = mul8(w, c);
  s = mul8(partners(w, half), s);
  const bool some_off = a.rot < D;
  TO* dst = static_cast<TO*>(it.kind ? a.k_out : a.q_out);
  if (dst) dst += (t * it.heads + h) * D + pc.at;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float r = inverse_norm(a.norm, row_sum<LPR>(dot8(x[u], x[u])), 1.f / D, a.eps);
    Row8 y = mul8(x[u], c);
    if (a.rot) {
      const Row8 z = fma8(partners(x[u], half), s, y);
      y = some_off ? pick8(pc.on, z, y) : z;  // 0 x infinity stays out of what does not turn
    }
    y = mul8(y, all8(r));
    if (bad) y = all8(kNan);
    if (h + u * GPW < it.heads) {
      if (dst) store8p(dst + u * GPW * D, pc.gap, y);
      if (cell) store8p(cell + u * GPW * ps * D, pc.gap, y);
    }
  }
}

// Backward: dx per row, and with weights the sums of g x r over this block's items: each lane
// adds its 8 columns in the order of the tokens it meets, then the block's rows of lanes in
// ascending order; k_norm_rope_dw adds the blocks.  Forward and gradient of 16384 tokens of 32 / 8 heads,
// d = 128, rotated, with weights, bf16: 183 us (3.7 TB/s), 213 with two row sets at a time on five blocks an
// SM instead of four on four: what bounds it is how many loads are in flight, and registers bound
// those.
template <int D, typename TI, typename TG, int U, bool W>
__global__ void __launch_bounds__(kNormThreads, 4) k_norm_rope_bwd(const NormRope a, const int runs) {
  constexpr int LPR = RowLanes<D>::LPR, GPW = RowLanes<D>::GPW;
  const int lane = threadIdx.x & 31;
  const int block = blockIdx.x / runs, blocks = gridDim.x / runs;  // of this run of heads
  const HeadRun it = head_run<U * GPW>(a, blockIdx.x % runs);
  const int h = it.h0 + lane / LPR;
  const Pieces pc = pieces_of<D>(a, lane);
  const bool half = a.layout == GDN_ROPE_HALF, some_off = a.rot < D;
  const float* wp = it.kind ? a.wk : a.wq;
  const Row8 w = W && wp ? load8p(wp + pc.at, pc.gap) : all8(1.f);
  const float cn = a.norm == GDN_NORM_RMS ? 1.f / D : a.norm == GDN_NORM_L2 ? 1.f : 0.f;
  Row8 acc = all8(0.f);
  const int64_t step = (int64_t)blocks * (kNormThreads / 32);
  int64_t t = (int64_t)block * (kNormThreads / 32) + (threadIdx.x >> 5);
  int next_p = a.rot && t < a.T ? a.pos[t] : 0;
  for (; t < a.T; t += step) {
    const int p = next_p;
    if (a.rot && t + step < a.T) next_p = a.pos[t + step];  // a turn ahead: the angles wait for it
    const int64_t at = (t * it.heads + h) * D + pc.at;
    const TI* src = (it.kind ? static_cast<const TI*>(a.k) + t * a.k_stride
                             : static_cast<const TI*>(a.q) + t * a.q_stride) + h * D + pc.at;
    const TG* gsrc = static_cast<const TG*>(it.kind ? a.gk : a.gq) + at;
    TI* dst = static_cast<TI*>(it.kind ? a.dk : a.dq) + at;
    Row8 x[U], g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = h + u * GPW < it.heads;
      x[u] = in ? load8p(src + u * GPW * D, pc.gap) : all8(0.f);
      g[u] = in ? load8p(gsrc + u * GPW * D, pc.gap) : all8(0.f);
    }
    const bool bad = a.rot && (p < 0 || p >= a.table_rows);
    Row8 c, s;
    angles_of(a, bad ? 0 : p, -1.f, pc, half, c, s);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (a.rot) {
        const Row8 z = fma8(partners(g[u], half), s, mul8(g[u], c));
        g[u] = some_off ? pick8(pc.on, z, g[u]) : z;
      }
      const Row8 gw = W ? mul8(g[u], w) : g[u];
      const float r = inverse_norm(a.norm, row_sum<LPR>(dot8(x[u], x[u])), 1.f / D, a.eps);
      const float xg = row_sum<LPR>(dot8(x[u], gw));
      const float f = -__fmul_rn(__fmul_rn(cn, __fmul_rn(r, __fmul_rn(r, r))), xg);
      Row8 dx = fma8(all8(f), x[u], mul8(gw, all8(r)));
      if (bad) dx = all8(kNan);
      if (h + u * GPW < it.heads) {
        store8p(dst + u * GPW * D, pc.gap, dx);
        if (W && !bad) acc = fma8(g[u], mul8(x[u], all8(r)), acc);
      }
    }
  }
  if (!W || !a.partial) return;
  constexpr int NR = kNormThreads / LPR;  // rows of lanes in the block
  __shared__ float sh[NR][D];
  store8p(&sh[threadIdx.x / LPR][pc.at], pc.gap, acc);
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kNormThreads) {
    float sum = 0.f;
#pragma unroll 8
    for (int r = 0; r < NR; ++r) sum = __fadd_rn(sum, sh[r][e]);
    a.partial[((int64_t)(blockIdx.x % runs) * blocks + block) * D + e] = sum;
  }
}

// dw[e] = sum over blocks of partial[block][e]: those of q's runs come first, then k's (blockIdx.y).  8 columns per
// CTA, 32 threads a column with ascending strided sums, then a fixed tree.
__global__ void __launch_bounds__(256) k_norm_rope_dw(const float* __restrict__ partial, int q_blocks, int k_blocks, int D,
                                                      float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sh[8][33];
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3, e = blockIdx.x * 8 + c;
  const int first = blockIdx.y ? q_blocks : 0, blocks = blockIdx.y ? k_blocks : q_blocks;
  float s = 0.f;
#pragma unroll 4
  for (int b = r; b < blocks; b += 32) s = __fadd_rn(s, partial[(int64_t)(first + b) * D + e]);
  sh[c][r] = s;
  __syncthreads();
  float x = sh[threadIdx.x >> 5][threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) (blockIdx.y ? dwk : dwq)[blockIdx.x * 8 + (threadIdx.x >> 5)] = x;
}

template <int D, typename TI, typename TO>
void norm_rope_t(const NormRope& a, cudaStream_t st) {
  // Few rows: one row set per warp, which ends sooner (4 tokens of 16 / 2 heads: 2.1 us against 2.8; 256 of
  // 16 / 4: 2.6 against 3.2); from about 8 warps a scheduler on, four at once keep more loads in
  // flight (1024 tokens of 16 / 4 heads: 4.2 us against 5.2; 16384 of 32 / 8: 85.6 against 158).
  constexpr int GPW = RowLanes<D>::GPW, WARPS = kNormThreads / 32;
  const int hv = a.v_pages ? a.hk : 0;
  const unsigned x = (unsigned)(((int64_t)a.T + WARPS - 1) / WARPS);
  const int runs = head_runs<GPW>(a.hq, a.hk, hv);
  if ((int64_t)a.T * runs <= 152 * 32)
    k_norm_rope<D, TI, TO, 1><<<x * runs, kNormThreads, 0, st>>>(a, runs);
  else {
    const int r4 = head_runs<4 * GPW>(a.hq, a.hk, hv);
    k_norm_rope<D, TI, TO, 4><<<x * r4, kNormThreads, 0, st>>>(a, r4);
  }
}

template <int D, typename TI, typename TG>
void norm_rope_bwd_t(const NormRope& a, cudaStream_t st) {
  constexpr int U = 4, RUN = U * RowLanes<D>::GPW, WARPS = kNormThreads / 32;
  const int nq = head_runs<RUN>(a.hq, 0, 0), runs = head_runs<RUN>(a.hq, a.hk, 0);
  int64_t x = ((int64_t)a.T + WARPS - 1) / WARPS;
  if (a.partial) {
    const int64_t most = kNormBwdBlocks / runs > 1 ? kNormBwdBlocks / runs : 1;
    if (x > most) x = most;
  }
  const unsigned grid = (unsigned)(x * runs);
  if (a.wq || a.wk || a.partial)
    k_norm_rope_bwd<D, TI, TG, U, true><<<grid, kNormThreads, 0, st>>>(a, runs);
  else
    k_norm_rope_bwd<D, TI, TG, U, false><<<grid, kNormThreads, 0, st>>>(a, runs);
  if (a.partial)
    k_norm_rope_dw<<<dim3(D / 8, 2), 256, 0, st>>>(a.partial, nq * (int)x, (runs - nq) * (int)x, D, a.dwq, a.dwk);
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
