// attn_window.cu -- sliding-window attention and its gradient on fp32 SIMT: fp32 inputs (whose
// products stay in 32 bits) and bf16 ones with d = 32.  bf16 with d = 64 or 128 runs on the
// tensor cores (attn_window_tc.cu).
//
// Tiles of 16 R rows x 64 columns (queries x keys, or keys x queries for dk, dv) in shared memory
// (rows padded by 4 floats, so that 16-byte reads of 8 neighbouring rows meet 8 different bank
// groups), 256 threads; a thread (ty, tx) of 16 x 16 owns scores (R ty + r, 16 c + tx) and, of a
// 16 R x D accumulator, rows R ty + r and columns 4 tx + 64 c .. + 3.  Products run on packed pairs
// (f32x2): the dots over pairs of columns, the accumulators over pairs of output columns, for which
// the probabilities lie doubled and transposed in shared memory, so that one 16-byte read gives
// the multipliers of two rows.  One pass over the keys with a running maximum and sum per row.
// The gradient is two kernels, each deterministic: per query block dq (and do . o, which the
// other needs), per key block dk and dv, where a cluster of CTAs shares out the group's heads and
// adds its sums in ascending order through its shared memory; before them, for bf16, k_window_delta.
// (One CTA per key block, head after head, took 77 us in the first case below, whose 39 blocks of 2 key
// heads leave half of the SMs without one; 8 x 2048 tokens took 3.67 ms in all instead of 3.01.)
// R is 4, or 2 where 64-row tiles would leave SMs without work: a row's arithmetic is the same in
// both (the column blocks do not move), so its bits do not depend on the choice.
// Forward and gradient, fp32, d = 64: 7 sequences of 54 to 271 tokens, 4 / 2 heads, 80 us with R = 2, 113
// with 4; 4 of 512, 8 / 2 heads, 327 against 315 (near the rule's edge); 8 of 2048, window 512, 3.48 ms
// against 3.01 with R = 4.
// The short cases are bound by the latency of a tile's chain of products, barriers and exchanges,
// the long ones by shared memory's reads beside the fp32 units.
#include "attn_window.cuh"
#include "tc.cuh"

namespace gdn {

namespace {

using namespace win;

constexpr int BN = 64, kThreads = 256;  // columns of a tile

template <int D>
__host__ __device__ constexpr int pitch() {
  return D + 4;
}

// row stride of the doubled, transposed probabilities of `rows` rows
template <int R>
__host__ __device__ constexpr int pp() {
  return 2 * 16 * R + 4;
}

// rows [row0, row0 + ROWS) of [rows, H, D] at head h into a tile; rows at or past `end` are zeros
template <int D, typename T, int ROWS>
__device__ __forceinline__ void load_tile(float* tile, const void* src, int64_t base, int row0, int end, int H, int h) {
  constexpr int V = D / 4;
  for (int e = threadIdx.x; e < ROWS * V; e += kThreads) {
    const int r = e / V, c = 4 * (e % V);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + r < end) x = load4(static_cast<const T*>(src) + ((base + row0 + r) * H + h) * D + c);
    *reinterpret_cast<float4*>(tile + r * pitch<D>() + c) = x;
  }
}

// The next column tile on its way in registers while the present one is worked on.
template <int D, typename T>
struct NextTile {
  static constexpr int V = D / 4, N = 64 * V / kThreads;
  float4 x[N];
  __device__ __forceinline__ void fetch(const void* src, int64_t base, int row0, int end, int H, int h) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int e = k * kThreads + threadIdx.x, r = e / V, c = 4 * (e % V);
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row0 + r < end) x[k] = load4(static_cast<const T*>(src) + ((base + row0 + r) * H + h) * D + c);
    }
  }
  __device__ __forceinline__ void put(float* tile) const {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int e = k * kThreads + threadIdx.x;
      *reinterpret_cast<float4*>(tile + (e / V) * pitch<D>() + 4 * (e % V)) = x[k];
    }
  }
};

// x[r][c] = a_row(R ty + r) . b_row(16 c + tx)
template <int D, int R>
__device__ __forceinline__ void rows_dot(const float* A, const float* B, int ty, int tx, float (&x)[R][4]) {
  float2 acc[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[r][c] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < D; k += 4) {
    float4 a[R], b[4];
#pragma unroll
    for (int r = 0; r < R; ++r) a[r] = *reinterpret_cast<const float4*>(A + (R * ty + r) * pitch<D>() + k);
#pragma unroll
    for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4*>(B + (16 * c + tx) * pitch<D>() + k);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[r][c] = fma2(make_float2(a[r].x, a[r].y), make_float2(b[c].x, b[c].y), acc[r][c]);
        acc[r][c] = fma2(make_float2(a[r].z, a[r].w), make_float2(b[c].z, b[c].w), acc[r][c]);
      }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) x[r][c] = __fadd_rn(acc[r][c].x, acc[r][c].y);
}

// the thread's values of a tile, doubled, into the transposed place [column][row]
template <int R>
__device__ __forceinline__ void put_doubled(float* P, int ty, int tx, const float (&x)[R][4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int r = 0; r < R; r += 2)
      *reinterpret_cast<float4*>(P + (16 * c + tx) * pp<R>() + 2 * (R * ty + r)) =
          make_float4(x[r][c], x[r][c], x[r + 1][c], x[r + 1][c]);
}

template <int D, int R>
struct Acc {  // R rows x (D / 64 float4 columns; half of the lanes at D = 32)
  static constexpr int C = D >= 64 ? D / 64 : 1;
  float4 v[R][C];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) v[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ static bool mine(int tx) { return D >= 64 || tx < D / 4; }
  // += P[R ty + r][n] * B[n][cols], n = 0 .. 63, P as put_doubled leaves it
  __device__ __forceinline__ void add(const float* P, const float* B, int ty, int tx) {
    if (!mine(tx)) return;
#pragma unroll 4
    for (int n = 0; n < 64; ++n) {
      float2 p[R];
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        const float4 x = *reinterpret_cast<const float4*>(P + n * pp<R>() + 2 * (R * ty + r));
        p[r] = make_float2(x.x, x.y);
        p[r + 1] = make_float2(x.z, x.w);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float4 b = *reinterpret_cast<const float4*>(B + n * pitch<D>() + 4 * tx + 64 * c);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float2 lo = fma2(p[r], make_float2(b.x, b.y), make_float2(v[r][c].x, v[r][c].y));
          const float2 hi = fma2(p[r], make_float2(b.z, b.w), make_float2(v[r][c].z, v[r][c].w));
          v[r][c] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(void* dst, int64_t base, int row0, int end, int H, int h, int ty, int tx,
                                        const float (&f)[R]) const {
    if (!mine(tx)) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = row0 + R * ty + r;
      if (row >= end) continue;
#pragma unroll
      for (int c = 0; c < C; ++c)
        store4(static_cast<T*>(dst) + ((base + row) * H + h) * D + 4 * tx + 64 * c,
               make_float4(__fmul_rn(v[r][c].x, f[r]), __fmul_rn(v[r][c].y, f[r]), __fmul_rn(v[r][c].z, f[r]),
                           __fmul_rn(v[r][c].w, f[r])));
    }
  }
};

// over the 16 lanes of a row of threads
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float row_add(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

template <int D, typename T, int R>
__global__ void __launch_bounds__(kThreads) k_window_fwd(const WindowAttn a) {
  extern __shared__ float sh[];
  constexpr int BM = 16 * R, ROWS = BM * pitch<D>(), COLS = BN * pitch<D>();
  float *Qs = sh, *Ks = Qs + ROWS, *Vs = Ks + COLS, *Ps = Vs + COLS;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_tables(a);
  // a sequence's last blocks see the most keys: they start first
  int row0;
  const Seq q = find_seq(a, (int64_t)gridDim.x - 1 - blockIdx.x, BM, false, row0);
  if (!q.ok) return;
  const int h = blockIdx.y, kvh = h / (a.hq / a.hkv), ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int p0 = row0 + q.Lk - q.Lq, p1 = min(row0 + BM, q.Lq) - 1 + q.Lk - q.Lq;
  const KeyBlocks kb(p0, p1, q.Lk, a.window, a.sinks, BN);
  load_tile<D, T, BM>(Qs, a.q, q.q0, row0, q.Lq, a.hq, h);
  const float sc = __fmul_rn(a.scale, kLog2e);
  float m[R], l[R];
  Acc<D, R> o;
  o.zero();
#pragma unroll
  for (int r = 0; r < R; ++r) m[r] = -INFINITY, l[r] = 0.f;
  NextTile<D, T> kn, vn;
  if (kb.count()) {
    kn.fetch(a.k, q.k0, kb.block(0) * BN, q.Lk, a.hkv, kvh);
    vn.fetch(a.v, q.k0, kb.block(0) * BN, q.Lk, a.hkv, kvh);
  }
  for (int b = 0; b < kb.count(); ++b) {
    const int j0 = kb.block(b) * BN;
    __syncthreads();
    kn.put(Ks);
    vn.put(Vs);
    __syncthreads();
    if (b + 1 < kb.count()) {
      kn.fetch(a.k, q.k0, kb.block(b + 1) * BN, q.Lk, a.hkv, kvh);
      vn.fetch(a.v, q.k0, kb.block(b + 1) * BN, q.Lk, a.hkv, kvh);
    }
    float x[R][4];
    rows_dot<D, R>(Qs, Ks, ty, tx, x);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int p = p0 + R * ty + r;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[r][c] = visible(p, j0 + 16 * c + tx, a.window, a.sinks) ? __fmul_rn(x[r][c], sc) : -INFINITY;
        mx = fmaxf(mx, x[r][c]);
      }
      mx = fmaxf(m[r], row_max(mx));
      const float base = mx == -INFINITY ? 0.f : mx;  // a row that has seen nothing yet
      const float alpha = exp2_approx(__fsub_rn(m[r], base));
      m[r] = mx;
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p_ = exp2_approx(__fsub_rn(x[r][c], base));
        s = __fadd_rn(s, p_);
        x[r][c] = p_;
      }
      l[r] = __fmaf_rn(l[r], alpha, s);
#pragma unroll
      for (int c = 0; c < (Acc<D, R>::C); ++c) {
        float4& v = o.v[r][c];
        v = make_float4(__fmul_rn(v.x, alpha), __fmul_rn(v.y, alpha), __fmul_rn(v.z, alpha), __fmul_rn(v.w, alpha));
      }
    }
    put_doubled<R>(Ps, ty, tx, x);
    __syncwarp();  // a row's place is written and read by the same 16 lanes
    o.add(Ps, Vs, ty, tx);
  }
  float inv[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float s = row_add(l[r]);
    inv[r] = s > 0.f ? __frcp_rn(s) : s == 0.f ? 0.f : s;  // a row that sees nothing: zeros; NaN stays
    const int row = row0 + R * ty + r;
    if (tx == 0 && row < q.Lq)
      a.lse[(int64_t)(q.q0 + row) * a.hq + h] = s == 0.f ? -INFINITY : __fmul_rn(__fadd_rn(m[r], log2f(s)), kLn2);
  }
  o.template store<T>(a.out, q.q0, row0, q.Lq, a.hq, h, ty, tx, inv);
}

// p and ds / scale of one tile: p = exp(scale q.k - lse), ds = p (do.v - delta), zero where
// nothing is visible.  x holds q.k on entry and p on return, y do.v and then ds.
template <int R>
__device__ __forceinline__ void grad_scores(const WindowAttn& a, float sc, const int* pos, const int* key, const float* lse2,
                                            const float* delta, bool rows_are_queries, float (&x)[R][4], float (&y)[R][4]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int qi = rows_are_queries ? r : c, ki = rows_are_queries ? c : r;
      const bool see = visible(pos[qi], key[ki], a.window, a.sinks) && lse2[qi] != -INFINITY;
      const float p = see ? exp2_approx(__fsub_rn(__fmul_rn(x[r][c], sc), lse2[qi])) : 0.f;
      y[r][c] = see ? __fmul_rn(p, __fsub_rn(y[r][c], delta[qi])) : 0.f;
      x[r][c] = p;
    }
}

template <int D, typename T, int R>
__global__ void __launch_bounds__(kThreads) k_window_dq(const WindowAttn a) {
  extern __shared__ float sh[];
  constexpr int BM = 16 * R, ROWS = BM * pitch<D>(), COLS = BN * pitch<D>();
  float *Qs = sh, *Os = Qs + ROWS, *Ks = Os + ROWS, *Vs = Ks + COLS, *Ps = Vs + COLS;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_tables(a);
  int row0;
  const Seq q = find_seq(a, (int64_t)gridDim.x - 1 - blockIdx.x, BM, false, row0);
  if (!q.ok) return;
  const int h = blockIdx.y, kvh = h / (a.hq / a.hkv), ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int p0 = row0 + q.Lk - q.Lq, p1 = min(row0 + BM, q.Lq) - 1 + q.Lk - q.Lq;
  const KeyBlocks kb(p0, p1, q.Lk, a.window, a.sinks, BN);
  load_tile<D, T, BM>(Qs, a.q, q.q0, row0, q.Lq, a.hq, h);
  load_tile<D, T, BM>(Os, a.dout, q.q0, row0, q.Lq, a.hq, h);
  load_tile<D, T, BM>(Ks, a.out, q.q0, row0, q.Lq, a.hq, h);
  __syncthreads();
  const float sc = __fmul_rn(a.scale, kLog2e);
  int pos[R];
  float lse2[R], delta[R];
  Acc<D, R> dq;
  dq.zero();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = R * ty + r;
    float s = 0.f;
    if (Acc<D, R>::mine(tx))
#pragma unroll
      for (int c = 0; c < (Acc<D, R>::C); ++c) {
        const float4 o = *reinterpret_cast<const float4*>(Ks + row * pitch<D>() + 4 * tx + 64 * c);
        const float4 g = *reinterpret_cast<const float4*>(Os + row * pitch<D>() + 4 * tx + 64 * c);
        s = __fmaf_rn(o.w, g.w, __fmaf_rn(o.z, g.z, __fmaf_rn(o.y, g.y, __fmaf_rn(o.x, g.x, s))));
      }
    delta[r] = row_add(s);
    pos[r] = p0 + row;
    lse2[r] = -INFINITY;
    if (row0 + row < q.Lq) {
      const int64_t at = (int64_t)(q.q0 + row0 + row) * a.hq + h;
      lse2[r] = __fmul_rn(a.lse[at], kLog2e);
      if (sizeof(T) == 2 && few_keys(pos[r], a.few)) delta[r] = a.delta[at];
      else if (tx == 0) a.delta[at] = delta[r];
    }
  }
  NextTile<D, T> kn, vn;
  if (kb.count()) {
    kn.fetch(a.k, q.k0, kb.block(0) * BN, q.Lk, a.hkv, kvh);
    vn.fetch(a.v, q.k0, kb.block(0) * BN, q.Lk, a.hkv, kvh);
  }
  for (int b = 0; b < kb.count(); ++b) {
    const int j0 = kb.block(b) * BN;
    __syncthreads();
    kn.put(Ks);
    vn.put(Vs);
    __syncthreads();
    if (b + 1 < kb.count()) {
      kn.fetch(a.k, q.k0, kb.block(b + 1) * BN, q.Lk, a.hkv, kvh);
      vn.fetch(a.v, q.k0, kb.block(b + 1) * BN, q.Lk, a.hkv, kvh);
    }
    float x[R][4], y[R][4];
    rows_dot<D, R>(Qs, Ks, ty, tx, x);
    rows_dot<D, R>(Os, Vs, ty, tx, y);
    const int key[4] = {j0 + tx, j0 + 16 + tx, j0 + 32 + tx, j0 + 48 + tx};
    grad_scores<R>(a, sc, pos, key, lse2, delta, true, x, y);
    put_doubled<R>(Ps, ty, tx, y);
    __syncwarp();
    dq.add(Ps, Ks, ty, tx);
  }
  float f[R];
#pragma unroll
  for (int r = 0; r < R; ++r) f[r] = a.scale;
  dq.template store<T>(a.dq, q.q0, row0, q.Lq, a.hq, h, ty, tx, f);
}

// delta of the rows that see at most kFewKeys keys: delta = sum_j p_j (do . v_j) over the visible keys.  A CTA takes 16
// rows of a key head, whose keys (at most 31: 16 + window - 1 + first ones) lie in shared memory; a warp forms S = Q K^T
// and T = dO V^T of a query head on warp-level MMAs and sums over each row.  With a window and first tokens of at most
// kFewKeys together every row is such a row (16 to an item); else those at a sequence's first positions (an item per
// sequence).  dq's products start beside it.  The gradient with delta from the output everywhere, and so: packed training
// case (32387 tokens of 16 / 4 heads, window 2048) 1179 and 1175 us; 4 sequences of 512, 8 / 2 heads, 55.2 and 56.1; 64 of
// 20 to 40 tokens 41.6 and 45.2 (a chain of loads); 32768 tokens, window 12 and 4 first ones, 502 and 522 (lanes that form a
// row's products one after the other from shared memory instead took 1020).
template <int D>
__global__ void __launch_bounds__(256) k_window_delta(const WindowAttn a, const bool by_head) {
  asm volatile("griddepcontrol.launch_dependents;");  // dq's other warps may start
  const bool every_row = a.few > kFewKeys;
  constexpr int ROWS = 16, KEYS = 32, P = 2 * D + 16, KS = D / 16;  // P: bytes of a row; 8 of them in 8 bank groups
  __shared__ __align__(16) unsigned char ks[KEYS * P], vs[KEYS * P];
  using T = __nv_bfloat16;
  int row0;
  Seq q;
  if (every_row) {
    q = find_seq(a, blockIdx.x, ROWS, false, row0);
  } else {
    q.s = blockIdx.x;
    q.ok = valid_range(a.cu_q, q.s, a.Tq) && valid_range(a.cu_k, q.s, a.Tk);
    q.q0 = a.cu_q[q.s], q.Lq = a.cu_q[q.s + 1] - q.q0;
    q.k0 = a.cu_k[q.s], q.Lk = a.cu_k[q.s + 1] - q.k0;
    row0 = max(0, q.Lq - q.Lk);  // at position 0, or past it where keys lie before the queries
  }
  if (!q.ok || row0 >= q.Lq) return;
  const int p0 = row0 + q.Lk - q.Lq, p1 = min(row0 + ROWS, q.Lq) - 1 + q.Lk - q.Lq;  // positions of the rows
  if (p1 < 0 || !few_keys(max(p0, 0), a.few)) return;
  // place i holds key i (first ones) or lo + i - first
  const int first = every_row ? min(a.sinks, p1 + 1) : 0, lo = every_row ? max(first, p0 - a.window + 1) : 0;
  const int keys = min(every_row ? KEYS : kFewKeys, first + max(0, p1 + 1 - lo));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, group = a.hq / a.hkv;
  // this lane's rows: lane / 4 and 8 more
  const int ra = min(row0 + (lane >> 2), q.Lq - 1), rb = min(row0 + (lane >> 2) + 8, q.Lq - 1);
  uint32_t qa[KS][4], ga[KS][4];
  auto load = [&](int g) {
    const int64_t h = blockIdx.y * group + g;
    const int64_t xa = ((int64_t)(q.q0 + ra) * a.hq + h) * D + 2 * (lane & 3), xb = ((int64_t)(q.q0 + rb) * a.hq + h) * D + 2 * (lane & 3);
    const T *qp = static_cast<const T*>(a.q), *gp = static_cast<const T*>(a.dout);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t at = (e & 1 ? xb : xa) + 16 * k + 8 * (e >> 1);
        qa[k][e] = *reinterpret_cast<const uint32_t*>(qp + at);
        ga[k][e] = *reinterpret_cast<const uint32_t*>(gp + at);
      }
  };
  if (warp < group) load(warp);
  for (int e = threadIdx.x; e < keys * (D / 8); e += blockDim.x) {
    const int i = e / (D / 8), c = e % (D / 8), j = i < first ? i : lo + i - first;
    const int64_t at = ((int64_t)(q.k0 + j) * a.hkv + blockIdx.y) * D + 8 * c;
    *reinterpret_cast<uint4*>(ks + i * P + 16 * c) = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + at);
    *reinterpret_cast<uint4*>(vs + i * P + 16 * c) = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + at);
  }
  __syncthreads();
  const uint32_t at = tc::smem_u32(ks) + ((lane & 7) + ((lane >> 4) << 3)) * P + ((lane >> 3) & 1) * 16;
  const uint32_t to_v = tc::smem_u32(vs) - tc::smem_u32(ks);
  const float sc = __fmul_rn(a.scale, kLog2e);
  for (int g = warp; g < group; g += warps) {
    if (g != warp) load(g);
    float s[4][4], t[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = t[n][e] = 0.f;
#pragma unroll
    for (int n = 0; n < 4; n += 2) {
      if (8 * n >= keys) break;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t b[4];
        tc::ldsm_x4(at + 8 * n * P + 32 * k, b);
        tc::mma16816(s[n], qa[k], b[0], b[1]);
        tc::mma16816(s[n + 1], qa[k], b[2], b[3]);
        tc::ldsm_x4(at + to_v + 8 * n * P + 32 * k, b);
        tc::mma16816(t[n], ga[k], b[0], b[1]);
        tc::mma16816(t[n + 1], ga[k], b[2], b[3]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + (lane >> 2) + 8 * r, pos = row + q.Lk - q.Lq;
      float m = -INFINITY, l = 0.f, x = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 8 * n + 2 * (lane & 3) + e, j = i < first ? i : lo + i - first;
          float& y = s[n][2 * r + e];
          y = i < keys && visible(pos, j, a.window, a.sinks) ? __fmul_rn(y, sc) : -INFINITY;
          m = fmaxf(m, y);
        }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y = s[n][2 * r + e];
          const float p = y == -INFINITY ? 0.f : exp2_approx(__fsub_rn(y, m));
          l = __fadd_rn(l, p);
          x = y == -INFINITY ? x : __fmaf_rn(p, t[n][2 * r + e], x);
        }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, o));
        x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
      }
      if ((lane & 3) == 0 && row < q.Lq && few_keys(pos, a.few)) {
        const int64_t h = blockIdx.y * group + g;
        a.delta[by_head ? (a.hq + h) * a.Tq + q.q0 + row : (int64_t)(q.q0 + row) * a.hq + h] = __fdiv_rn(x, l);
      }
    }
  }
}

// CTAs of a key block: a power of two, from the group alone, so that it fixes the order of the sums
inline int dkv_cluster(int group) { return group >= 8 ? 8 : group >= 4 ? 4 : group >= 2 ? 2 : 1; }

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 load4_of(uint32_t smem, int rank) {
  float4 x;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}"
      : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
      : "r"(smem), "r"(rank)
      : "memory");
  return x;
}

template <int D, typename T, int R>
__global__ void __launch_bounds__(kThreads) k_window_dkv(const WindowAttn a, const int ctas) {
  extern __shared__ float sh[];
  constexpr int BM = 16 * R, ROWS = BM * pitch<D>(), COLS = BN * pitch<D>();
  float *Ks = sh, *Vs = Ks + ROWS, *Qs = Vs + ROWS, *Os = Qs + COLS, *Ps = Os + COLS, *Ds = Ps + 64 * pp<R>();
  int j0;
  const Seq q = find_seq(a, blockIdx.x, BM, true, j0);
  if (!q.ok) return;
  const int kvh = blockIdx.y / ctas, rank = blockIdx.y % ctas, group = a.hq / a.hkv;
  const int per = (group + ctas - 1) / ctas, h0 = rank * per, heads = max(0, min(per, group - h0));  // of this CTA
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  load_tile<D, T, BM>(Ks, a.k, q.k0, j0, q.Lk, a.hkv, kvh);
  load_tile<D, T, BM>(Vs, a.v, q.k0, j0, q.Lk, a.hkv, kvh);
  const QueryRange qr(q, j0, min(j0 + BM, q.Lk), a.window, a.sinks);
  const float sc = __fmul_rn(a.scale, kLog2e);
  const int off = q.Lk - q.Lq, b0 = qr.lo / BN, b1 = qr.hi > qr.lo ? (qr.hi + BN - 1) / BN : b0;
  int key[R];
#pragma unroll
  for (int r = 0; r < R; ++r) key[r] = j0 + R * ty + r;
  Acc<D, R> dk, dv;
  dk.zero();
  dv.zero();
  // column tiles: the query blocks of the heads, one head after the other
  const int nb = b1 - b0, tiles = nb * heads;
  NextTile<D, T> qn, on;
  float lse_n[4], delta_n[4];  // of the thread's columns
  auto fetch = [&](int i) {
    const int h = kvh * group + h0 + i / nb, row0 = (b0 + i % nb) * BN;
    qn.fetch(a.q, q.q0, row0, q.Lq, a.hq, h);
    on.fetch(a.dout, q.q0, row0, q.Lq, a.hq, h);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = row0 + 16 * c + tx;
      lse_n[c] = -INFINITY;
      delta_n[c] = 0.f;
      if (row < q.Lq) {
        const int64_t at = (int64_t)(q.q0 + row) * a.hq + h;
        lse_n[c] = a.lse[at];
        delta_n[c] = a.delta[at];
      }
    }
  };
  if (tiles) fetch(0);
  for (int i = 0; i < tiles; ++i) {
    const int row0 = (b0 + i % nb) * BN;
    __syncthreads();
    qn.put(Qs);
    on.put(Os);
    int pos[4];
    float lse2[4], delta[4], x[R][4], y[R][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      pos[c] = row0 + 16 * c + tx + off;
      lse2[c] = __fmul_rn(lse_n[c], kLog2e);
      delta[c] = delta_n[c];
    }
    __syncthreads();
    if (i + 1 < tiles) fetch(i + 1);
    rows_dot<D, R>(Ks, Qs, ty, tx, x);  // transposed: rows are keys
    rows_dot<D, R>(Vs, Os, ty, tx, y);
    grad_scores<R>(a, sc, pos, key, lse2, delta, false, x, y);
    put_doubled<R>(Ps, ty, tx, x);
    put_doubled<R>(Ds, ty, tx, y);
    __syncwarp();
    dv.add(Ps, Os, ty, tx);
    dk.add(Ds, Qs, ty, tx);
  }
  // the cluster's sums meet in its shared memory; each CTA adds and stores its share of them
  using A = Acc<D, R>;
  float4* mine = reinterpret_cast<float4*>(Qs);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < A::C; ++c) {
      mine[(r * A::C + c) * kThreads + threadIdx.x] = dk.v[r][c];
      mine[((R + r) * A::C + c) * kThreads + threadIdx.x] = dv.v[r][c];
    }
  cluster_sync();
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(mine + threadIdx.x);
  for (int s = rank; s < 2 * R * A::C; s += ctas) {
    const int r = s / A::C % R, c = s % A::C, row = j0 + R * ty + r;
    const bool k = s < R * A::C;
    float4 x = load4_of(at + s * kThreads * 16, 0);
    for (int o = 1; o < ctas && o * per < group; ++o) {
      const float4 y = load4_of(at + s * kThreads * 16, o);
      x = make_float4(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y), __fadd_rn(x.z, y.z), __fadd_rn(x.w, y.w));
    }
    const float f = k ? a.scale : 1.f;
    if (A::mine(tx) && row < q.Lk)
      store4(static_cast<T*>(k ? a.dk : a.dv) + ((int64_t)(q.k0 + row) * a.hkv + kvh) * D + 4 * tx + 64 * c,
             make_float4(__fmul_rn(x.x, f), __fmul_rn(x.y, f), __fmul_rn(x.z, f), __fmul_rn(x.w, f)));
  }
  cluster_sync();  // until all have read
}

template <void (*FN)(WindowAttn)>
void launch(dim3 grid, size_t floats, const WindowAttn& a, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  ensure_smem(FN, (int)(floats * sizeof(float)), ready);
  FN<<<grid, kThreads, floats * sizeof(float), st>>>(a);
}

// 32-row tiles where 64-row ones would make fewer than two CTAs per SM
inline bool small_tiles(int rows, int N, int heads) { return item_count(rows, 64, N) * heads < 2 * 152; }

template <int D, typename T, int R>
void fwd_r(const WindowAttn& a, cudaStream_t st) {
  launch<k_window_fwd<D, T, R>>(dim3((unsigned)item_count(a.Tq, 16 * R, a.N), a.hq),
                                (16 * R + 2 * 64) * pitch<D>() + 64 * pp<R>(), a, st);
}
template <int D, typename T, int R>
void dq_r(const WindowAttn& a, cudaStream_t st) {
  launch<k_window_dq<D, T, R>>(dim3((unsigned)item_count(a.Tq, 16 * R, a.N), a.hq),
                               (2 * 16 * R + 2 * 64) * pitch<D>() + 64 * pp<R>(), a, st);
}
template <int D, typename T, int R>
void dkv_r(const WindowAttn& a, cudaStream_t st) {
  constexpr size_t BYTES = ((2 * 16 * R + 2 * 64) * pitch<D>() + 2 * 64 * pp<R>()) * sizeof(float);
  static std::atomic<uint64_t> ready{0};
  ensure_smem(k_window_dkv<D, T, R>, (int)BYTES, ready);
  const int ctas = dkv_cluster(a.hq / a.hkv);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 1;
  attr.val.clusterDim.y = (unsigned)ctas;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)item_count(a.Tk, 16 * R, a.N), a.hkv * ctas);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = BYTES;
  c.stream = st;
  c.attrs = &attr;
  c.numAttrs = 1;
  cudaLaunchKernelEx(&c, k_window_dkv<D, T, R>, a, ctas);
}
template <int D, typename T>
void fwd_t(const WindowAttn& a, cudaStream_t st) {
  if (small_tiles(a.Tq, a.N, a.hq)) fwd_r<D, T, 2>(a, st); else fwd_r<D, T, 4>(a, st);
}
template <int D, typename T>
void dq_t(const WindowAttn& a, cudaStream_t st) {
  if (small_tiles(a.Tq, a.N, a.hq)) dq_r<D, T, 2>(a, st); else dq_r<D, T, 4>(a, st);
}
template <int D, typename T>
void dkv_t(const WindowAttn& a, cudaStream_t st) {
  if (small_tiles(a.Tk, a.N, a.hkv * dkv_cluster(a.hq / a.hkv))) dkv_r<D, T, 2>(a, st); else dkv_r<D, T, 4>(a, st);
}

}  // namespace

// bf16 with d = 64 or 128 runs on the tensor cores
#define GDN_BY_TYPE(f)                                  \
  if (bf16) f<32, __nv_bfloat16>(a, st);                \
  else if (a.d == 32) f<32, float>(a, st);              \
  else if (a.d == 64) f<64, float>(a, st);              \
  else f<128, float>(a, st);

bool launch_window_attn(const WindowAttn& a, bool bf16, cudaStream_t st) {
  if (bf16 && a.d != 32) return launch_window_fwd_tc(a, st);
  GDN_BY_TYPE(fwd_t)
  return true;
}
template <int D>
void delta_t(const WindowAttn& a, bool by_head, cudaStream_t st) {
  const int group = a.hq / a.hkv, threads = 32 * (group < 4 ? 4 : group < 8 ? group : 8);  // four to bring the keys in
  const dim3 grid((unsigned)(a.few > kFewKeys ? item_count(a.Tq, 16, a.N) : a.N), a.hkv);
  k_window_delta<D><<<grid, threads, 0, st>>>(a, by_head);
}
void launch_window_delta(const WindowAttn& a, cudaStream_t st) {
  if (a.d == 32) delta_t<32>(a, false, st);
  else if (a.d == 64) delta_t<64>(a, true, st);
  else delta_t<128>(a, true, st);
}
bool launch_window_dq(const WindowAttn& a, bool bf16, cudaStream_t st) {
  if (bf16 && a.d != 32) return launch_window_dq_tc(a, st);
  if (bf16) launch_window_delta(a, st);
  GDN_BY_TYPE(dq_t)
  return true;
}
bool launch_window_dkv(const WindowAttn& a, bool bf16, cudaStream_t st) {
  if (bf16 && a.d != 32) return launch_window_dkv_tc(a, st);
  GDN_BY_TYPE(dkv_t)
  return true;
}

}  // namespace gdn
