// attn_window.cu -- sliding-window attention and its gradient on fp32 SIMT: fp32 inputs (whose
// products stay in 32 bits) and bf16 ones with d = 32.  bf16 with d = 64 or 128 runs on the
// tensor cores (attn_window_tc.cu).
//
// Tiles of 64 queries x 64 keys in shared memory (rows padded by 4 floats, so that 16-byte reads
// of 8 neighbouring rows meet 8 different bank groups), 256 threads; a thread (ty, tx) of 16 x 16
// owns scores (4 ty + r, 16 c + tx) and, of a 64 x D accumulator, rows 4 ty + r and columns
// 4 tx + 64 c .. + 3.  One pass over the keys with a running maximum and sum per row.  The
// gradient is two kernels, each deterministic: per query block dq (and do . o, which the other
// needs), per key block dk and dv over the group's heads in ascending order.
#include "attn_window.cuh"

namespace gdn {

namespace {

using namespace win;

constexpr int BM = 64, BN = 64, kThreads = 256, PS = BN + 4;

template <int D>
__host__ __device__ constexpr int pitch() {
  return D + 4;
}

// rows [row0, row0 + 64) of [rows, H, D] at head h into a tile; rows at or past `end` are zeros
template <int D, typename T>
__device__ __forceinline__ void load_tile(float* tile, const void* src, int64_t base, int row0, int end, int H, int h) {
  constexpr int V = D / 4;
  for (int e = threadIdx.x; e < 64 * V; e += kThreads) {
    const int r = e / V, c = 4 * (e % V);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + r < end) x = load4(static_cast<const T*>(src) + ((base + row0 + r) * H + h) * D + c);
    *reinterpret_cast<float4*>(tile + r * pitch<D>() + c) = x;
  }
}

// x[r][c] = a_row(4 ty + r) . b_row(16 c + tx)
template <int D>
__device__ __forceinline__ void rows_dot(const float* A, const float* B, int ty, int tx, float (&x)[4][4]) {
  float2 acc[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[r][c] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < D; k += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4*>(A + (4 * ty + r) * pitch<D>() + k);
#pragma unroll
    for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4*>(B + (16 * c + tx) * pitch<D>() + k);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[r][c] = fma2(make_float2(a[r].x, a[r].y), make_float2(b[c].x, b[c].y), acc[r][c]);
        acc[r][c] = fma2(make_float2(a[r].z, a[r].w), make_float2(b[c].z, b[c].w), acc[r][c]);
      }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) x[r][c] = __fadd_rn(acc[r][c].x, acc[r][c].y);
}

template <int D>
struct Acc {  // 4 rows x (D / 64 float4 columns; half of the lanes at D = 32)
  static constexpr int C = D >= 64 ? D / 64 : 1;
  float4 v[4][C];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) v[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ static bool mine(int tx) { return D >= 64 || tx < D / 4; }
  // += P[4 ty + r][n] * B[n][cols], n = 0 .. 63 (transposed: P[n][4 ty + r])
  template <bool TRANS>
  __device__ __forceinline__ void add(const float* P, const float* B, int ty, int tx) {
    if (!mine(tx)) return;
#pragma unroll 4
    for (int n = 0; n < 64; ++n) {
      float p[4];
      if (TRANS) {
        const float4 x = *reinterpret_cast<const float4*>(P + n * PS + 4 * ty);
        p[0] = x.x, p[1] = x.y, p[2] = x.z, p[3] = x.w;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = P[(4 * ty + r) * PS + n];
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float4 b = *reinterpret_cast<const float4*>(B + n * pitch<D>() + 4 * tx + 64 * c);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float2 p2 = make_float2(p[r], p[r]);
          const float2 lo = fma2(p2, make_float2(b.x, b.y), make_float2(v[r][c].x, v[r][c].y));
          const float2 hi = fma2(p2, make_float2(b.z, b.w), make_float2(v[r][c].z, v[r][c].w));
          v[r][c] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(void* dst, int64_t base, int row0, int end, int H, int h, int ty, int tx,
                                        const float (&f)[4]) const {
    if (!mine(tx)) return;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = row0 + 4 * ty + r;
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

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) k_window_fwd(const WindowAttn a) {
  extern __shared__ float sh[];
  float *Qs = sh, *Ks = Qs + 64 * pitch<D>(), *Vs = Ks + 64 * pitch<D>(), *Ps = Vs + 64 * pitch<D>();
  if (blockIdx.x == 0 && blockIdx.y == 0) check_tables(a);
  // a sequence's last blocks see the most keys: they start first
  int row0;
  const Seq q = find_seq(a, (int64_t)gridDim.x - 1 - blockIdx.x, BM, false, row0);
  if (!q.ok) return;
  const int h = blockIdx.y, kvh = h / (a.hq / a.hkv), ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int p0 = row0 + q.Lk - q.Lq, p1 = min(row0 + BM, q.Lq) - 1 + q.Lk - q.Lq;
  const KeyBlocks kb(p0, p1, q.Lk, a.window, a.sinks, BN);
  load_tile<D, T>(Qs, a.q, q.q0, row0, q.Lq, a.hq, h);
  const float sc = __fmul_rn(a.scale, kLog2e);
  float m[4], l[4];
  Acc<D> o;
  o.zero();
#pragma unroll
  for (int r = 0; r < 4; ++r) m[r] = -INFINITY, l[r] = 0.f;
  for (int b = 0; b < kb.count(); ++b) {
    const int j0 = kb.block(b) * BN;
    __syncthreads();
    load_tile<D, T>(Ks, a.k, q.k0, j0, q.Lk, a.hkv, kvh);
    load_tile<D, T>(Vs, a.v, q.k0, j0, q.Lk, a.hkv, kvh);
    __syncthreads();
    float x[4][4];
    rows_dot<D>(Qs, Ks, ty, tx, x);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int p = p0 + 4 * ty + r;
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
        Ps[(4 * ty + r) * PS + 16 * c + tx] = p_;
      }
      l[r] = __fmaf_rn(l[r], alpha, s);
#pragma unroll
      for (int c = 0; c < Acc<D>::C; ++c) {
        float4& v = o.v[r][c];
        v = make_float4(__fmul_rn(v.x, alpha), __fmul_rn(v.y, alpha), __fmul_rn(v.z, alpha), __fmul_rn(v.w, alpha));
      }
    }
    __syncwarp();  // a row of Ps is written and read by the same 16 lanes
    o.template add<false>(Ps, Vs, ty, tx);
  }
  float inv[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float s = row_add(l[r]);
    inv[r] = s > 0.f ? __frcp_rn(s) : s == 0.f ? 0.f : s;  // a row that sees nothing: zeros; NaN stays
    const int row = row0 + 4 * ty + r;
    if (tx == 0 && row < q.Lq)
      a.lse[(int64_t)(q.q0 + row) * a.hq + h] = s == 0.f ? -INFINITY : __fmul_rn(__fadd_rn(m[r], log2f(s)), kLn2);
  }
  o.template store<T>(a.out, q.q0, row0, q.Lq, a.hq, h, ty, tx, inv);
}

// p and ds / scale of one tile: p = exp(scale q.k - lse), ds = p (do.v - delta), zero where
// nothing is visible.  x holds q.k on entry and p on return, y do.v and then ds.
__device__ __forceinline__ void grad_scores(const WindowAttn& a, float sc, const int (&pos)[4], const int (&key)[4],
                                            const float (&lse2)[4], const float (&delta)[4], bool rows_are_queries,
                                            float (&x)[4][4], float (&y)[4][4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int qi = rows_are_queries ? r : c, ki = rows_are_queries ? c : r;
      const bool see = visible(pos[qi], key[ki], a.window, a.sinks) && lse2[qi] != -INFINITY;
      const float p = see ? exp2_approx(__fsub_rn(__fmul_rn(x[r][c], sc), lse2[qi])) : 0.f;
      y[r][c] = see ? __fmul_rn(p, __fsub_rn(y[r][c], delta[qi])) : 0.f;
      x[r][c] = p;
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) k_window_dq(const WindowAttn a) {
  extern __shared__ float sh[];
  float *Qs = sh, *Os = Qs + 64 * pitch<D>(), *Ks = Os + 64 * pitch<D>(), *Vs = Ks + 64 * pitch<D>(),
        *Ps = Vs + 64 * pitch<D>();
  if (blockIdx.x == 0 && blockIdx.y == 0) check_tables(a);
  int row0;
  const Seq q = find_seq(a, (int64_t)gridDim.x - 1 - blockIdx.x, BM, false, row0);
  if (!q.ok) return;
  const int h = blockIdx.y, kvh = h / (a.hq / a.hkv), ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int p0 = row0 + q.Lk - q.Lq, p1 = min(row0 + BM, q.Lq) - 1 + q.Lk - q.Lq;
  const KeyBlocks kb(p0, p1, q.Lk, a.window, a.sinks, BN);
  load_tile<D, T>(Qs, a.q, q.q0, row0, q.Lq, a.hq, h);
  load_tile<D, T>(Os, a.dout, q.q0, row0, q.Lq, a.hq, h);
  load_tile<D, T>(Ks, a.out, q.q0, row0, q.Lq, a.hq, h);
  __syncthreads();
  const float sc = __fmul_rn(a.scale, kLog2e);
  int pos[4];
  float lse2[4], delta[4];
  Acc<D> dq;
  dq.zero();
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 4 * ty + r;
    float s = 0.f;
    if (Acc<D>::mine(tx))
#pragma unroll
      for (int c = 0; c < Acc<D>::C; ++c) {
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
      if (tx == 0) a.delta[at] = delta[r];
    }
  }
  for (int b = 0; b < kb.count(); ++b) {
    const int j0 = kb.block(b) * BN;
    __syncthreads();
    load_tile<D, T>(Ks, a.k, q.k0, j0, q.Lk, a.hkv, kvh);
    load_tile<D, T>(Vs, a.v, q.k0, j0, q.Lk, a.hkv, kvh);
    __syncthreads();
    float x[4][4], y[4][4];
    rows_dot<D>(Qs, Ks, ty, tx, x);
    rows_dot<D>(Os, Vs, ty, tx, y);
    const int key[4] = {j0 + tx, j0 + 16 + tx, j0 + 32 + tx, j0 + 48 + tx};
    grad_scores(a, sc, pos, key, lse2, delta, true, x, y);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) Ps[(4 * ty + r) * PS + 16 * c + tx] = y[r][c];
    __syncwarp();
    dq.template add<false>(Ps, Ks, ty, tx);
  }
  const float f[4] = {a.scale, a.scale, a.scale, a.scale};
  dq.template store<T>(a.dq, q.q0, row0, q.Lq, a.hq, h, ty, tx, f);
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) k_window_dkv(const WindowAttn a) {
  extern __shared__ float sh[];
  float *Ks = sh, *Vs = Ks + 64 * pitch<D>(), *Qs = Vs + 64 * pitch<D>(), *Os = Qs + 64 * pitch<D>(),
        *Ps = Os + 64 * pitch<D>(), *Ds = Ps + 64 * PS;
  int j0;
  const Seq q = find_seq(a, blockIdx.x, BN, true, j0);
  if (!q.ok) return;
  const int kvh = blockIdx.y, group = a.hq / a.hkv, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  load_tile<D, T>(Ks, a.k, q.k0, j0, q.Lk, a.hkv, kvh);
  load_tile<D, T>(Vs, a.v, q.k0, j0, q.Lk, a.hkv, kvh);
  const QueryRange qr(q, j0, min(j0 + BN, q.Lk), a.window, a.sinks);
  const float sc = __fmul_rn(a.scale, kLog2e);
  const int off = q.Lk - q.Lq, b0 = qr.lo / BM, b1 = qr.hi > qr.lo ? (qr.hi + BM - 1) / BM : b0;
  int key[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) key[r] = j0 + 4 * ty + r;
  Acc<D> dk, dv;
  dk.zero();
  dv.zero();
  for (int g = 0; g < group; ++g) {
    const int h = kvh * group + g;
    for (int b = b0; b < b1; ++b) {
      const int row0 = b * BM;
      __syncthreads();
      load_tile<D, T>(Qs, a.q, q.q0, row0, q.Lq, a.hq, h);
      load_tile<D, T>(Os, a.dout, q.q0, row0, q.Lq, a.hq, h);
      __syncthreads();
      int pos[4];
      float lse2[4], delta[4], x[4][4], y[4][4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int row = row0 + 16 * c + tx;
        pos[c] = row + off;
        lse2[c] = -INFINITY;
        delta[c] = 0.f;
        if (row < q.Lq) {
          const int64_t at = (int64_t)(q.q0 + row) * a.hq + h;
          lse2[c] = __fmul_rn(a.lse[at], kLog2e);
          delta[c] = a.delta[at];
        }
      }
      rows_dot<D>(Ks, Qs, ty, tx, x);  // transposed: rows are keys
      rows_dot<D>(Vs, Os, ty, tx, y);
      grad_scores(a, sc, pos, key, lse2, delta, false, x, y);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          Ps[(4 * ty + r) * PS + 16 * c + tx] = x[r][c];
          Ds[(4 * ty + r) * PS + 16 * c + tx] = y[r][c];
        }
      __syncwarp();
      dv.template add<false>(Ps, Os, ty, tx);
      dk.template add<false>(Ds, Qs, ty, tx);
    }
  }
  const float one[4] = {1.f, 1.f, 1.f, 1.f}, f[4] = {a.scale, a.scale, a.scale, a.scale};
  dv.template store<T>(a.dv, q.k0, j0, q.Lk, a.hkv, kvh, ty, tx, one);
  dk.template store<T>(a.dk, q.k0, j0, q.Lk, a.hkv, kvh, ty, tx, f);
}

template <void (*FN)(WindowAttn)>
void launch(dim3 grid, size_t floats, const WindowAttn& a, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  ensure_smem(FN, (int)(floats * sizeof(float)), ready);
  FN<<<grid, kThreads, floats * sizeof(float), st>>>(a);
}

template <int D, typename T>
void fwd_t(const WindowAttn& a, cudaStream_t st) {
  launch<k_window_fwd<D, T>>(dim3((unsigned)item_count(a.Tq, BM, a.N), a.hq), 3 * 64 * pitch<D>() + 64 * PS, a, st);
}
template <int D, typename T>
void dq_t(const WindowAttn& a, cudaStream_t st) {
  launch<k_window_dq<D, T>>(dim3((unsigned)item_count(a.Tq, BM, a.N), a.hq), 4 * 64 * pitch<D>() + 64 * PS, a, st);
}
template <int D, typename T>
void dkv_t(const WindowAttn& a, cudaStream_t st) {
  launch<k_window_dkv<D, T>>(dim3((unsigned)item_count(a.Tk, BN, a.N), a.hkv), 4 * 64 * pitch<D>() + 2 * 64 * PS, a,
         st);
}

}  // namespace

#define GDN_BY_TYPE(f)                            \
  if (bf16) {                                     \
    if (a.d == 32) f<32, __nv_bfloat16>(a, st);   \
    else if (a.d == 64) f<64, __nv_bfloat16>(a, st); \
    else f<128, __nv_bfloat16>(a, st);            \
  } else {                                        \
    if (a.d == 32) f<32, float>(a, st);           \
    else if (a.d == 64) f<64, float>(a, st);      \
    else f<128, float>(a, st);                    \
  }

bool launch_window_attn(const WindowAttn& a, bool bf16, cudaStream_t st) {
  if (window_on_tensor_cores(a, bf16)) return launch_window_fwd_tc(a, st);
  GDN_BY_TYPE(fwd_t)
  return true;
}
bool launch_window_dq(const WindowAttn& a, bool bf16, cudaStream_t st) {
  if (window_on_tensor_cores(a, bf16)) return launch_window_dq_tc(a, st);
  GDN_BY_TYPE(dq_t)
  return true;
}
bool launch_window_dkv(const WindowAttn& a, bool bf16, cudaStream_t st) {
  if (window_on_tensor_cores(a, bf16)) return launch_window_dkv_tc(a, st);
  GDN_BY_TYPE(dkv_t)
  return true;
}

}  // namespace gdn
