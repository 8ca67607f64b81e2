// attn_decode.cu -- attention of one new token per request over the paged cache.
//
// A request's visible keys (the first `sinks` and the last `window`, or all) are numbered
// u = 0 .. n - 1 in key order, so that masks never cut a tile: only its end is short.  They are
// split into runs of split_keys(n), a function of n alone, and each CTA takes one run of one
// key head for up to 16 query heads:
//     s_u = scale q . k_u,  m = max s,  l = sum e^(s - m),  a = sum e^(s - m) v_u
// in one pass with a running maximum (scores in units of log2 e, so that e^x is one exp2).
// With one run the CTA writes the output a / l; otherwise it leaves (m, l, a) in the workspace
// and k_decode_join adds a request's runs in ascending order.
#include "attn.h"

namespace gdn {

namespace {

constexpr int kDecThreads = 128, kDecWarps = kDecThreads / 32;
constexpr int kHeadsPerCta = 16;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a CTA needs to know of its request.
struct Request {
  int len, n;        // cached tokens (0 if the length is not valid), visible keys
  int head, skip;    // key of visible index u: u < head ? u : u + skip
  bool bad;
  __device__ __forceinline__ Request(const PagedDecode& a, int i) {
    len = a.seq_lens[i];
    bad = len < 0 || len > a.max_len;
    if (bad) len = 0;
    n = visible_keys(len, a.window, a.sinks);
    skip = len - n;
    head = skip > 0 ? a.sinks : 0;
  }
  __device__ __forceinline__ int key(int u) const { return u < head ? u : u + skip; }
};

// Row (page, key head) of key j, or -1 for a page outside the cache.
__device__ __forceinline__ int64_t key_row(const PagedDecode& a, const int32_t* bt, int kvh, int j) {
  const int b = j >> a.page_shift;
  const int page = b < a.max_blocks ? bt[b] : -1;
  if (page < 0 || page >= a.num_pages) return -1;
  return ((((int64_t)page * a.hkv + kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1)));
}

// Error word: every visible key of request i lies on a page of the cache.  All threads call it.
__device__ int check_request(const PagedDecode& a, int i) {
  const Request rq(a, i);
  if (rq.bad) return GDN_DEVERR_POS;
  const int32_t* bt = a.block_table + (int64_t)i * a.max_blocks;
  const int first = rq.n ? rq.key(rq.head) >> a.page_shift : 0, last = rq.n ? (rq.len - 1) >> a.page_shift : -1;
  const int head_pages = rq.head ? ((rq.head - 1) >> a.page_shift) + 1 : 0;
  bool bad = false;
  for (int b = threadIdx.x; b < head_pages + (last - first + 1); b += blockDim.x) {
    const int p = b < head_pages ? b : first + b - head_pages;
    const int page = p < a.max_blocks ? bt[p] : -1;
    bad |= page < 0 || page >= a.num_pages;
  }
  return __syncthreads_or(bad) ? GDN_DEVERR_PAGES : 0;
}

// The warps' (m, l, a) of one CTA joined in warp order and written: as the output when the
// request has one run, else as the run's record.  sm, sl: [heads][warps]; sa: [warps][heads][D].
template <int D, typename T>
__device__ __forceinline__ void finish_run(const PagedDecode& a, int i, int h0, int heads, int run, bool single,
                                           const float* sm, const float* sl, const float* sa, int sa_heads) {
  for (int e = threadIdx.x; e < heads * D; e += kDecThreads) {
    const int h = e / D, c = e % D;
    float m = sm[h * kDecWarps];
#pragma unroll
    for (int w = 1; w < kDecWarps; ++w) m = fmaxf(m, sm[h * kDecWarps + w]);
    float l = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float mw = sm[h * kDecWarps + w];
      const float f = mw == -INFINITY ? 0.f : exp2_approx(__fsub_rn(mw, m));
      l = __fmaf_rn(f, sl[h * kDecWarps + w], l);
      acc = __fmaf_rn(f, sa[(w * sa_heads + h) * D + c], acc);
    }
    const int64_t row = (int64_t)i * a.hq + h0 + h;
    if (single) {
      store_out(static_cast<T*>(a.out) + row * D + c, __fdiv_rn(acc, l));
      if (a.lse && c == 0) a.lse[row] = __fmul_rn(__fadd_rn(m, log2f(l)), kLn2);
    } else {
      const int64_t rec = row * a.max_splits + run;
      a.partial[rec * D + c] = acc;
      if (c == 0) {
        float* ml = a.partial + (int64_t)a.N * a.hq * a.max_splits * D + rec * 2;
        ml[0] = m;
        ml[1] = l;
      }
    }
  }
}

// Rows of a request without keys (zeros) or with a length that is not valid (NaN).
template <int D, typename T>
__device__ __forceinline__ void write_empty(const PagedDecode& a, int i, int h0, int heads, bool bad) {
  const float x = bad ? __builtin_nanf("") : 0.f;
  for (int e = threadIdx.x; e < heads * D; e += kDecThreads) {
    const int64_t row = (int64_t)i * a.hq + h0 + e / D;
    store_out(static_cast<T*>(a.out) + row * D + e % D, x);
    if (a.lse && e % D == 0) a.lse[row] = bad ? x : -INFINITY;
  }
}

// The error word of a call: set by the join kernel's CTAs, after this kernel's first CTA has
// cleared it; without a join kernel that CTA looks at every request itself.
__device__ __forceinline__ void error_word(const PagedDecode& a) {
  if (blockIdx.x || blockIdx.y || blockIdx.z) return;
  int err = 0;
  if (a.max_splits == 1)
    for (int i = 0; i < a.N && !err; ++i) err = check_request(a, i);
  if (threadIdx.x == 0) a.hdr->err = err;
}

// ---------------------------------------------------------------------------- SIMT ----
// fp32 caches, and bf16 ones with d = 32.  A lane holds 4 columns, LPR = D / 4 lanes a key, and a warp takes 8 keys
// at a time.  Per lane group the partial dots of 8 / KPW keys with 4 heads are LPR values, which
// one halving exchange turns into one whole score per lane (LPR - 1 shuffles instead of
// log2(LPR) per score), where its exponential is formed.
template <int D, typename T, int NC>
__global__ void __launch_bounds__(kDecThreads) k_decode_simt(const PagedDecode a) {
  constexpr int LPR = D / 4, KPW = 32 / LPR, KT = 8 / KPW;
  static_assert(KT * 4 == LPR, "one score per lane");
  __shared__ float qs[NC * 4][D];
  __shared__ float sm[NC * 4][kDecWarps], sl[NC * 4][kDecWarps];
  __shared__ float sa[kDecWarps][NC * 4][D];
  error_word(a);
  const int i = blockIdx.z, run = blockIdx.x, group = a.hq / a.hkv;
  const int parts = (group + kHeadsPerCta - 1) / kHeadsPerCta, kvh = blockIdx.y / parts;
  const int g0 = (blockIdx.y % parts) * kHeadsPerCta, heads = min(kHeadsPerCta, group - g0);
  const int h0 = kvh * group + g0;
  const Request rq(a, i);
  const int runs = split_count(rq.n);
  if (run >= runs) {
    if (run == 0) write_empty<D, T>(a, i, h0, heads, rq.bad);
    return;
  }
  const float qscale = __fmul_rn(a.scale, kLog2e);
  for (int e = threadIdx.x; e < NC * 4 * D; e += kDecThreads) {
    const int h = e / D;
    qs[h][e % D] =
        h < heads ? __fmul_rn(to_f32(static_cast<const T*>(a.q)[((int64_t)i * a.hq + h0 + h) * D + e % D]), qscale) : 0.f;
  }
  __syncthreads();
  const int per = split_keys(rq.n), u_end = min(rq.n, (run + 1) * per);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane / LPR, b = lane % LPR;
  const int32_t* bt = a.block_table + (int64_t)i * a.max_blocks;
  const T *kp = static_cast<const T*>(a.k_pages) + 4 * b, *vp = static_cast<const T*>(a.v_pages) + 4 * b;
  float m[NC], l[NC];
  float4 acc[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    m[c] = -INFINITY;
    l[c] = 0.f;
#pragma unroll
    for (int h = 0; h < 4; ++h) acc[c][h] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  bool bad = false;
  for (int u0 = run * per + warp * 8; u0 < u_end; u0 += kDecWarps * 8) {
    float4 kk[KT], vv[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int u = u0 + grp * KT + t;
      kk[t] = vv[t] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (u < u_end) {
        const int64_t row = key_row(a, bt, kvh, rq.key(u));
        if (row >= 0) {
          kk[t] = load4(kp + row * D);
          vv[t] = load4(vp + row * D);
        } else {
          bad = true;
        }
      }
    }
    const bool live = u0 + grp * KT + (b >> 2) < u_end;  // the key of this lane's score
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float val[LPR];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float4 q4 = *reinterpret_cast<const float4*>(&qs[c * 4 + h][4 * b]);
#pragma unroll
        for (int t = 0; t < KT; ++t)
          val[t * 4 + h] = __fmaf_rn(
              q4.w, kk[t].w, __fmaf_rn(q4.z, kk[t].z, __fmaf_rn(q4.y, kk[t].y, __fmul_rn(q4.x, kk[t].x))));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int j = 0; j < o; ++j) {
          const bool up = (lane & o) != 0;
          const float send = up ? val[j] : val[j + o], keep = up ? val[j + o] : val[j];
          val[j] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
      }
      const float s = live ? val[0] : -INFINITY;  // head b & 3
      float mx = s;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(mx, m[c]);
      const float base = mx == -INFINITY ? 0.f : mx;
      const float alpha = exp2_approx(__fsub_rn(m[c], base)), p = exp2_approx(__fsub_rn(s, base));
      m[c] = mx;
      l[c] = __fmaf_rn(l[c], alpha, p);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float al = __shfl_sync(0xffffffffu, alpha, h);
        float4 x = acc[c][h];
        x = make_float4(__fmul_rn(x.x, al), __fmul_rn(x.y, al), __fmul_rn(x.z, al), __fmul_rn(x.w, al));
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          const float ph = __shfl_sync(0xffffffffu, p, grp * LPR + t * 4 + h);
          x = make_float4(__fmaf_rn(ph, vv[t].x, x.x), __fmaf_rn(ph, vv[t].y, x.y), __fmaf_rn(ph, vv[t].z, x.z),
                          __fmaf_rn(ph, vv[t].w, x.w));
        }
        acc[c][h] = x;
      }
    }
  }
  bad = __any_sync(0xffffffffu, bad);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float lc = l[c];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) lc = __fadd_rn(lc, __shfl_xor_sync(0xffffffffu, lc, o));
    if (lane < 4) {
      sm[c * 4 + lane][warp] = m[c];
      sl[c * 4 + lane][warp] = bad ? __builtin_nanf("") : lc;
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      float4 x = acc[c][h];
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        x.x = __fadd_rn(x.x, __shfl_xor_sync(0xffffffffu, x.x, o));
        x.y = __fadd_rn(x.y, __shfl_xor_sync(0xffffffffu, x.y, o));
        x.z = __fadd_rn(x.z, __shfl_xor_sync(0xffffffffu, x.z, o));
        x.w = __fadd_rn(x.w, __shfl_xor_sync(0xffffffffu, x.w, o));
      }
      if (grp == 0) *reinterpret_cast<float4*>(&sa[warp][c * 4 + h][4 * b]) = x;
    }
  }
  __syncthreads();
  finish_run<D, T>(a, i, h0, heads, run, runs == 1, &sm[0][0], &sl[0][0], &sa[0][0][0], NC * 4);
}

// ---------------------------------------------------------------------------- join ----
// One warp per (request, head): adds the runs' records in ascending order.  The first head's
// CTA of a request also checks it for the error word.
template <int D, typename T>
__global__ void __launch_bounds__(128) k_decode_join(const PagedDecode a) {
  constexpr int V = D / 32;
  const int i = blockIdx.y, h = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const Request rq(a, i);
  const int runs = split_count(rq.n);
  if (h < a.hq && runs > 1) {
    const int64_t row = (int64_t)i * a.hq + h;
    const float* rec = a.partial + row * a.max_splits * D;
    const float* ml = a.partial + ((int64_t)a.N * a.hq * D + row * 2) * a.max_splits;
    float m = -INFINITY;
    for (int r = lane; r < runs; r += 32) m = fmaxf(m, ml[2 * r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 4
    for (int r = 0; r < runs; ++r) {
      const float f = exp2_approx(__fsub_rn(ml[2 * r], m));
      l = __fmaf_rn(f, ml[2 * r + 1], l);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = __fmaf_rn(f, rec[(int64_t)r * D + v * 32 + lane], acc[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      store_out(static_cast<T*>(a.out) + row * D + v * 32 + lane, __fdiv_rn(acc[v], l));
    if (a.lse && lane == 0) a.lse[row] = __fmul_rn(__fadd_rn(m, log2f(l)), kLn2);
  }
  if (blockIdx.x == 0) {
    const int err = check_request(a, i);
    if (err && threadIdx.x == 0) set_error(a.hdr, err);
  }
}

template <int D, typename T>
void decode_t(const PagedDecode& a, cudaStream_t st) {
  const int group = a.hq / a.hkv, parts = (group + kHeadsPerCta - 1) / kHeadsPerCta;
  const dim3 grid(a.max_splits, a.hkv * parts, a.N);
  const int nc = group <= 4 ? 1 : group <= 8 ? 2 : 4;
  if (nc == 1)
    k_decode_simt<D, T, 1><<<grid, kDecThreads, 0, st>>>(a);
  else if (nc == 2)
    k_decode_simt<D, T, 2><<<grid, kDecThreads, 0, st>>>(a);
  else
    k_decode_simt<D, T, 4><<<grid, kDecThreads, 0, st>>>(a);
  if (a.max_splits > 1) k_decode_join<D, T><<<dim3((a.hq + 3) / 4, a.N), 128, 0, st>>>(a);
}

}  // namespace

// The largest number of runs of any request that sees at most `max_visible` keys.
int paged_decode_max_splits(int max_visible) {
  int best = 1;
  for (const int edge : {2048, 8192}) {
    const int n = max_visible < edge ? max_visible : edge;
    if (n > 0 && split_count(n) > best) best = split_count(n);
  }
  if (max_visible > 0 && split_count(max_visible) > best) best = split_count(max_visible);
  return best;
}

int launch_paged_decode(const PagedDecode& a, bool bf16, cudaStream_t st) {
  if (bf16) {
    if (a.d == 32) decode_t<32, __nv_bfloat16>(a, st);
    else if (a.d == 64) decode_t<64, __nv_bfloat16>(a, st);
    else decode_t<128, __nv_bfloat16>(a, st);
  } else {
    if (a.d == 32) decode_t<32, float>(a, st);
    else if (a.d == 64) decode_t<64, float>(a, st);
    else decode_t<128, float>(a, st);
  }
  return a.max_splits > 1 ? 2 : 1;
}

}  // namespace gdn
