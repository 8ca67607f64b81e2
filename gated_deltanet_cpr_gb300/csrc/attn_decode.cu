// attn_decode.cu -- attention of one new token per request over the paged cache.
//
// A request's visible keys (the first `sinks` and the last `window`, or all) are numbered
// u = 0 .. n - 1 in key order, so that masks never cut a tile: only its end is short.  They are
// split into runs of split_of(n, key heads); one warp takes a run of one key head for up to 16
// of its query heads in one pass with a running maximum (scores in units of log2 e, so that
// e^x is one exp2):
//     s_u = scale q . k_u,  m = max s,  l = sum e^(s - m),  a = sum e^(s - m) v_u
// and writes the output a / l, or, where a request has several runs, leaves (m, l, a) in the
// workspace for k_decode_join, which adds them in ascending order.
//
// The kernel is bound by the cache's bytes, so what matters is that loads never pause.  A warp
// works alone: it walks over runs (the grid fills the SMs once), and copies keys and values
// asynchronously into its own ring, a tile or two ahead and across the end of a run, with the next
// tile's pages looked up meanwhile.  256 requests of about 2112 tokens, 32 / 8 heads, d = 128: 328 us,
// 6.8 TB/s of the cache, which is a copy's rate.  A kernel of one CTA of four warps per run,
// which waits for its first keys and joins its warps at the end, reached 72% (runs of 256 keys) to
// 94% (1024 keys) of it.  Few requests are bound by the latency of one run, the launch and the join:
// 4 of about 700 tokens take 9.0 us.
#include "attn.h"
#include "tc.cuh"

namespace gdn {

namespace {

constexpr int kHeadsPerRun = 16;
constexpr int kSms = 152;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a warp needs to know of a request.
struct Request {
  int len, n;        // cached tokens (0 if the length is not valid), visible keys
  int head, skip;    // key of visible index u: u < head ? u : u + skip
  bool bad;
  __device__ __forceinline__ Request(const PagedDecode& a, int length) {
    len = length;
    bad = len < 0 || len > a.max_len;
    if (bad) len = 0;
    n = visible_keys(len, a.window, a.sinks);
    skip = len - n;
    head = skip > 0 ? a.sinks : 0;
  }
  __device__ __forceinline__ int key(int u) const { return u < head ? u : u + skip; }
};

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void* gmem, bool load) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(load ? 16 : 0) : "memory");
}

// One run: request i, key head and part of its query heads, which run, and its keys [u, end); bad:
// a key's page is outside the cache.  Keys are numbered without a sign: a request may end a tile
// short of 2^31, and the walk steps past its end.
struct Run {
  int i, y, run, runs;
  uint32_t u, end;
  int head, skip, bad;
  __device__ __forceinline__ int key(uint32_t x) const { return (int)x < head ? (int)x : (int)x + skip; }
};

// Where a run's (m, l, a) or output goes: rows of its heads.
struct Sink {
  float* acc;   // record of head 0's run, or NULL: the run is the whole request
  float2* ml;
  int64_t acc_step, ml_step;  // from one head to the next
  void* out;                  // row of head 0
  float* lse;
  int heads;
  __device__ __forceinline__ Sink(const PagedDecode& a, const Run& r, int h0, int heads_, int elem) : heads(heads_) {
    const int64_t row = (int64_t)r.i * a.hq + h0;
    out = static_cast<char*>(a.out) + row * a.d * elem;
    lse = a.lse ? a.lse + row : nullptr;
    acc = nullptr;
    ml = nullptr;
    acc_step = ml_step = 0;
    if (r.runs > 1) {
      const int64_t rec = row * a.max_splits + r.run;
      acc = a.partial + rec * a.d;
      ml = reinterpret_cast<float2*>(a.partial + (int64_t)a.N * a.hq * a.max_splits * a.d) + rec;
      acc_step = (int64_t)a.max_splits * a.d;
      ml_step = a.max_splits;
    }
  }
  __device__ __forceinline__ void stats(int h, float m, float l) const {
    if (ml) ml[h * ml_step] = make_float2(m, l);
    else if (lse) lse[h] = __fmul_rn(__fadd_rn(m, log2f(l)), kLn2);
  }
};

// ---------------------------------------------------------------------------- SIMT ----
// fp32 caches, and bf16 ones with d = 32.  A lane holds 4 columns, LPR = D / 4 lanes a key, and a
// tile is 32 / H keys.  Per lane group the partial dots of its KT keys with H heads (2 or 4) are LPR
// values, which one halving exchange turns into one whole score per lane (LPR - 1 shuffles
// instead of log2(LPR) per score), where its exponential is formed.  NC chunks of H heads.
template <int D, typename T, int H, int NC>
struct SimtEngine {
  using Elem = T;
  static constexpr int DIM = D, KEYS = 32 / H, ROWB = D * sizeof(T), EXTRA = NC * H * D * 4;
  static constexpr int RING = KEYS * ROWB > 4096 ? 2 : 3;
  static constexpr int LPR = D / 4, KPW = 32 / LPR, KT = KEYS / KPW;
  static constexpr bool MANY_REGS = NC == 4;  // more than 168 a thread
  static_assert(KT * H == LPR, "one score per lane");
  const float* qs;  // [NC * H][D], scaled
  float m[NC], l[NC];
  float4 acc[NC][H];

  __device__ __forceinline__ static uint32_t place(int r, int c) { return r * ROWB + c * 16; }

  __device__ __forceinline__ void start(const PagedDecode& a, int64_t row, int heads, unsigned char* extra, int lane) {
    float* q = reinterpret_cast<float*>(extra);
    const float scale = __fmul_rn(a.scale, kLog2e);
    const T* src = static_cast<const T*>(a.q) + row * D;
    __syncwarp();
#pragma unroll 4
    for (int e = lane; e < NC * H * D; e += 32) q[e] = e < heads * D ? __fmul_rn(to_f32(src[e]), scale) : 0.f;
    __syncwarp();
    qs = q;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      m[c] = -INFINITY;
      l[c] = 0.f;
#pragma unroll
      for (int h = 0; h < H; ++h) acc[c][h] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }

  __device__ __forceinline__ void tile(const PagedDecode&, const unsigned char* st, int keys, int lane) {
    const int grp = lane / LPR, b = lane % LPR;
    const T* p0 = reinterpret_cast<const T*>(st) + grp * KT * D + 4 * b;
    const bool live = grp * KT + b / H < keys;  // the key of this lane's score
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float val[LPR];
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const float4 k4 = load4(p0 + t * D);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float4 q4 = *reinterpret_cast<const float4*>(qs + (c * H + h) * D + 4 * b);
          val[t * H + h] =
              __fmaf_rn(q4.w, k4.w, __fmaf_rn(q4.z, k4.z, __fmaf_rn(q4.y, k4.y, __fmul_rn(q4.x, k4.x))));
        }
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
      const float s = live ? val[0] : -INFINITY;  // head b % H
      float mx = s;
#pragma unroll
      for (int o = H; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(mx, m[c]);
      const float base = mx == -INFINITY ? 0.f : mx;
      const float alpha = exp2_approx(__fsub_rn(m[c], base)), p = exp2_approx(__fsub_rn(s, base));
      m[c] = mx;
      l[c] = __fmaf_rn(l[c], alpha, p);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float al = __shfl_sync(0xffffffffu, alpha, h);
        float4& x = acc[c][h];
        x = make_float4(__fmul_rn(x.x, al), __fmul_rn(x.y, al), __fmul_rn(x.z, al), __fmul_rn(x.w, al));
      }
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const float4 v4 = load4(p0 + (KEYS + t) * D);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float ph = __shfl_sync(0xffffffffu, p, grp * LPR + t * H + h);
          float4& x = acc[c][h];
          x = make_float4(__fmaf_rn(ph, v4.x, x.x), __fmaf_rn(ph, v4.y, x.y), __fmaf_rn(ph, v4.z, x.z),
                          __fmaf_rn(ph, v4.w, x.w));
        }
      }
    }
  }

  __device__ __forceinline__ void finish(const Sink& k, bool bad, int lane) {
    const int grp = lane / LPR, b = lane % LPR;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float lc = l[c];
#pragma unroll
      for (int o = H; o < 32; o <<= 1) lc = __fadd_rn(lc, __shfl_xor_sync(0xffffffffu, lc, o));
      if (bad) lc = __builtin_nanf("");
      if (lane < H && c * H + lane < k.heads) k.stats(c * H + lane, m[c], lc);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float4 x = acc[c][h];
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
          x.x = __fadd_rn(x.x, __shfl_xor_sync(0xffffffffu, x.x, o));
          x.y = __fadd_rn(x.y, __shfl_xor_sync(0xffffffffu, x.y, o));
          x.z = __fadd_rn(x.z, __shfl_xor_sync(0xffffffffu, x.z, o));
          x.w = __fadd_rn(x.w, __shfl_xor_sync(0xffffffffu, x.w, o));
        }
        const float lh = __shfl_sync(0xffffffffu, lc, h);
        if (grp || c * H + h >= k.heads) continue;
        if (k.acc)
          store4(k.acc + (c * H + h) * k.acc_step + 4 * b, x);
        else
          store4(static_cast<T*>(k.out) + (c * H + h) * D + 4 * b,
                 make_float4(__fdiv_rn(x.x, lh), __fdiv_rn(x.y, lh), __fdiv_rn(x.z, lh), __fdiv_rn(x.w, lh)));
      }
    }
  }
};

// ----------------------------------------------------------------------- tensor cores ----
// bf16 caches with d = 64 or 128.  fp32 lanes would spend 4 FMA per byte on 16 heads, more than
// they have, so the products run on warp-level MMAs (m16n8k16), far below their rate.  A tile is
// 32 keys: scores [16 heads x 32 keys], the running maximum and sum, then P V with P as the sum of
// two bf16 (so that its rounding does not show in the output).  Rows are swizzled so that the 8
// rows of a matrix load lie in 8 bank groups: piece c of row r at c ^ (r & 7).
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}
// the part of (lo, hi) that pack2 lost
__device__ __forceinline__ uint32_t pack2_rest(float lo, float hi, uint32_t packed) {
  return pack2(__fsub_rn(lo, __uint_as_float(packed << 16)), __fsub_rn(hi, __uint_as_float(packed & 0xffff0000u)));
}

template <int D>
struct MmaEngine {
  using Elem = __nv_bfloat16;
  static constexpr int DIM = D, KEYS = 32, ROWB = D * 2, RING = 2, EXTRA = 0, KS = D / 16, NT = KEYS / 8;
  static constexpr bool MANY_REGS = false;
  uint32_t q[KS][4];
  float m[2], l[2], o[D / 8][4];

  __device__ __forceinline__ static uint32_t place(int r, int c) { return r * ROWB + ((c ^ (r & 7)) << 4); }

  __device__ __forceinline__ void start(const PagedDecode& a, int64_t row, int heads, unsigned char*, int lane) {
    // query fragments: rows = heads lane / 4 and + 8, columns 16 k + 2 (lane % 4) and + 8
    const Elem* qp = static_cast<const Elem*>(a.q) + row * D + 2 * (lane & 3);
    const int r0 = lane >> 2, r1 = r0 + 8;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        q[k][2 * e] = r0 < heads ? *reinterpret_cast<const uint32_t*>(qp + r0 * D + 16 * k + 8 * e) : 0u;
        q[k][2 * e + 1] = r1 < heads ? *reinterpret_cast<const uint32_t*>(qp + r1 * D + 16 * k + 8 * e) : 0u;
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  }

  __device__ __forceinline__ void tile(const PagedDecode& a, const unsigned char* stage, int keys, int lane) {
    const uint32_t st = tc::smem_u32(stage);
    // matrix-load addresses: row of the tile, and which 16-byte piece of a pair
    const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1, vr = lane & 15, vc = lane >> 4;
    const float sc = __fmul_rn(a.scale, kLog2e);
    float x[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t b[4];
        tc::ldsm_x4(st + place(kr + 8 * n, 2 * k + kc), b);
        tc::mma16816(x[n], q[k], b[0], b[1]);
        tc::mma16816(x[n + 1], q[k], b[2], b[3]);
      }
    if (keys < KEYS) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (2 * (lane & 3) + 8 * n + (e & 1) >= keys) x[n][e] = -INFINITY;
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], x[n][e]);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      mx[r] = fmaxf(m[r], __fmul_rn(mx[r], sc));
    }
    if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float f = m[r] == -INFINITY ? 0.f : exp2_approx(__fsub_rn(m[r], mx[r]));
        m[r] = mx[r];
        l[r] = __fmul_rn(l[r], f);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][2 * r] = __fmul_rn(o[j][2 * r], f);
          o[j][2 * r + 1] = __fmul_rn(o[j][2 * r + 1], f);
        }
      }
    }
    const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[n][e] = exp2_approx(__fmaf_rn(x[n][e], sc, -base[e >> 1]));
        l[e >> 1] = __fadd_rn(l[e >> 1], x[n][e]);
      }
#pragma unroll
    for (int n = 0; n < NT; n += 2) {  // 16 keys
      const uint32_t hi[4] = {pack2(x[n][0], x[n][1]), pack2(x[n][2], x[n][3]), pack2(x[n + 1][0], x[n + 1][1]),
                              pack2(x[n + 1][2], x[n + 1][3])};
      const uint32_t lo[4] = {pack2_rest(x[n][0], x[n][1], hi[0]), pack2_rest(x[n][2], x[n][3], hi[1]),
                              pack2_rest(x[n + 1][0], x[n + 1][1], hi[2]), pack2_rest(x[n + 1][2], x[n + 1][3], hi[3])};
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t b[4];
        tc::ldsm_x4_trans(st + KEYS * ROWB + place(vr + 8 * n, 2 * j + vc), b);
        tc::mma16816(o[2 * j], hi, b[0], b[1]);
        tc::mma16816(o[2 * j + 1], hi, b[2], b[3]);
        tc::mma16816(o[2 * j], lo, b[0], b[1]);
        tc::mma16816(o[2 * j + 1], lo, b[2], b[3]);
      }
    }
  }

  __device__ __forceinline__ void finish(const Sink& k, bool bad, int lane) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] = __fadd_rn(l[r], __shfl_xor_sync(0xffffffffu, l[r], 1));
      l[r] = __fadd_rn(l[r], __shfl_xor_sync(0xffffffffu, l[r], 2));
      if (bad) l[r] = __builtin_nanf("");
      const int h = (lane >> 2) + 8 * r;
      if (h >= k.heads) continue;
      if ((lane & 3) == 0) k.stats(h, m[r], l[r]);
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const int c = 8 * j + 2 * (lane & 3);
        if (k.acc)
          *reinterpret_cast<float2*>(k.acc + h * k.acc_step + c) = make_float2(o[j][2 * r], o[j][2 * r + 1]);
        else
          *reinterpret_cast<uint32_t*>(static_cast<Elem*>(k.out) + h * D + c) =
              pack2(__fdiv_rn(o[j][2 * r], l[r]), __fdiv_rn(o[j][2 * r + 1], l[r]));
      }
    }
  }
};

// ---------------------------------------------------------------------------- walk ----
// One CTA per SM with as many warps as its shared memory has rings for (7, or as many on each
// scheduler: 13 warps instead of 12 at d = 64 cost 200 requests 249 us against 225).  First slots are
// dealt out across the SMs before a second warp of any gets one, so that a few runs spread over
// all of them: with several smaller CTAs an SM, some SMs got three busy ones and some none (7 requests
// of 4 to 22 thousand tokens, d = 64: 28.1 us against 23.9; 4 of about 700: 10.2 against 9.0).
template <typename E>
struct DecodeSmem {
  static constexpr int STAGE = 2 * E::KEYS * E::ROWB, RING = E::RING * STAGE, EXTRA = RING, QUEUE = EXTRA + E::EXTRA;
  static constexpr int WARP = (QUEUE + 4 * (int)sizeof(Run) + 127) / 128 * 128, MOST = 227 * 1024 / WARP;
  static constexpr int WARPS = MOST < 8 ? MOST : MOST < 12 || E::MANY_REGS ? 8 : 12, HALF = 116 * 1024;
  static constexpr int BYTES = WARPS * WARP > HALF ? WARPS * WARP : HALF;  // more than half: one CTA per SM
};

// The fetching side of a warp: which tile comes next, and where its keys lie.
template <typename E>
struct Walk {
  // (run, request, part) slots are numbered with the run slowest and dealt out in chunks of `chunk`
  // <= 32 consecutive ones, one per lane: the first by the warp's number, further ones from a
  // counter, as runs differ in length and many slots of short requests are empty.
  uint32_t total, chunk;
  int32_t* counter;
  uint32_t base;                 // the chunk after the present one, looked up a run ahead of its use:
  int next_i, next_y, next_run;  // this lane's slot of it (next_run < 0: none)
  int next_len;                  // and its request's length
  uint32_t left;                 // slots of the present chunk that hold a run and are still to come
  Run mine;                      // this lane's run of it
  Run r;                         // the run being fetched
  bool live;                     // there is one
  int page;                      // lane < KEYS: page of key r.u + lane, on its way during the tile before

  __device__ __forceinline__ void look_ahead(const PagedDecode& a, int parts, int lane) {
    const uint32_t w = base + (uint32_t)lane, ny = (uint32_t)(a.hkv * parts), rows = (uint32_t)a.N * ny;
    next_run = -1;
    if (w >= total || lane >= (int)chunk) return;
    next_run = (int)(w / rows);
    const uint32_t v = w - (uint32_t)next_run * rows;
    next_i = (int)(v / ny);
    next_y = (int)(v - (uint32_t)next_i * ny);
    next_len = a.seq_lens[next_i];
  }

  // The next run of this warp.  Requests without keys have their rows written here.
  __device__ void seek(const PagedDecode& a, int parts, int lane) {
    live = false;
    while (!left) {
      if (base >= total) return;
      bool have = false;
      if (next_run >= 0) {
        const Request rq(a, next_len);
        const Split s = split_of(rq.n, a.hkv);
        mine.i = next_i;
        mine.y = next_y;
        mine.run = next_run;
        mine.runs = s.runs;
        have = next_run < s.runs;
        mine.u = (uint32_t)next_run * (uint32_t)s.keys;
        mine.end = min((uint32_t)rq.n, mine.u + (uint32_t)s.keys);
        mine.head = rq.head;
        mine.skip = rq.skip;
        if (s.runs == 0 && next_run == 0) write_empty(a, mine, parts, rq.bad);
      }
      left = __ballot_sync(0xffffffffu, have);
      int n = 0;
      if (!counter) base = total;
      else if (lane == 0) n = atomicAdd(counter, 1);
      if (counter) base = (gridDim.x * DecodeSmem<E>::WARPS + (uint32_t)__shfl_sync(0xffffffffu, n, 0)) * chunk;
      look_ahead(a, parts, lane);
    }
    const int src = __ffs(left) - 1;
    left &= left - 1;
    r.i = __shfl_sync(0xffffffffu, mine.i, src);
    r.y = __shfl_sync(0xffffffffu, mine.y, src);
    r.run = __shfl_sync(0xffffffffu, mine.run, src);
    r.runs = __shfl_sync(0xffffffffu, mine.runs, src);
    r.u = __shfl_sync(0xffffffffu, mine.u, src);
    r.end = __shfl_sync(0xffffffffu, mine.end, src);
    r.head = __shfl_sync(0xffffffffu, mine.head, src);
    r.skip = __shfl_sync(0xffffffffu, mine.skip, src);
    live = true;
  }

  // zeros for a request without keys, NaN for a length that is not valid; one lane
  __device__ static void write_empty(const PagedDecode& a, const Run& c, int parts, bool bad) {
    const int group = a.hq / a.hkv, g0 = (c.y % parts) * kHeadsPerRun, heads = min(kHeadsPerRun, group - g0);
    const int64_t row = (int64_t)c.i * a.hq + (c.y / parts) * group + g0;
    const float x = bad ? __builtin_nanf("") : 0.f;
    for (int e = 0; e < heads * E::DIM; e += 4)
      store4(static_cast<typename E::Elem*>(a.out) + row * E::DIM + e, make_float4(x, x, x, x));
    if (a.lse)
      for (int h = 0; h < heads; ++h) a.lse[row + h] = bad ? x : -INFINITY;
  }

  __device__ __forceinline__ bool has_key(int lane) const { return lane < E::KEYS && r.u + lane < r.end; }

  __device__ __forceinline__ void look_up(const PagedDecode& a, int lane) {
    page = -1;
    if (!live || !has_key(lane)) return;
    const int b = r.key(r.u + lane) >> a.page_shift;
    if (b < a.max_blocks) page = a.block_table[(int64_t)r.i * a.max_blocks + b];
  }

  // The current tile into `stage`, then on to the next one (its rows are looked up meanwhile).
  // Eight lanes copy 128 bytes of a row (its last 64 or 128 at smaller rows); a lane meets the
  // rows G, G + step, ..., so that one shuffle and one address serve all of a row's pieces.
  __device__ __forceinline__ void fetch(const PagedDecode& a, int parts, uint32_t stage, int lane, Run* queue, int& tail) {
    if (live) {
      uint32_t row = ~0u;  // of this lane's key in the pages: none, or its page is outside the cache
      const bool lost = has_key(lane) && (page < 0 || page >= a.num_pages);
      if (has_key(lane) && !lost)
        row = (uint32_t)((((int64_t)page * a.hkv + r.y / parts) << a.page_shift) +
                         (r.key(r.u + lane) & ((1 << a.page_shift) - 1)));
      if (__any_sync(0xffffffffu, lost) && lane == 0) queue[(tail - 1) & 3].bad = 1;
      constexpr int PIECES = E::ROWB / 16, LANES = PIECES < 8 ? PIECES : 8;  // lanes of a row
      constexpr int ROWS = 32 / LANES, PARTS = PIECES / LANES;                // rows at a time, pieces of a lane
      const int g = lane / LANES, c = lane % LANES;
#pragma unroll
      for (int r0 = 0; r0 < E::KEYS; r0 += ROWS) {
        const uint32_t at = __shfl_sync(0xffffffffu, row, (r0 + g) % E::KEYS);
        if (ROWS > E::KEYS && g >= E::KEYS) break;
        const bool load = at != ~0u;
        const int64_t off = load ? (int64_t)at * E::ROWB + 16 * c : 0;
        const char *kp = static_cast<const char*>(a.k_pages) + off, *vp = static_cast<const char*>(a.v_pages) + off;
        const uint32_t dst = stage + E::place(r0 + g, c);
#pragma unroll
        for (int e = 0; e < PARTS; ++e) {  // place() moves by 128 bytes from piece c to c + 8
          cp_async16_or_zero(dst + 128 * e, kp + 128 * e, load);
          cp_async16_or_zero(dst + E::KEYS * E::ROWB + 128 * e, vp + 128 * e, load);
        }
      }
      step(a, parts, lane, queue, tail);
    }
    tc::cp_async_commit();
  }

  __device__ __forceinline__ void step(const PagedDecode& a, int parts, int lane, Run* queue, int& tail) {
    r.u += E::KEYS;
    if (r.u >= r.end) {
      seek(a, parts, lane);
      if (live) push(a, parts, queue, tail, lane);
    }
    look_up(a, lane);
  }
  // a run that is fetched from here on: at most the computed one, two fetched tiles' and the next are open
  __device__ __forceinline__ void push(const PagedDecode& a, int parts, Run* queue, int& tail, int lane) {
    r.bad = 0;
    if (lane == 0) queue[tail & 3] = r;
    const int group = a.hq / a.hkv, g0 = (r.y % parts) * kHeadsPerRun, heads = min(kHeadsPerRun, group - g0);
    const char* q = static_cast<const char*>(a.q) + ((int64_t)r.i * a.hq + (r.y / parts) * group + g0) * E::ROWB;
    for (int e = lane * 128; e < heads * E::ROWB; e += 32 * 128) tc::prefetch_l2(q + e);
    ++tail;
  }
};

template <typename E>
__global__ void __launch_bounds__(32 * DecodeSmem<E>::WARPS, 1) k_decode(const PagedDecode a, const int parts, const uint32_t chunk, int32_t* counter) {
  using L = DecodeSmem<E>;
  extern __shared__ __align__(128) unsigned char all[];
  unsigned char* sh = all + (threadIdx.x >> 5) * L::WARP;
  asm volatile("griddepcontrol.launch_dependents;");  // the join kernel may get ready
  const int lane = threadIdx.x & 31, group = a.hq / a.hkv;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->err = 0;  // set by the join kernel
  Run* queue = reinterpret_cast<Run*>(sh + L::QUEUE);
  const uint32_t ring = tc::smem_u32(sh);
  Walk<E> f;
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
    f.fetch(a, parts, ring + put * L::STAGE, lane, queue, tail);
    put = put + 1 == E::RING ? 0 : put + 1;
  }
  E eng;
  while (head != tail) {
    __syncwarp();
    Run r = queue[head & 3];
    const int g0 = (r.y % parts) * kHeadsPerRun, heads = min(kHeadsPerRun, group - g0);
    const int h0 = (r.y / parts) * group + g0;
    eng.start(a, (int64_t)r.i * a.hq + h0, heads, sh + L::EXTRA, lane);
    for (; r.u < r.end; r.u += E::KEYS) {
      // the next tile on its way first, into the place that every lane has read
      f.fetch(a, parts, ring + put * L::STAGE, lane, queue, tail);
      put = put + 1 == E::RING ? 0 : put + 1;
      asm volatile("cp.async.wait_group %0;" ::"n"(E::RING - 1) : "memory");
      __syncwarp();
      eng.tile(a, sh + get * L::STAGE, (int)(r.end - r.u), lane);
      get = get + 1 == E::RING ? 0 : get + 1;
      __syncwarp();
    }
    __syncwarp();
    eng.finish(Sink(a, r, h0, heads, sizeof(typename E::Elem)), queue[head & 3].bad != 0, lane);
    ++head;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------------------- join ----
// D / 4 lanes per (request, head) add the runs' records in ascending order, 16 at a time so that their
// loads are in flight together; more than 16 runs are shared out to the groups of lanes of a
// block that has the head to itself (SPLIT), whose sums are added in order.  How a request's runs are added
// depends on their number alone.  A request's CTAs also check its length and the pages of its
// visible keys for the error word.
constexpr int kJoinAtOnce = 16;
template <int D, typename T, bool SPLIT>
__global__ void __launch_bounds__(SPLIT ? 256 : 128) k_decode_join(const PagedDecode a) {
  constexpr int THREADS = SPLIT ? 256 : 128, LANES = D / 4, GROUPS = THREADS / LANES, B = kJoinAtOnce;
  __shared__ float4 so[SPLIT ? GROUPS : 1][LANES];
  __shared__ float2 sml[SPLIT ? GROUPS : 1];
  // what does not come from the runs' kernel is read while that still runs
  const int g = threadIdx.x / LANES, lane = threadIdx.x % LANES, c = 4 * lane;
  const int i = blockIdx.y, h = SPLIT ? blockIdx.x : blockIdx.x * GROUPS + g;
  const Request rq(a, a.seq_lens[i]);
  const int runs = split_of(rq.n, a.hkv).runs;
  const bool shared = SPLIT && runs > B;
  const int per = shared ? (runs + GROUPS - 1) / GROUPS : runs;
  const int begin = shared ? min(runs, g * per) : 0, end = shared ? min(runs, begin + per) : runs;
  bool lost = false;  // a page of the request's visible keys is outside the cache
  if (rq.n) {
    const int first = rq.key(rq.head) >> a.page_shift, last = (rq.len - 1) >> a.page_shift;
    const int head_pages = rq.head ? ((rq.head - 1) >> a.page_shift) + 1 : 0;
    for (int b = blockIdx.x * THREADS + threadIdx.x; b < head_pages + last - first + 1; b += gridDim.x * THREADS) {
      const int p = b < head_pages ? b : first + b - head_pages;
      const int page = p < a.max_blocks ? a.block_table[(int64_t)i * a.max_blocks + p] : -1;
      lost |= page < 0 || page >= a.num_pages;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the runs' kernel has finished
  if (rq.bad && threadIdx.x == 0) set_error(a.hdr, GDN_DEVERR_POS);
  if (lost) set_error(a.hdr, GDN_DEVERR_PAGES);
  if (runs > 1 && h < a.hq && (shared || !SPLIT || g == 0)) {
    const int64_t row = (int64_t)i * a.hq + h;
    const float* rec = a.partial + row * a.max_splits * D + c;
    const float2* mls =
        reinterpret_cast<const float2*>(a.partial + (int64_t)a.N * a.hq * a.max_splits * D) + row * a.max_splits;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float2 (&ml)[B], const float4 (&x)[B]) {
      float mx = m;
#pragma unroll
      for (int r = 0; r < B; ++r) mx = fmaxf(mx, ml[r].x);
      const float base = mx == -INFINITY ? 0.f : mx, f0 = exp2_approx(__fsub_rn(m, base));
      m = mx;
      l = __fmul_rn(l, f0);
      o = make_float4(__fmul_rn(o.x, f0), __fmul_rn(o.y, f0), __fmul_rn(o.z, f0), __fmul_rn(o.w, f0));
#pragma unroll
      for (int r = 0; r < B; ++r) {
        const float f = exp2_approx(__fsub_rn(ml[r].x, base));
        l = __fmaf_rn(f, ml[r].y, l);
        o = make_float4(__fmaf_rn(f, x[r].x, o.x), __fmaf_rn(f, x[r].y, o.y), __fmaf_rn(f, x[r].z, o.z),
                        __fmaf_rn(f, x[r].w, o.w));
      }
    };
    float2 ml[B];
    float4 x[B];
    for (int r0 = begin; r0 < end; r0 += B) {
#pragma unroll
      for (int r = 0; r < B; ++r) {
        ml[r] = make_float2(-INFINITY, 0.f);
        x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < end) {
          ml[r] = mls[r0 + r];
          x[r] = *reinterpret_cast<const float4*>(rec + (int64_t)(r0 + r) * D);
        }
      }
      add(ml, x);
    }
    if (shared) {
      so[g][lane] = o;
      if (lane == 0) sml[g] = make_float2(m, l);
      __syncthreads();  // every thread of the block is here: `shared` is the request's
      m = -INFINITY, l = 0.f, o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int g0 = 0; g0 < GROUPS; g0 += B) {
#pragma unroll
        for (int r = 0; r < B; ++r) {
          ml[r] = g0 + r < GROUPS ? sml[g0 + r] : make_float2(-INFINITY, 0.f);
          x[r] = g0 + r < GROUPS ? so[g0 + r][lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        add(ml, x);
      }
    }
    if (g == 0 || !SPLIT) {
      store4(static_cast<T*>(a.out) + row * D + c,
             make_float4(__fdiv_rn(o.x, l), __fdiv_rn(o.y, l), __fdiv_rn(o.z, l), __fdiv_rn(o.w, l)));
      if (a.lse && c == 0) a.lse[row] = __fmul_rn(__fadd_rn(m, log2f(l)), kLn2);
    }
  }
}

// The counter of a call whose warps take more than one chunk; the runs' kernel starts beside this.
__global__ void k_decode_clear(int32_t* counter) {
  asm volatile("griddepcontrol.launch_dependents;");
  *counter = 0;
}

template <typename E>
int launch_decode(const PagedDecode& a, cudaStream_t st) {
  constexpr int D = E::DIM, BYTES = DecodeSmem<E>::BYTES;
  static std::atomic<uint64_t> ready{0};
  ensure_smem(k_decode<E>, BYTES, ready);
  const int group = a.hq / a.hkv, parts = (group + kHeadsPerRun - 1) / kHeadsPerRun;
  const int64_t total = (int64_t)a.N * a.hkv * parts * a.max_splits, ctas = total < kSms ? total : kSms;
  const int64_t warps = ctas * DecodeSmem<E>::WARPS;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.stream = st;
  c.attrs = &attr;
  c.numAttrs = 0;
  int32_t* counter = nullptr;
  if (total > warps) {
    counter = a.hdr->pad;
    k_decode_clear<<<1, 1, 0, st>>>(counter);
    c.numAttrs = 1;
  }
  // about eight chunks a warp, of single slots unless there are many
  const int64_t chunk = total / (8 * warps);
  c.gridDim = dim3((unsigned)ctas);
  c.blockDim = dim3(32 * DecodeSmem<E>::WARPS);
  c.dynamicSmemBytes = BYTES;
  cudaLaunchKernelEx(&c, k_decode<E>, a, parts, (uint32_t)(chunk < 1 ? 1 : chunk > 32 ? 32 : chunk), counter);
  const bool split = a.max_splits > kJoinAtOnce;
  c.gridDim = dim3(split ? a.hq : (a.hq + 512 / D - 1) / (512 / D), a.N);
  c.blockDim = dim3(split ? 256 : 128);
  c.dynamicSmemBytes = 0;
  c.numAttrs = 1;
  if (split)
    cudaLaunchKernelEx(&c, k_decode_join<D, typename E::Elem, true>, a);
  else
    cudaLaunchKernelEx(&c, k_decode_join<D, typename E::Elem, false>, a);
  return counter ? 3 : 2;
}

template <int D, typename T>
int decode_t(const PagedDecode& a, cudaStream_t st) {
  const int group = a.hq / a.hkv;
  if constexpr (D >= 64 && sizeof(T) == 2) {
    return launch_decode<MmaEngine<D>>(a, st);
  } else {
    if (group <= 2) return launch_decode<SimtEngine<D, T, 2, 1>>(a, st);
    if (group <= 4) return launch_decode<SimtEngine<D, T, 4, 1>>(a, st);
    if (group <= 8) return launch_decode<SimtEngine<D, T, 4, 2>>(a, st);
    return launch_decode<SimtEngine<D, T, 4, 4>>(a, st);
  }
}

}  // namespace

// A bound on the runs of any request that sees at most `max_visible` keys: target_runs grows with n
// between the lengths where target_shift changes, and a request has at most target_runs runs.
int paged_decode_max_splits(int max_visible, int hkv) {
  int best = 1;
  for (const int64_t x : {128, 256, 512, 0}) {
    const int64_t last = x ? (kRunsPerRequest * x - 1) / hkv : max_visible;  // the last n before the next length
    const int n = (int)(last < max_visible ? last : max_visible);
    if (n > 0 && target_runs(n, hkv) > best) best = target_runs(n, hkv);
  }
  return best;
}

int launch_paged_decode(const PagedDecode& a, bool bf16, cudaStream_t st) {
  if (bf16) {
    if (a.d == 32) return decode_t<32, __nv_bfloat16>(a, st);
    if (a.d == 64) return decode_t<64, __nv_bfloat16>(a, st);
    return decode_t<128, __nv_bfloat16>(a, st);
  } else {
    if (a.d == 32) return decode_t<32, float>(a, st);
    if (a.d == 64) return decode_t<64, float>(a, st);
    return decode_t<128, float>(a, st);
  }
}

}  // namespace gdn
