// attn_decode.cuh -- what decode attention over the paged cache and over the 8-bit one share: a warp takes a run of a
// request's visible keys and leaves (m, l, a) or the output, and k_decode_join adds a request's runs in ascending
// order.  An engine E has a Kind with the types Args (the call) and Request (of a length: its runs), check(), what
// is wrong with a request's pages, and divisor(), the sum of its probabilities on the scale of its records' a; and a type Run.
#pragma once

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

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void* gmem, bool load) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(load ? 16 : 0) : "memory");
}

// Where a run's (m, l, a) or output goes: rows of its heads.
struct Sink {
  float* acc;   // record of head 0's run, or NULL: the run is the whole request
  float2* ml;
  int64_t acc_step, ml_step;  // from one head to the next
  void* out;                  // row of head 0
  float* lse;
  int heads;
  template <typename R>
  __device__ __forceinline__ Sink(const PagedDecode& a, const R& r, int h0, int heads_, int elem) : heads(heads_) {
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

// --------------------------------------------------------------------- dealing out ----
// One CTA per SM with as many warps as its shared memory has rings for (7, or as many on each
// scheduler: 13 warps instead of 12 at d = 64 cost 200 requests 249 us against 225).  First slots are
// dealt out across the SMs before a second warp of any gets one, so that a few runs spread over
// all of them: with several smaller CTAs an SM, some SMs got three busy ones and some none (7 requests
// of 4 to 22 thousand tokens, d = 64: 28.1 us against 23.9; 4 of about 700: 10.2 against 9.0).
template <typename E>
struct DecodeSmem {
  static constexpr int STAGE = E::STAGE, RING = E::RING * STAGE, EXTRA = RING, QUEUE = EXTRA + E::EXTRA;
  static constexpr int WARP = (QUEUE + 4 * (int)sizeof(typename E::Run) + 127) / 128 * 128, MOST = 227 * 1024 / WARP;
  static constexpr int FEW = MOST < E::MOST_WARPS ? MOST : E::MOST_WARPS;
  static constexpr int WARPS = FEW < 8 ? FEW : FEW / 4 * 4, HALF = 116 * 1024;
  static constexpr int BYTES = WARPS * WARP > HALF ? WARPS * WARP : HALF;  // more than half: one CTA per SM
};

// ---------------------------------------------------------------------------- join ----
// D / 4 lanes per (request, head) add the runs' records in ascending order, 16 at a time so that their
// loads are in flight together; more than 16 runs are shared out to the groups of lanes of a
// block that has the head to itself (SPLIT), whose sums are added in order.  How a request's runs are added
// depends on their number alone.  A request's CTAs also check its length and the pages of its
// visible keys for the error word.
constexpr int kJoinAtOnce = 16;
template <typename Kind, int D, typename T, bool SPLIT>
__global__ void __launch_bounds__(SPLIT ? 256 : 128) k_decode_join(const typename Kind::Args a) {
  constexpr int THREADS = SPLIT ? 256 : 128, LANES = D / 4, GROUPS = THREADS / LANES, B = kJoinAtOnce;
  __shared__ float4 so[SPLIT ? GROUPS : 1][LANES];
  __shared__ float2 sml[SPLIT ? GROUPS : 1];
  // what does not come from the runs' kernel is read while that still runs
  const int g = threadIdx.x / LANES, lane = threadIdx.x % LANES, c = 4 * lane;
  const int i = blockIdx.y, h = SPLIT ? blockIdx.x : blockIdx.x * GROUPS + g;
  const typename Kind::Request rq(a, a.seq_lens[i]);
  const int runs = rq.runs(a);
  const bool shared = SPLIT && runs > B;
  const int per = shared ? (runs + GROUPS - 1) / GROUPS : runs;
  const int begin = shared ? min(runs, g * per) : 0, end = shared ? min(runs, begin + per) : runs;
  // what is wrong with the request's pages; its blocks share the work
  const int wrong = Kind::check(a, rq, i, blockIdx.x * THREADS + threadIdx.x, gridDim.x * THREADS);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the runs' kernel has finished
  if (rq.bad && threadIdx.x == 0) set_error(a.hdr, GDN_DEVERR_POS);
  if (wrong) set_error(a.hdr, wrong);
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
      const float by = Kind::divisor(rq, l);
      store4(static_cast<T*>(a.out) + row * D + c,
             make_float4(__fdiv_rn(o.x, by), __fdiv_rn(o.y, by), __fdiv_rn(o.z, by), __fdiv_rn(o.w, by)));
      if (a.lse && c == 0) a.lse[row] = __fmul_rn(__fadd_rn(m, log2f(l)), kLn2);
    }
  }
}

// The counter of a call whose warps take more than one chunk; the runs' kernel starts beside this.
__global__ void k_decode_clear(int32_t* counter) {
  asm volatile("griddepcontrol.launch_dependents;");
  *counter = 0;
}

// Queues a call: `kernel` walks over the runs, k_decode_join joins them.
template <typename E>
int launch_decode(void (*kernel)(typename E::Args, int, uint32_t, int32_t*), const typename E::Args& a, cudaStream_t st) {
  constexpr int D = E::DIM, BYTES = DecodeSmem<E>::BYTES;
  static std::atomic<uint64_t> ready{0};
  ensure_smem(kernel, BYTES, ready);
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
  cudaLaunchKernelEx(&c, kernel, a, parts, (uint32_t)(chunk < 1 ? 1 : chunk > 32 ? 32 : chunk), counter);
  const bool split = a.max_splits > kJoinAtOnce;
  c.gridDim = dim3(split ? a.hq : (a.hq + 512 / D - 1) / (512 / D), a.N);
  c.blockDim = dim3(split ? 256 : 128);
  c.dynamicSmemBytes = 0;
  c.numAttrs = 1;
  if (split)
    cudaLaunchKernelEx(&c, k_decode_join<typename E::Kind, D, typename E::Elem, true>, a);
  else
    cudaLaunchKernelEx(&c, k_decode_join<typename E::Kind, D, typename E::Elem, false>, a);
  return counter ? 3 : 2;
}

}  // namespace

}  // namespace gdn
