// attn.h -- internal interface of the attention-layer operators: the C-ABI host code
// (attn_host.cu) checks arguments and calls these launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/gdn_cpr.h"
#include "common.cuh"

namespace gdn {

// ------------------------------------------------------------- norms and rotation ----
struct NormRope {
  int T, hq, hk, rot, table_rows;
  int norm, layout;  // gdn_norm, gdn_rope_layout
  float eps;
  int64_t q_stride, k_stride, v_stride;
  const void *q, *k, *v;
  const float *wq, *wk, *cos, *sin;
  const int32_t* pos;
  void *q_out, *k_out, *k_pages, *v_pages;
  int page_shift;
  int64_t slots;
  const int32_t* slot_map;
  // backward
  const void *gq, *gk;
  void *dq, *dk;
  float* partial;  // [blocks][2][d] sums of the weights' gradients
  float *dwq, *dwk;
};
// launchers return how many kernels they queued where that varies
void launch_norm_rope(const NormRope& a, int d, bool in_bf16, bool out_bf16, cudaStream_t st);
int launch_norm_rope_bwd(const NormRope& a, int d, bool in_bf16, bool grad_bf16, cudaStream_t st);
// at most, as many as are resident; fixes the order of the weights' sums (1216: 1 to 2% slower, 1824: 3%)
constexpr int kNormBwdBlocks = 608;

// ------------------------------------------------------------------- page tables ----
constexpr int kPageMapMaxSeqs = 8192;
struct PageMap {
  int N, T, page_shift, max_blocks, num_free;
  const int32_t *lens, *new_lens, *free_pages;
  int32_t *block_table, *seq_lens, *cu, *positions, *slot_map, *pages_used;
  WsHeader* hdr;
};
void launch_page_map(const PageMap& a, cudaStream_t st);

// ------------------------------------------------------------------ paged decode ----
struct PagedDecode {
  int N, hq, hkv, d, window, sinks, max_len;
  float scale;
  const void *q, *k_pages, *v_pages;
  int num_pages, page_shift, max_blocks;
  const int32_t *block_table, *seq_lens;
  void* out;
  float* lse;
  float* partial;  // [N, hq, max_splits] records of d + 2 floats
  int max_splits;
  WsHeader* hdr;
};
// Visible keys of a request with `len` keys (device and host use the same rule).
__host__ __device__ inline int visible_keys(int len, int window, int sinks) {
  if (window <= 0 || len <= window) return len;
  const int behind = len - window;
  return window + (sinks < behind ? sinks : behind);
}
// Keys of one run, from the request's visible keys and the number of key heads alone, so that a
// request's result does not depend on the batch: about kRunsPerRequest runs over a request's heads,
// of 64 to 512 keys, evened out and a multiple of 32 (a tile).  With 16 runs 48 requests of 1004
// visible keys took 37.7 us against 35.6, with 64 runs 256 requests of about 2112 keys took 350 against
// 328; with at most 256 keys a run these took 346, and 7 requests of 4 to 22 thousand 29.0 against 23.8
// (but 6 of 15 to 30 thousand at d = 128, whose runs just fill the warps, 60 against 69).
constexpr int kRunsPerRequest = 32;
__host__ __device__ inline int target_shift(int n, int hkv) {
  const int64_t x = (int64_t)n * hkv;
  return x < 128 * kRunsPerRequest ? 6 : x < 256 * kRunsPerRequest ? 7 : x < 512 * kRunsPerRequest ? 8 : 9;
}
__host__ __device__ inline int target_runs(int n, int hkv) {
  const int s = target_shift(n, hkv), r = (int)(((unsigned)n + (1u << s >> 1)) >> s);  // n + 256 may pass 2^31
  return r < 1 ? 1 : r;
}
struct Split {
  int keys, runs;  // of a run, of a request
};
__host__ __device__ inline Split split_of(int n, int hkv) {
  const unsigned r = (unsigned)target_runs(n, hkv);
  Split s;
  s.keys = (int)((((unsigned)n + r - 1) / r + 31) / 32 * 32);
  s.runs = n == 0 ? 0 : (int)(((unsigned)n + s.keys - 1) / (unsigned)s.keys);
  return s;
}
int paged_decode_max_splits(int max_visible, int hkv);
int launch_paged_decode(const PagedDecode& a, bool bf16, cudaStream_t st);

// -------------------------------------------------------------- window attention ----
struct WindowAttn {
  int N, Tq, Tk, hq, hkv, d, window, sinks;
  float scale;
  const int32_t *cu_q, *cu_k;
  const void *q, *k, *v;
  void* out;
  float* lse;
  // backward
  const void* dout;
  void *dq, *dk, *dv;
  int few;       // rows at positions [0, few) have their delta from k_window_delta; 0 in fp32
  float* delta;  // 2 Tq hq floats that dq leaves for dk, dv: do . o [Tq, hq] (fp32 SIMT), or
                 // lse log2 e [hq, Tq] (infinite for a row that sees nothing) and do . o [hq, Tq]
  WsHeader* hdr;
  int fault_wait;  // test hook of the tensor-core kernels: they start a copy, wait for a phase that nothing
                   // completes, and give up
};
// false: nothing was queued
bool launch_window_attn(const WindowAttn& a, bool bf16, cudaStream_t st);
// tensor-core kernels: bf16, d = 64 or 128; false if a tensor map cannot be made
bool launch_window_fwd_tc(const WindowAttn& a, cudaStream_t st);
bool launch_window_dq_tc(const WindowAttn& a, cudaStream_t st);
bool launch_window_dkv_tc(const WindowAttn& a, cudaStream_t st);
// bf16: delta of the rows that see 1 to kFewKeys keys, from do . v and the probabilities.  From the output, which is
// rounded to bf16, it is off by u |do . o|, and with few keys do . v_j - delta is not much larger: on unit-size
// inputs 39% of the rows that see 2 keys got a dq more than 5e-3 off (some by its own size), 4% with 8 keys,
// 1% with 16, 0.2% with 32; a delta in 32 bits leaves 0.04% at most.
constexpr int kFewKeys = 16;
// These are the rows at positions [0, few): a row sees min(position + 1, window + sinks) keys.
inline int few_positions(int window, int sinks) {
  return window > 0 && (int64_t)window + sinks <= kFewKeys ? INT32_MAX : kFewKeys;
}
__device__ __forceinline__ bool few_keys(int pos, int few) { return (unsigned)pos < (unsigned)few; }
void launch_window_delta(const WindowAttn& a, cudaStream_t st);
// the gradient: dq (and delta, of few-key rows by a kernel before it), then dk and dv, which read delta
bool launch_window_dq(const WindowAttn& a, bool bf16, cudaStream_t st);
bool launch_window_dkv(const WindowAttn& a, bool bf16, cudaStream_t st);

// Opts a kernel into `bytes` of dynamic shared memory, once per (kernel, device): a call of the
// runtime costs as much as a launch.  `done` is the kernel's own flag word.
template <typename F>
inline void ensure_smem(F* fn, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess)
    done.fetch_or(bit, std::memory_order_release);
}

// ------------------------------------------------------------------------ device ----
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}

}  // namespace gdn
