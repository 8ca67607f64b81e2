// attn_window_tc.cu -- sliding-window attention for bf16 with d = 64 or 128 on the tensor cores.
//
// Forward.  A CTA (one per SM, persistent) takes work items of one head and 256 query rows as two tiles
// of 128.  Per key block of 128 and tile, S = Q K^T goes to TMEM; the tile's four softmax warps
// (one thread per row, so a row's maximum and sum need no exchange) take it into registers, which
// frees its place for the other tile's S, and leave P = exp2(c S - c m) as bf16 in a place of its own,
// from which O += P V reads it.  So TMEM holds S [128 columns], P of both tiles [2 x 64] and O of both
// [2 x d]; the scores of a tile's next block are formed while its warps work on the last, and the
// warps wait for the tensor core only where it is behind.  (With P written over S, the next S
// had to wait for P V: 921 us against 830 for 32768 tokens, window 4096, 16 / 4 heads, d = 128.  Two
// issuing warps instead of one then gave 707, items from a counter 690.)
// What bounds it: the tensor core (S and O += P V are 512 clocks each per 128 x 128 at d = 128).  That case takes
// 661 us in bursts of 30 calls (SM clock 2070 MHz; 1.56 PFLOP/s of visible scores' work, 84% of a large bf16
// library product's rate) and 690 to 720 over seconds, at the power limit (1930 MHz; 1.43 to 1.49, 77 to 81%).
// Where a window is short or sequences are, an item's start and end count (packed sequences of 1446 to 7386
// tokens, window 2048: 334 us at 57% tensor activity).
// The probabilities are rounded to bf16 for their product (the row sums are of the unrounded fp32
// values); S, O, m, l stay in 32 bits.  The maximum that P is scaled by is only moved, and O
// rescaled, when a true maximum of the warp's rows passes it by more than 2^8: P then stays below 2^8,
// where bf16 and fp32 are as exact as below 1, and the rescaling (a TMEM round trip) is rare.  Only the
// sequence's own rows count there, so that its bits do not depend on what follows it.  Blocks that no
// row of a tile sees are skipped tile by tile.
//
// Warps: 0-3 softmax of tile 0, 4-7 of tile 1, 8 issues the scores' products, 9 loads (TMA), 10
// issues P V, 11 only completes the warpgroup whose registers the softmax warps take over.  The loader
// publishes the items, runs ahead by the ring of key and value blocks, and zeroes the rows of a
// value block that lie past the sequence's end (they belong to another sequence, may hold NaN,
// and 0 x NaN is not 0).
#include <mutex>

#include "attn_tc.cuh"
#include "attn_window.cuh"

namespace gdn {

namespace {

using namespace win;
using namespace tc;

constexpr int BM = 128, BN = 128;  // rows of a query tile, keys of a block
constexpr int kWarps = 12, kThreads = 32 * kWarps, kScoreWarp = 8, kLoadWarp = 9, kAccWarp = 10;
// 384 threads x 168 registers at launch = 256 x 208 + 128 x 88: a softmax thread holds a row's 128
// scores
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kSms = 152;

struct Item {
  int ok;  // 0: no more items
  int h, row0;
  Seq q;
};

// Key blocks of one tile of query rows, and of an item's two tiles together.
struct Tile {
  int rows, head, from, to;
  __device__ __forceinline__ Tile(const WindowAttn& a, const Item& it, int r0) {
    const int off = it.q.Lk - it.q.Lq;
    rows = max(0, min(BM, it.q.Lq - r0));
    head = from = to = 0;
    if (rows) {
      const KeyBlocks kb(r0 + off, r0 + rows - 1 + off, it.q.Lk, a.window, a.sinks, BN);
      head = kb.head, from = kb.from, to = kb.to;
    }
  }
  __device__ __forceinline__ void uniform_all() { head = uniform(head), from = uniform(from), to = uniform(to); }
  __device__ __forceinline__ bool any() const { return head + to - from > 0; }
  __device__ __forceinline__ bool need(int b) const { return b < head || (b >= from && b < to); }
};
struct Plan {
  Tile t0, t1;
  int head, from, to;
  __device__ __forceinline__ Plan(const WindowAttn& a, const Item& it) : t0(a, it, it.row0), t1(a, it, it.row0 + BM) {
    if (!t1.any()) head = t0.head, from = t0.from, to = t0.to;
    else if (!t0.any()) head = t1.head, from = t1.from, to = t1.to;
    else from = min(t0.from, t1.from), to = max(t0.to, t1.to), head = min(max(t0.head, t1.head), from);
  }
  __device__ __forceinline__ int count() const { return head + to - from; }
  __device__ __forceinline__ int block(int i) const { return i < head ? i : from + (i - head); }
  __device__ __forceinline__ bool need(int t, int b) const { return t ? t1.need(b) : t0.need(b); }
  __device__ __forceinline__ void uniform_all() {
    t0.uniform_all();
    t1.uniform_all();
    head = uniform(head), from = uniform(from), to = uniform(to);
  }
};

// bits c < n of a word
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

template <int D>
struct FwdSmem {
  static constexpr int TILE = BM * D * 2, STAGES = D == 128 ? 4 : 8;
  static constexpr int Q = 0, KV = 2 * TILE, BARS = KV + STAGES * TILE;
  static constexpr int BYTES = BARS + 1024 + 1024;  // barriers and items; alignment
};

struct FwdBars {
  uint64_t item_full[2], item_empty[2], q_full, q_empty, kv_full[8], kv_empty[8], s_full[2], s_free, p_full[2], pv_done[2],
      o_empty[2], aux, drain[2];
  uint32_t tmem;
  Item item[2];
};
static_assert(sizeof(FwdBars) <= 1024, "fits its place");

// FAULT: the test hook's form, which gives up at once.
template <int D, bool FAULT>
__global__ void __launch_bounds__(kThreads, 1)
    k_window_fwd_tc(const WindowAttn a, const int64_t items, int* next_item, const __grid_constant__ CUtensorMap mq,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using L = FwdSmem<D>;
  extern __shared__ unsigned char raw[];
  unsigned char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  FwdBars& B = *reinterpret_cast<FwdBars*>(sm + L::BARS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0) check_tables(a);
  if (warp == kScoreWarp) tmem_alloc(&B.tmem, 512);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.item_full[i], 1);
      mbar_init(&B.item_empty[i], 10);  // all warps but the loader and the idle one
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_full[i], 4);
      mbar_init(&B.pv_done[i], 1);
      mbar_init(&B.o_empty[i], 4);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&B.kv_full[i], 1);
      mbar_init(&B.kv_empty[i], 1);
    }
    mbar_init(&B.s_free, 4);
    mbar_init(&B.q_full, 1);
    mbar_init(&B.q_empty, 1);
    mbar_init(&B.aux, 1);
    mbar_init(&B.drain[0], 1);
    mbar_init(&B.drain[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t tm = B.tmem;
  const uint32_t tS = tm, tP[2] = {tm + 128, tm + 192}, tO[2] = {tm + 256, tm + 256 + D};
  bool ok = true;

  if constexpr (FAULT) {
    ok = wait_for_nothing(&mq, sm + L::Q, BM * 128, &B.q_full, &B.drain[0], warp == kLoadWarp && a.Tq > 0);
  } else if (warp >= 8) {
    regs_less<kOtherRegs>();
    if (warp == kLoadWarp) {
    // ------------------------------------------------------------------ loader ----
    uint32_t n = 0, stage = 0, round = 0, aux = 0, qn = 0;
    int64_t w = blockIdx.x;
    while (ok) {
      Item it;
      it.ok = w < items * a.hq;
      if (it.ok) {
        it.h = (int)(w % a.hq);
        it.q = find_seq(a, items - 1 - w / a.hq, 2 * BM, false, it.row0);  // a sequence's last blocks see most
        int nx = 0;
        if (lane == 0 && next_item) nx = atomicAdd(next_item, 1);
        w = next_item ? (int64_t)gridDim.x + __shfl_sync(0xffffffffu, nx, 0) : items * a.hq;
        if (!it.q.ok) continue;
      }
      const uint32_t slot = n & 1;
      ok = ok && mbar_wait(&B.item_empty[slot], ((n >> 1) & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        B.item[slot] = it;
        mbar_arrive(&B.item_full[slot]);
      }
      ++n;
      if (!it.ok) break;
      const Plan p(a, it);
      if (!p.count()) continue;
      ok = mbar_wait(&B.q_empty, (qn & 1) ^ 1);
      if (!ok) break;
      ++qn;
      if (lane == 0) {
        mbar_expect_tx(&B.q_full, L::TILE * ((p.t0.rows ? 1 : 0) + (p.t1.rows ? 1 : 0)));
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (t ? p.t1.rows : p.t0.rows)
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sm + L::Q + t * L::TILE + c * BM * 128, &mq, 64 * c, it.h, it.q.q0 + it.row0 + BM * t,
                          &B.q_full);
      }
      const int kvh = it.h / (a.hq / a.hkv);
      for (int i = 0; i < p.count() && ok; ++i) {
        const int j0 = p.block(i) * BN;
        for (int kv = 0; kv < 2; ++kv) {
          ok = mbar_wait(&B.kv_empty[stage], (round & 1) ^ 1);
          if (!ok) break;
          unsigned char* dst = sm + L::KV + stage * L::TILE;
          const bool tail = kv == 1 && j0 + BN > it.q.Lk;
          uint64_t* bar = tail ? &B.aux : &B.kv_full[stage];
          if (lane == 0) {
            mbar_expect_tx(bar, L::TILE);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(dst + c * BN * 128, kv ? &mv : &mk, 64 * c, kvh, it.q.k0 + j0, bar);
          }
          if (tail) {
            ok = mbar_wait(&B.aux, aux & 1);
            ++aux;
            if (!ok) break;
            const int r0 = it.q.Lk - j0;
            for (int e = lane; e < (BN - r0) * 8 * (D / 64); e += 32) {
              const int c = e / ((BN - r0) * 8), x = e % ((BN - r0) * 8);
              *reinterpret_cast<uint4*>(dst + c * BN * 128 + r0 * 128 + x * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.kv_full[stage]);
          }
          if (++stage == L::STAGES) stage = 0, ++round;
        }
      }
    }
    } else if (warp == kScoreWarp || warp == kAccWarp) {
      // --------------------------------------------------------------------- MMA ----
      // One warp issues the scores' products, another P V: an issuing thread stands still while its
      // products run, and each wait costs it a few hundred cycles.  The warps stay converged, and
      // each group of MMAs is issued by its elected lane: the compiler then knows that there is one,
      // and keeps descriptors in uniform registers.
      const bool scores = warp == kScoreWarp;
      const uint32_t iS = idesc_bf16(BM, BN), iO = idesc_bf16(BM, D) | IDESC_B_MN;
      const uint64_t dQ = desc_k_sw128(smem_u32(sm + L::Q)), dK = desc_k_sw128(smem_u32(sm + L::KV));
      const uint64_t dV = desc_mn_sw128(smem_u32(sm + L::KV), BN * 128);
      constexpr int STEP = L::TILE / 16;  // of a descriptor, from one tile to the next
      uint32_t n = 0, qn = 0, sn = 0, np[2] = {0, 0}, no[2] = {0, 0};
      uint32_t stage = scores ? 0 : 1, round = 0;  // of the next key or value block
      while (ok) {
        const uint32_t slot = n & 1;
        ok = warp_wait(&B.item_full[slot], (n >> 1) & 1);
        if (!ok) break;
        Item it = B.item[slot];
        __syncwarp();
        if (elect_one()) mbar_arrive(&B.item_empty[slot]);
        ++n;
        if (!uniform(it.ok)) break;
        Plan p(a, it);
        p.uniform_all();
        const int cnt = p.count();
        if (!cnt) continue;
        if (scores) {
          ok = warp_wait(&B.q_full, qn & 1);
          ++qn;
        }
        bool started[2] = {false, false};
        for (int i = 0; i < cnt && ok; ++i) {
          const int b = p.block(i);
          ok = warp_wait(&B.kv_full[stage], round & 1);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || !p.need(t, b)) continue;
            if (scores) {
              ok = warp_wait(&B.s_free, (sn & 1) ^ 1);  // the last scores are in registers
              ++sn;
              if (!ok) continue;
              fence_after_sync();
              if (elect_one()) {
                mma_rows<D, BM, BN>(tS, dQ + t * STEP, dK + stage * STEP, iS);
                mma_commit(&B.s_full[t]);
              }
            } else {
              ok = warp_wait(&B.p_full[t], np[t] & 1);
              ++np[t];
              if (!started[t]) {  // the last item's output has left TMEM
                ok = ok && warp_wait(&B.o_empty[t], (no[t] & 1) ^ 1);
                ++no[t];
              }
              if (!ok) continue;
              fence_after_sync();
              if (elect_one()) {
                mma_ts_cols<BN>(tO[t], tP[t], dV + stage * STEP, iO, started[t]);
                mma_commit(&B.pv_done[t]);
              }
              started[t] = true;
            }
          }
          if (!ok) break;
          if (elect_one()) {
            mma_commit(&B.kv_empty[stage]);
            if (scores && i + 1 == cnt) mma_commit(&B.q_empty);
          }
          stage += 2;
          if (stage >= L::STAGES) stage -= L::STAGES, ++round;
        }
      }
    }
  } else {
    // ----------------------------------------------------------------- softmax ----
    regs_more<kSoftmaxRegs>();
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t sS = tmem_lane_addr(tS, warp, 0), sP = tmem_lane_addr(tm + 128 + 64 * t, warp, 0), sO = tmem_lane_addr(tm + 256 + D * t, warp, 0);
    const float sc = __fmul_rn(a.scale, kLog2e);
    const float2 sc2 = make_float2(sc, sc);
    uint32_t n = 0, ns = 0, npv = 0;
    while (ok) {
      const uint32_t slot = n & 1;
      ok = mbar_wait(&B.item_full[slot], (n >> 1) & 1);
      if (!ok) break;
      const Item it = B.item[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.item_empty[slot]);
      ++n;
      if (!it.ok) break;
      const Plan p(a, it);
      const Tile tile = t ? p.t1 : p.t0;
      if (!tile.rows) continue;
      const int cnt = tile.head + tile.to - tile.from, r0 = it.row0 + BM * t, p0 = r0 + it.q.Lk - it.q.Lq;
      const int p1 = p0 + tile.rows - 1, pos = p0 + row;
      const int lo = a.window > 0 ? pos - a.window + 1 : 0;
      // The maximum that P and O are scaled by.  Rows past the sequence's end, which hold another's queries,
      // start above all: they never decide by which maximum the warp's other rows are scaled.
      float m = row < tile.rows ? -INFINITY : INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      bool started = false;
      for (int i = 0; i < cnt; ++i) {
        const int j0 = (i < tile.head ? i : tile.from + (i - tile.head)) * BN;
        ok = mbar_wait(&B.s_full[t], ns & 1);
        ++ns;
        if (!ok) break;
        fence_after_sync();
        float s[BN];
        tmem_ld128(sS, s);
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.s_free);
        if (j0 + BN - 1 > p0 || (a.window > 0 && p1 - j0 >= a.window && j0 + BN > a.sinks)) {  // some row does not see all of it
#pragma unroll
          for (int g = 0; g < BN; g += 32) {
            const int at = j0 + g;
            const uint32_t see = below(pos + 1 - at) & (~below(lo - at) | below(a.sinks - at));
#pragma unroll
            for (int c = 0; c < 32; ++c) s[g + c] = (see & (1u << c)) ? s[g + c] : -INFINITY;
          }
        }
        float mx = fmaxf(s[0], s[1]), my = fmaxf(s[2], s[3]);
#pragma unroll
        for (int c = 4; c < BN; c += 4) mx = max3(mx, s[c], s[c + 1]), my = max3(my, s[c + 2], s[c + 3]);
        mx = fmaxf(mx, my);
        const bool move = __fmul_rn(__fsub_rn(mx, m), sc) > 8.f;  // true for a live row's first finite maximum
        if (started) {  // P V of the last block is done: P's place is free, and O at rest
          ok = mbar_wait(&B.pv_done[t], (npv - 1) & 1);
          if (!ok) break;
          fence_after_sync();
        }
        if (__any_sync(0xffffffffu, move)) {
          const float mn = fmaxf(m, mx);
          if (started) {
            const float f = m == -INFINITY ? 0.f : exp2_approx(__fmul_rn(__fsub_rn(m, mn), sc));
            l2.x = __fmul_rn(l2.x, f);
            l2.y = __fmul_rn(l2.y, f);
#pragma unroll
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld16(sO + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __fmul_rn(o[e], f);
              tmem_st16(sO + c, o);
            }
          }
          m = mn;
        }
        const float mc = m == -INFINITY ? 0.f : -__fmul_rn(m, sc);
        const float2 mc2 = make_float2(mc, mc);
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float2 x = fma2(make_float2(s[32 * part + 2 * c], s[32 * part + 2 * c + 1]), sc2, mc2);
            x.x = exp2_approx(x.x);
            x.y = exp2_approx(x.y);
            l2 = add2(l2, x);
            pk[c] = pack_bf16(x.x, x.y);
          }
          tmem_st16u(sP + 16 * part, pk);
        }
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.p_full[t]);
        started = true;
        ++npv;
      }
      if (!ok) break;
      // the row's output
      const float l = __fadd_rn(l2.x, l2.y), inv = __frcp_rn(l);
      const int64_t at = (int64_t)(it.q.q0 + r0 + row) * a.hq + it.h;
      const bool write = row < tile.rows;
      if (started) {
        ok = mbar_wait(&B.pv_done[t], (npv - 1) & 1);
        if (!ok) break;
        fence_after_sync();
      }
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at * D;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (started) tmem_ld32(sO + c, o);
        if (write) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (started && l != 0.f)
              u = make_uint4(pack_bf16(__fmul_rn(o[e], inv), __fmul_rn(o[e + 1], inv)),
                             pack_bf16(__fmul_rn(o[e + 2], inv), __fmul_rn(o[e + 3], inv)),
                             pack_bf16(__fmul_rn(o[e + 4], inv), __fmul_rn(o[e + 5], inv)),
                             pack_bf16(__fmul_rn(o[e + 6], inv), __fmul_rn(o[e + 7], inv)));
            *reinterpret_cast<uint4*>(out + c + e) = u;
          }
        }
      }
      if (started) {
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.o_empty[t]);
      }
      if (write) a.lse[at] = l == 0.f ? -INFINITY : __fmul_rn(__fadd_rn(__fmul_rn(m, sc), log2f(l)), kLn2);
    }
  }
  if (!ok) set_error(a.hdr, GDN_DEVERR_TIMEOUT);
  if (__syncthreads_or(!ok)) {
    // something gave up: copies and MMAs that were issued end before the memory is given back
    if (warp == kLoadWarp && lane == 0) {
      for (int i = 0; i < L::STAGES; ++i) settle(&B.kv_full[i]);
      settle(&B.q_full);
      settle(&B.aux);
    }
    if (warp == kScoreWarp || warp == kAccWarp) settle_mma(&B.drain[warp == kAccWarp]);
  }
  __syncthreads();
  if (warp == kScoreWarp) tmem_dealloc(tm, 512);
}

template <int D, bool FAULT>
bool fwd_tc(const WindowAttn& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  if (!make_rows_map(&mq, a.q, a.Tq, a.hq, D, BM, a.hdr) || !make_rows_map(&mk, a.k, a.Tk, a.hkv, D, BN, a.hdr) ||
      !make_rows_map(&mv, a.v, a.Tk, a.hkv, D, BN, a.hdr))
    return false;
  const int64_t items = item_count(a.Tq, 2 * BM, a.N), work = items * a.hq;
  static std::atomic<uint64_t> ready{0};
  ensure_smem(k_window_fwd_tc<D, FAULT>, FwdSmem<D>::BYTES, ready);
  // more items than CTAs: they take the next one from a counter, as sequences' blocks differ in work
  int* next_item = nullptr;
  if (work > kSms) {
    if (cudaMemsetAsync(a.hdr, 0, sizeof(WsHeader), st) != cudaSuccess) return false;
    next_item = a.hdr->pad;
  }
  k_window_fwd_tc<D, FAULT><<<(unsigned)(work < kSms ? work : kSms), kThreads, FwdSmem<D>::BYTES, st>>>(
      a, items, next_item, mq, mk, mv);
  return true;
}

}  // namespace

bool make_rows_map(CUtensorMap* map, const void* base, int T, int H, int d, int rows, const void* any) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Encode encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<Encode>(f);
  });
  if (!encode) return false;
  if (T == 0) base = any, T = 1;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool launch_window_fwd_tc(const WindowAttn& a, cudaStream_t st) {
  if (a.fault_wait) return a.d == 128 ? fwd_tc<128, true>(a, st) : fwd_tc<64, true>(a, st);
  return a.d == 128 ? fwd_tc<128, false>(a, st) : fwd_tc<64, false>(a, st);
}

}  // namespace gdn
