// attn_window_bwd_tc.cu -- gradient of sliding-window attention for bf16 with d = 64 or 128 on the
// tensor cores.  Two kernels of one form, so that nothing is added across CTAs and the result
// does not depend on their order:
//   dq      rows = 128 queries of a head, columns = blocks of 128 keys:   dQ += dS K
//   dk, dv  rows = 128 keys of a key head, columns = blocks of 64 queries of each head of the group in
//           ascending order:   dK += dS^T Q,  dV += P^T dO
// with P = exp2(c Q K^T - lse log2 e) and dS = P (dO V^T - delta) formed anew in both (7 products
// where one kernel that adds dQ across CTAs would need 5).  The row tiles X, Y (Q and dO, or K and
// V) stay in shared memory; column tiles U, W come by TMA.  S = X U^T and T = Y W^T go to TMEM; two
// groups of four warps, a thread per row, take them into registers, which frees their place for
// the next block's, and leave dS and P as bf16 in one of two places of their own, from which the
// accumulating products read them while the groups are at the next block.  In dq the groups share
// a block's columns, in dk, dv they take alternate blocks.
// P and dS are rounded to bf16 for their products, as their other operands are; everything else
// stays in 32 bits.  delta = do . o takes the forward's output, which is rounded to bf16, but for rows that see
// few keys, where dP - delta would show it (k_window_delta).
// What bounds them: a 128 x 128 block needs 512 clocks of the tensor core per product at d = 128, and
// shared memory, at 128 bytes a clock, 512 for S and T each, 256 for an accumulating product and
// 512 to take in U and W: 1792 against 1536 in dq.  At 128 x 64 (dk, dv, whose accumulators leave
// TMEM no room for more) it is 1280 against 1024.  Packed training case (32387 tokens of 16/4 heads,
// window 2048): dq 531 us at 54% tensor activity, dk and dv 619 us at 61%.  With the rows in TMEM and
// 64 columns dq took 599 us; with one ring for U and W 627; with S and T issued by two warps 521,
// but dk and dv then 764; with one loading warp for both rings dq 636 and dk, dv 754; with four groups
// of 32 columns dq 539.
#include "attn_tc.cuh"
#include "attn_window.cuh"

namespace gdn {

namespace {

using namespace win;
using namespace tc;

constexpr int BR = 128;  // rows of a block
template <bool DKV>
constexpr int kCols = DKV ? 64 : 128;  // its columns
constexpr int kThreads = 384, kScoreWarp = 8, kLoadWarp = 9, kAccWarp = 10, kLoadWarp2 = 11;
// 384 threads x 168 registers at launch = 256 x 208 + 128 x 88
constexpr int kRowRegs = 208, kOtherRegs = 88;
constexpr int kSms = 152;

struct Item {
  int ok;  // 0: no more items
  int h, row0;
  Seq q;
};

// bits c < n of a word
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// The column blocks of an item: for dq key blocks, for dk and dv the query blocks of each head.
template <bool DKV>
struct Cols {
  static constexpr int BC = kCols<DKV>;
  int rows, cnt, head, from, nb, off;
  __device__ __forceinline__ Cols(const WindowAttn& a, const Item& it) {
    off = it.q.Lk - it.q.Lq;
    head = 0;
    if (DKV) {
      rows = min(BR, it.q.Lk - it.row0);
      const QueryRange r(it.q, it.row0, it.row0 + rows, a.window, a.sinks);
      from = r.lo / BC;
      nb = r.hi > r.lo ? (r.hi + BC - 1) / BC - from : 0;
      cnt = nb * (a.hq / a.hkv);
    } else {
      rows = min(BR, it.q.Lq - it.row0);
      const int p0 = it.row0 + off;
      const KeyBlocks kb(p0, p0 + rows - 1, it.q.Lk, a.window, a.sinks, BC);
      head = kb.head;
      from = kb.from;
      cnt = nb = kb.count();
    }
  }
  // first column of block i, and for dk, dv its head within the group
  __device__ __forceinline__ int col0(int i) const {
    if (DKV) return (from + i % nb) * BC;
    return (i < head ? i : from + (i - head)) * BC;
  }
  __device__ __forceinline__ int group_head(int i) const { return DKV ? i / nb : 0; }
};

// Tiles U and W have rings of their own: dq's W is free as soon as T is formed.
template <int D, bool DKV>
struct Smem {
  static constexpr int BC = kCols<DKV>, ROWS = BR * D * 2, COLS = BC * D * 2;
  static constexpr int NU = DKV ? 4 : D == 128 ? 3 : 4, NW = DKV ? 4 : D == 128 ? 2 : 3;
  static constexpr int X = 0, Y = ROWS, U = 2 * ROWS, W = U + NU * COLS, VEC = W + NW * COLS;
  static constexpr int BARS = VEC + (DKV ? NU * 2 * BC * 4 : 2 * BR * 4);
  static constexpr int BYTES = BARS + 1024 + 1024;
};

// Place in a ring of N tiles.
template <int N>
struct Ring {
  uint32_t at = 0, round = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) at = 0, ++round;
  }
};

// TMEM columns: S and T, two places of dS (and P) as bf16, the accumulators.
template <int D, bool DKV>
struct Tmem {
  static constexpr int BC = kCols<DKV>, PD = 2 * BC, PD_STEP = (DKV ? 2 : 1) * BC / 2, ACC = PD + 2 * PD_STEP;
  static_assert(ACC + (DKV ? 2 : 1) * D <= 512, "TMEM has 512 columns");
};

struct Bars {
  uint64_t item_full[2], item_empty[2], x_full, x_empty, u_full[4], u_empty[4], w_full[4], w_empty[4], s_full[2], s_free,
      p_full[2], p_free[2], acc_full, acc_empty, vec_full, vec_free, aux[2], drain[2];
  uint32_t tmem;
  Item item[2];
};
static_assert(sizeof(Bars) <= 1024, "fits its place");

// Item number w.  dq: a sequence's last blocks see the most keys and come first.  dk, dv: with
// first keys that stay visible, a sequence's first block meets every query: these come first.
template <bool DKV>
__device__ __forceinline__ bool find_item(const WindowAttn& a, int64_t w, int64_t blocks, Item& it) {
  const int heads = DKV ? a.hkv : a.hq;
  it.h = (int)(w % heads);
  int64_t b = w / heads;
  if (!DKV) {
    it.q = find_seq(a, blocks - 1 - b, BR, false, it.row0);
    return it.q.ok;
  }
  const bool first = b < a.N;
  if (first) {  // block 0 of sequence b
    const int s = (int)b;
    b = a.cu_k[s] / BR + s;
  } else {
    b -= a.N;
  }
  it.q = find_seq(a, b, BR, true, it.row0);
  return it.q.ok && (it.row0 == 0) == first;
}

__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// FAULT: the test hook's form, which gives up at once.
template <int D, bool DKV, bool FAULT>
__global__ void __launch_bounds__(kThreads, 1)
    k_window_bwd_tc(const WindowAttn a, const int64_t blocks, const int64_t work, int* next_item, float* vec,
                    const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                    const __grid_constant__ CUtensorMap mu, const __grid_constant__ CUtensorMap mw) {
  using L = Smem<D, DKV>;
  constexpr int BC = L::BC, HB = 64;  // HB: columns of a group: half of dq's block, every second block of dk, dv
  constexpr int WARPS = DKV ? 4 : 8;  // row warps at a block
  using M = Tmem<D, DKV>;
  extern __shared__ unsigned char raw[];
  unsigned char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Bars& B = *reinterpret_cast<Bars*>(sm + L::BARS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!DKV && blockIdx.x == 0) check_tables(a);
  if (warp == kScoreWarp) tmem_alloc(&B.tmem, 512);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.item_full[i], 1);
      mbar_init(&B.item_empty[i], 11);  // all warps but the one that hands them out
      mbar_init(&B.aux[i], 1);
      mbar_init(&B.drain[i], 1);
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_full[i], WARPS);
      mbar_init(&B.p_free[i], 1);
    }
    for (int i = 0; i < L::NU; ++i) {
      mbar_init(&B.u_full[i], DKV ? 33 : 1);  // the tile; the loader's lanes' vectors
      mbar_init(&B.u_empty[i], DKV ? 5 : 1);  // MMA; the row warps, which read the vectors
    }
    for (int i = 0; i < L::NW; ++i) {
      mbar_init(&B.w_full[i], 1);
      mbar_init(&B.w_empty[i], 1);
    }
    mbar_init(&B.s_free, WARPS);
    mbar_init(&B.x_full, 1);
    mbar_init(&B.x_empty, 1);
    mbar_init(&B.vec_full, 4);
    mbar_init(&B.vec_free, 4);
    mbar_init(&B.acc_full, 1);
    mbar_init(&B.acc_empty, 8);
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t tm = B.tmem;
  bool ok = true;

  if constexpr (FAULT) {
    if (!DKV) asm volatile("griddepcontrol.wait;" ::: "memory");
    ok = wait_for_nothing(&mx, sm + L::X, BR * 128, &B.x_full, &B.drain[0],
                          warp == kLoadWarp && (DKV ? a.Tk : a.Tq) > 0);
  } else if (warp >= 8) {
    regs_less<kOtherRegs>();
    if (warp == kLoadWarp || warp == kLoadWarp2) {
      // --------------------------------------------------------------- loaders ----
      // One hands out the items and loads the row tiles, the tiles U and the vectors, the other the tiles W.
      const bool first = warp == kLoadWarp;
      const uint32_t N = first ? L::NU : L::NW;
      uint64_t *const full = first ? B.u_full : B.w_full, *const empty = first ? B.u_empty : B.w_empty;
      uint64_t* const aux = &B.aux[first ? 0 : 1];
      const CUtensorMap* const map = first ? &mu : &mw;
      unsigned char* const tiles = sm + (first ? L::U : L::W);
      uint32_t n = 0, tails = 0, xn = 0, at = 0, round = 0;
      int64_t w = blockIdx.x;
      while (ok) {
        Item it;
        const uint32_t slot = n & 1;
        if (first) {
          it.ok = w < work;
          if (it.ok) {
            const bool have = find_item<DKV>(a, w, blocks, it);
            int nx = 0;
            if (lane == 0) nx = atomicAdd(next_item, 1);
            w = (int64_t)gridDim.x + __shfl_sync(0xffffffffu, nx, 0);
            if (!have) continue;
          }
          ok = mbar_wait(&B.item_empty[slot], ((n >> 1) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            B.item[slot] = it;
            mbar_arrive(&B.item_full[slot]);
          }
        } else {
          ok = mbar_wait(&B.item_full[slot], (n >> 1) & 1);
          if (!ok) break;
          it = B.item[slot];
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.item_empty[slot]);
        }
        ++n;
        if (!it.ok) break;
        const Cols<DKV> c(a, it);
        if (!c.cnt) continue;
        if (first) {
          ok = mbar_wait(&B.x_empty, (xn & 1) ^ 1);
          if (!ok) break;
          ++xn;
          if (lane == 0) {
            mbar_expect_tx(&B.x_full, 2 * L::ROWS);
            const int row = (DKV ? it.q.k0 : it.q.q0) + it.row0;
            for (int e = 0; e < D / 64; ++e) {
              tma_load_3d(sm + L::X + e * BR * 128, &mx, 64 * e, it.h, row, &B.x_full);
              tma_load_3d(sm + L::Y + e * BR * 128, &my, 64 * e, it.h, row, &B.x_full);
            }
          }
        }
        const int group = a.hq / a.hkv, len = DKV ? it.q.Lq : it.q.Lk;
        int blk = 0, gh = 0;  // dk, dv: block of the head, head of the group
        for (int i = 0; i < c.cnt; ++i) {
          const int c0 = DKV ? (c.from + blk) * BC : c.col0(i), head = DKV ? it.h * group + gh : it.h / group;
          if (DKV && ++blk == c.nb) blk = 0, ++gh;
          const int left = len - c0;  // rows of this sequence in the tile
          ok = mbar_wait(&empty[at], (round & 1) ^ 1);
          if (!ok) break;
          unsigned char* dst = tiles + at * L::COLS;
          uint64_t* bar = left < BC ? aux : &full[at];
          if (lane == 0) {
            mbar_expect_tx(bar, L::COLS);
            const int row = (DKV ? it.q.q0 : it.q.k0) + c0;
            for (int e = 0; e < D / 64; ++e) tma_load_3d(dst + e * BC * 128, map, 64 * e, head, row, bar);
          }
          if (DKV && first) {
            float* v = reinterpret_cast<float*>(sm + L::VEC) + at * 2 * BC;
            const float* src = vec + (int64_t)head * a.Tq + it.q.q0 + c0;
            for (int e = lane; e < BC; e += 32)
              if (e < left) {
                cp_async4(v + e, src + e);
                cp_async4(v + BC + e, src + (int64_t)a.hq * a.Tq + e);
              }
            cp_async_arrive(&full[at]);
          }
          if (left < BC) {  // the rows past the sequence's end are another's: zeros instead
            ok = mbar_wait(aux, tails & 1);
            ++tails;
            if (!ok) break;
            const int per = (BC - left) * 8;
            for (int e = lane; e < per * (D / 64); e += 32)
              *reinterpret_cast<uint4*>(dst + (e / per) * BC * 128 + left * 128 + (e % per) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[at]);
          }
          if (++at == N) at = 0, ++round;
        }
      }
      cp_async_wait_all();
    } else if (warp == kScoreWarp || warp == kAccWarp) {
      // ------------------------------------------------------------------- MMA ----
      // One warp issues S and T, another the accumulating products: an issuing thread stands still
      // while its products run, and each wait costs it a few hundred cycles.  The warps stay
      // converged, and each group of MMAs is issued by its elected lane: the compiler then knows that
      // there is one, and keeps descriptors in uniform registers.
      const bool scores = warp == kScoreWarp;
      const uint32_t iS = idesc_bf16(BR, BC), iA = idesc_bf16(BR, D) | IDESC_B_MN;
      const uint64_t dX = desc_k_sw128(smem_u32(sm + L::X)), dY = desc_k_sw128(smem_u32(sm + L::Y));
      const uint64_t dU = desc_k_sw128(smem_u32(sm + L::U)), dUt = desc_mn_sw128(smem_u32(sm + L::U), BC * 128);
      constexpr int STEP = L::COLS / 16, UW = (L::W - L::U) / 16;  // of a descriptor: to the next tile, to W
      uint32_t n = 0, xn = 0, an = 0;
      Ring<L::NU> ru;
      Ring<L::NW> rw;
      uint32_t gb = 0;  // blocks so far
      while (ok) {
        const uint32_t slot = n & 1;
        ok = warp_wait(&B.item_full[slot], (n >> 1) & 1);
        if (!ok) break;
        Item it = B.item[slot];
        __syncwarp();
        if (elect_one()) mbar_arrive(&B.item_empty[slot]);
        ++n;
        if (!uniform(it.ok)) break;
        const int cnt = uniform(Cols<DKV>(a, it).cnt);
        if (!cnt) continue;
        if (scores) {
          ok = warp_wait(&B.x_full, xn & 1);
          ++xn;
        }
        for (int i = 0; i < cnt && ok; ++i) {
          if (scores) {
            ok = warp_wait(&B.u_full[ru.at], ru.round & 1);
            ok = ok && warp_wait(&B.w_full[rw.at], rw.round & 1);
            ok = ok && warp_wait(&B.s_free, (gb & 1) ^ 1);  // the last S, T are in registers
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
              mma_rows<D, BR, BC>(tm, dX, dU + ru.at * STEP, iS);
              mma_rows<D, BR, BC>(tm + BC, dY, dU + UW + rw.at * STEP, iS);
              mma_commit(&B.s_full[gb & 1]);
              if (!DKV) mma_commit(&B.w_empty[rw.at]);
              if (i + 1 == cnt) mma_commit(&B.x_empty);
            }
          } else {
            const uint32_t b = gb & 1, pd = tm + M::PD + M::PD_STEP * b;
            ok = warp_wait(&B.u_full[ru.at], ru.round & 1);
            if (DKV) ok = ok && warp_wait(&B.w_full[rw.at], rw.round & 1);
            ok = ok && warp_wait(&B.p_full[b], (gb >> 1) & 1);
            if (i == 0) {  // the last item's results have left TMEM
              ok = ok && warp_wait(&B.acc_empty, (an & 1) ^ 1);
              ++an;
            }
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
              mma_ts_cols<BC>(tm + M::ACC, pd, dUt + ru.at * STEP, iA, i > 0);
              if (DKV) mma_ts_cols<BC>(tm + M::ACC + D, pd + BC / 2, dUt + UW + rw.at * STEP, iA, i > 0);
              mma_commit(&B.p_free[b]);
              mma_commit(&B.u_empty[ru.at]);
              if (DKV) mma_commit(&B.w_empty[rw.at]);
              if (i + 1 == cnt) mma_commit(&B.acc_full);
            }
          }
          ++gb;
          ru.next();
          rw.next();
        }
      }
    }
  } else {
    // -------------------------------------------------------------------- rows ----
    regs_more<kRowRegs>();
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem_lane_addr(tm + (DKV ? 0 : HB * wg), warp, 0);
    const uint32_t tP = tmem_lane_addr(tm + M::PD + (DKV ? 0 : HB / 2 * wg), warp, 0);
    const float sc = __fmul_rn(a.scale, kLog2e);
    const float2 sc2 = make_float2(sc, sc);
    uint32_t n = 0, an = 0, gb = 0;  // gb: blocks so far
    if (!DKV && wg) asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows' delta that group 1 reads
    Ring<L::NU> ru;
    while (ok) {
      const uint32_t slot = n & 1;
      ok = mbar_wait(&B.item_full[slot], (n >> 1) & 1);
      if (!ok) break;
      const Item it = B.item[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.item_empty[slot]);
      ++n;
      if (!it.ok) break;
      const Cols<DKV> c(a, it);
      const bool live = row < c.rows;
      const int at = it.row0 + row + (DKV ? 0 : c.off);  // key, or the query's position
      float2 nl2, nd2;                                   // dq: -lse log2 e and -delta of the row
      if (!DKV) {
        // Group 1 forms delta = do . o of its rows, or takes it from k_window_delta, and hands it and lse to group 0.
        float dl = 0.f, ls = INFINITY;
        float* sh = reinterpret_cast<float*>(sm + L::VEC);
        if (wg) {
          if (live) {
            const int64_t r = (int64_t)(it.q.q0 + it.row0 + row) * a.hq + it.h;
            float* v = vec + (int64_t)it.h * a.Tq + it.q.q0 + it.row0 + row;
            const float l = a.lse[r];
            if (few_keys(at, a.few)) {
              dl = v[(int64_t)a.hq * a.Tq];
            } else {
              const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(a.out) + r * D;
              const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(a.dout) + r * D;
              float x0 = 0.f, x1 = 0.f;
#pragma unroll 8
              for (int e = 0; e < D; e += 8) {
                float x[8], y[8];
                load8(o + e, x);
                load8(g + e, y);
#pragma unroll
                for (int k = 0; k < 8; k += 2) x0 = __fmaf_rn(x[k], y[k], x0), x1 = __fmaf_rn(x[k + 1], y[k + 1], x1);
              }
              dl = __fadd_rn(x0, x1);
              v[(int64_t)a.hq * a.Tq] = dl;
            }
            if (l != -INFINITY) ls = __fmul_rn(l, kLog2e);  // a row that sees nothing: P = exp2(-inf) = 0
            v[0] = ls;
          }
          ok = mbar_wait(&B.vec_free, (n & 1));  // group 0 has the last item's (n counts from 1 here)
          if (!ok) break;
          sh[row] = ls;
          sh[BR + row] = dl;
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.vec_full);
        }
        if (!wg) {
          ok = mbar_wait(&B.vec_full, (n & 1) ^ 1);
          if (!ok) break;
          ls = sh[row];
          dl = sh[BR + row];
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.vec_free);
        }
        nl2 = make_float2(-ls, -ls);
        nd2 = make_float2(-dl, -dl);
      }
      for (int i = 0; i < c.cnt; ++i, ++gb, ru.next()) {
        if (DKV && (gb & 1) != wg) continue;
        const int c0 = c.col0(i), cg = c0 + (DKV ? 0 : HB * wg);  // the block's first column, and the group's
        if (DKV) {
          ok = mbar_wait(&B.u_full[ru.at], ru.round & 1);  // the vectors
          if (!ok) break;
        }
        ok = mbar_wait(&B.s_full[gb & 1], (gb >> 1) & 1);
        if (!ok) break;
        fence_after_sync();
        // which entries are visible, where not all are
        bool cut;
        uint32_t see[HB / 32];
        if (DKV) {
          const int p0 = c0 + c.off, pg = cg + c.off;  // positions of those columns
          cut = it.row0 + BR - 1 > p0 || c0 + BC > it.q.Lq ||
                (a.window > 0 && p0 + BC - 1 - it.row0 >= a.window && it.row0 + BR > a.sinks);
          const int end = (a.window > 0 && at >= a.sinks) ? min(it.q.Lq - cg, at + a.window - pg) : it.q.Lq - cg;
#pragma unroll
          for (int g = 0; g < HB / 32; ++g) see[g] = ~below(at - pg - 32 * g) & below(end - 32 * g);
        } else {
          const int p0 = it.row0 + c.off;
          cut = c0 + BC - 1 > p0 || (a.window > 0 && p0 + BR - 1 - c0 >= a.window && c0 + BC > a.sinks);
          const int lo = a.window > 0 ? at - a.window + 1 : 0;
#pragma unroll
          for (int g = 0; g < HB / 32; ++g)
            see[g] = below(at + 1 - cg - 32 * g) & (~below(lo - cg - 32 * g) | below(a.sinks - cg - 32 * g));
        }
        float s[HB], t[HB];
        tmem_ld64(tS, s);
        tmem_ld64(tS + BC, t);
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.s_free);  // S, T are in registers
        const uint32_t b = gb & 1, tD = tP + M::PD_STEP * b;
        ok = mbar_wait(&B.p_free[b], ((gb >> 1) & 1) ^ 1);  // what was there two blocks ago has been read
        if (!ok) break;
        const float4* lv = reinterpret_cast<const float4*>(sm + L::VEC) + ru.at * (2 * BC / 4);
        const float4* dv = lv + BC / 4;
#pragma unroll
        for (int g = 0; g < HB / 32; ++g) {
          uint32_t pp[16], pd[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float4 l4, d4;
            if (DKV) l4 = lv[8 * g + k], d4 = dv[8 * g + k];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int e = 32 * g + 4 * k + 2 * z;
              const float2 nl = DKV ? (z ? make_float2(-l4.z, -l4.w) : make_float2(-l4.x, -l4.y)) : nl2;
              const float2 nd = DKV ? (z ? make_float2(-d4.z, -d4.w) : make_float2(-d4.x, -d4.y)) : nd2;
              float2 p = fma2(make_float2(s[e], s[e + 1]), sc2, nl);
              p.x = exp2_approx(p.x);
              p.y = exp2_approx(p.y);
              float2 d = mul2(p, add2(make_float2(t[e], t[e + 1]), nd));
              pp[2 * k + z] = pack_bf16(p.x, p.y);
              pd[2 * k + z] = pack_bf16(d.x, d.y);
            }
          }
          if (cut) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const uint32_t keep = ((see[g] >> (2 * k)) & 1 ? 0xffffu : 0u) | ((see[g] >> (2 * k + 1)) & 1 ? 0xffff0000u : 0u);
              pd[k] &= keep;
              if (DKV) pp[k] &= keep;
            }
          }
          tmem_st16u(tD + 16 * g, pd);
          if (DKV) tmem_st16u(tD + BC / 2 + 16 * g, pp);
        }
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&B.p_full[b]);
          if (DKV) mbar_arrive(&B.u_empty[ru.at]);
        }
      }
      if (!ok) break;
      // results: dq's columns are shared between the groups; dk goes to group 0, dv to group 1
      if (c.cnt) {
        ok = mbar_wait(&B.acc_full, an & 1);
        ++an;
        if (!ok) break;
        fence_after_sync();
      }
      constexpr int W = DKV ? D : D / 2;  // columns of this group
      const int heads = DKV ? a.hkv : a.hq, col = DKV ? 0 : wg * W;
      const float f = DKV && wg == 1 ? 1.f : a.scale;
      const uint32_t tA = tmem_lane_addr(tm + M::ACC, warp, DKV ? D * wg : W * wg);
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(DKV ? (wg ? a.dv : a.dk) : a.dq) +
                           ((int64_t)((DKV ? it.q.k0 : it.q.q0) + it.row0 + row) * heads + it.h) * D + col;
#pragma unroll
      for (int e = 0; e < W; e += 32) {
        float x[32];
        if (c.cnt) {
          tmem_ld32(tA + e, x);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = 0.f;
        }
        if (live) {
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            *reinterpret_cast<uint4*>(dst + e + k) =
                make_uint4(pack_bf16(__fmul_rn(x[k], f), __fmul_rn(x[k + 1], f)),
                           pack_bf16(__fmul_rn(x[k + 2], f), __fmul_rn(x[k + 3], f)),
                           pack_bf16(__fmul_rn(x[k + 4], f), __fmul_rn(x[k + 5], f)),
                           pack_bf16(__fmul_rn(x[k + 6], f), __fmul_rn(x[k + 7], f)));
        }
      }
      if (c.cnt) {
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.acc_empty);
      }
    }
  }
  if (!ok) set_error(a.hdr, GDN_DEVERR_TIMEOUT);
  if (__syncthreads_or(!ok)) {
    // something gave up: copies and MMAs that were issued end before the memory is given back
    if (warp == kLoadWarp && lane == 0) {
      for (int i = 0; i < L::NU; ++i) settle(&B.u_full[i]);
      settle(&B.x_full);
      settle(&B.aux[0]);
    }
    if (warp == kLoadWarp2 && lane == 0) {
      for (int i = 0; i < L::NW; ++i) settle(&B.w_full[i]);
      settle(&B.aux[1]);
    }
    if (warp == kScoreWarp || warp == kAccWarp) settle_mma(&B.drain[warp == kAccWarp]);
  }
  __syncthreads();
  if (warp == kScoreWarp) tmem_dealloc(tm, 512);
}

template <int D, bool DKV, bool FAULT>
bool bwd_tc(const WindowAttn& a, cudaStream_t st) {
  CUtensorMap mx, my, mu, mw;
  constexpr int BC = kCols<DKV>;
  const bool ok = DKV ? make_rows_map(&mx, a.k, a.Tk, a.hkv, D, BR, a.hdr) &&
                            make_rows_map(&my, a.v, a.Tk, a.hkv, D, BR, a.hdr) &&
                            make_rows_map(&mu, a.q, a.Tq, a.hq, D, BC, a.hdr) &&
                            make_rows_map(&mw, a.dout, a.Tq, a.hq, D, BC, a.hdr)
                      : make_rows_map(&mx, a.q, a.Tq, a.hq, D, BR, a.hdr) &&
                            make_rows_map(&my, a.dout, a.Tq, a.hq, D, BR, a.hdr) &&
                            make_rows_map(&mu, a.k, a.Tk, a.hkv, D, BC, a.hdr) &&
                            make_rows_map(&mw, a.v, a.Tk, a.hkv, D, BC, a.hdr);
  if (!ok) return false;
  // dk, dv: N more items, the sequences' first blocks ahead of the others
  const int64_t blocks = item_count(DKV ? a.Tk : a.Tq, BR, a.N);
  const int64_t work = DKV ? (blocks + a.N) * a.hkv : blocks * a.hq;
  static std::atomic<uint64_t> ready{0};
  ensure_smem(k_window_bwd_tc<D, DKV, FAULT>, (Smem<D, DKV>::BYTES), ready);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(work < kSms ? work : kSms));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = Smem<D, DKV>::BYTES;
  c.stream = st;
  c.attrs = &attr;
  c.numAttrs = DKV ? 0 : 1;  // dq starts beside k_window_delta, for whose results its group 1 waits
  cudaLaunchKernelEx(&c, k_window_bwd_tc<D, DKV, FAULT>, a, blocks, work, a.hdr->pad + (DKV ? 1 : 0), a.delta, mx, my, mu,
                     mw);
  return true;
}

template <bool DKV>
bool by_size(const WindowAttn& a, cudaStream_t st) {
  if (a.fault_wait) return a.d == 128 ? bwd_tc<128, DKV, true>(a, st) : bwd_tc<64, DKV, true>(a, st);
  return a.d == 128 ? bwd_tc<128, DKV, false>(a, st) : bwd_tc<64, DKV, false>(a, st);
}

}  // namespace

bool launch_window_dq_tc(const WindowAttn& a, cudaStream_t st) {
  // the error word and the two item counters
  if (cudaMemsetAsync(a.hdr, 0, sizeof(WsHeader), st) != cudaSuccess) return false;
  launch_window_delta(a, st);
  return by_size<false>(a, st);
}
bool launch_window_dkv_tc(const WindowAttn& a, cudaStream_t st) {
  return by_size<true>(a, st);
}

}  // namespace gdn
