// attn_window_bwd_tc.cu -- gradient of sliding-window attention for bf16 with d = 64 or 128 on the
// tensor cores.  Two kernels of one form, so that nothing is added across CTAs and the result
// does not depend on their order:
//   dq      rows = 128 queries of a head, columns = blocks of 64 keys:   dQ += dS K
//   dk, dv  rows = 128 keys of a key head, columns = blocks of 64 queries of each head of the group in
//           ascending order:   dK += dS^T Q,  dV += P^T dO
// with P = exp2(c Q K^T - lse log2 e) and dS = P (dO V^T - delta) formed anew in both (7 products of
// 128 x 64 x d where one kernel that adds dQ across CTAs would need 5).  The row tiles X, Y (Q and
// dO, or K and V) stay on chip: Q and dO in TMEM, as the first operand of their products, K and V,
// for which TMEM has no room, in shared memory; column tiles U, W come by TMA.  S = X U^T and T = Y W^T go
// to TMEM; a group of four warps (a thread per row) takes them into registers, which frees their
// place for the next block's, and leaves dS and P as bf16 in a place of its own, from which the
// accumulating products read them.  The two groups take the column blocks in turn, so that one's
// arithmetic runs beside the other's and the products.
// P and dS are rounded to bf16 for their products; everything else stays in 32 bits.
// A 128 x 64 block costs 128 x 64 x d MACs per product at 4096 a clock; an operand from shared memory
// is read at 128 bytes a clock, so that with both operands there S and T (48 KB each at d = 128) take
// half as long again, and with the rows in TMEM they do not.
#include "attn_tc.cuh"
#include "attn_window.cuh"

namespace gdn {

namespace {

using namespace win;
using namespace tc;

constexpr int BR = 128, BC = 64;  // rows, columns of a block
constexpr int kThreads = 384, kScoreWarp = 8, kLoadWarp = 9, kAccWarp = 10;
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

template <int D, bool DKV>
struct Smem {
  static constexpr int ROWS = DKV ? BR * D * 2 : 0, COLS = BC * D * 2, STAGES = DKV ? 4 : 6;
  static constexpr int X = 0, Y = ROWS, ST = 2 * ROWS, VEC = ST + STAGES * 2 * COLS;
  static constexpr int BARS = VEC + (DKV ? STAGES * 2 * BC * 4 : 2 * BR * 4);
  static constexpr int BYTES = BARS + 1024 + 1024;
};

// TMEM columns: buffers of S and T (128 columns), dS and P of each group as bf16 (32 columns each),
// the accumulators, and for dq the rows X, Y (see above).
template <int D, bool DKV>
struct Tmem {
  static constexpr int ST_BUFS = D == 128 ? 1 : 2, PD_STEP = DKV ? 64 : 32;
  static constexpr int PD = 128 * ST_BUFS, ACC = PD + 2 * PD_STEP, X = ACC + (DKV ? 2 : 1) * D, Y = X + D / 2;
  static_assert(X + (DKV ? 0 : D) <= 512, "TMEM has 512 columns");
};

struct Bars {
  uint64_t item_full[2], item_empty[2], x_full, x_empty, st_full[6], st_empty[6], s_full[2], s_free[2],
      p_full[2], p_free[2], acc_full, acc_empty, vec_full, vec_free, aux;
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

template <int D, bool DKV>
__global__ void __launch_bounds__(kThreads, 1)
    k_window_bwd_tc(const WindowAttn a, const int64_t blocks, const int64_t work, int* next_item, float* vec,
                    const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                    const __grid_constant__ CUtensorMap mu, const __grid_constant__ CUtensorMap mw) {
  using L = Smem<D, DKV>;
  constexpr int STAGES = L::STAGES;
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
      mbar_init(&B.item_empty[i], 10);  // all warps but the loader and the idle one
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.s_free[i], 4);
      mbar_init(&B.p_full[i], 4);
      mbar_init(&B.p_free[i], 1);
    }
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&B.st_full[i], DKV ? 33 : 1);  // tiles; the loader's lanes' vectors
      mbar_init(&B.st_empty[i], DKV ? 5 : 1);  // MMA; the four warps that read the vectors
    }
    mbar_init(&B.x_full, DKV ? 1 : 8);  // TMA, or the row warps
    mbar_init(&B.x_empty, 1);
    mbar_init(&B.vec_full, 4);
    mbar_init(&B.vec_free, 4);
    mbar_init(&B.acc_full, 1);
    mbar_init(&B.acc_empty, 8);
    mbar_init(&B.aux, 1);
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t tm = B.tmem;
  bool ok = true;

  if (warp >= 8) {
    regs_less<kOtherRegs>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- loader ----
      uint32_t n = 0, stage = 0, round = 0, aux = 0, xn = 0;
      int64_t w = blockIdx.x;
      while (ok) {
        Item it;
        it.ok = w < work;
        if (it.ok) {
          const bool have = find_item<DKV>(a, w, blocks, it);
          int nx = 0;
          if (lane == 0) nx = atomicAdd(next_item, 1);
          w = (int64_t)gridDim.x + __shfl_sync(0xffffffffu, nx, 0);
          if (!have) continue;
        }
        const uint32_t slot = n & 1;
        ok = mbar_wait(&B.item_empty[slot], ((n >> 1) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          B.item[slot] = it;
          mbar_arrive(&B.item_full[slot]);
        }
        ++n;
        if (!it.ok) break;
        const Cols<DKV> c(a, it);
        if (!c.cnt) continue;
        if (DKV) {
          ok = mbar_wait(&B.x_empty, (xn & 1) ^ 1);
          if (!ok) break;
          ++xn;
          if (lane == 0) {
            mbar_expect_tx(&B.x_full, 2 * L::ROWS);
            const int row = it.q.k0 + it.row0;
            for (int e = 0; e < D / 64; ++e) {
              tma_load_3d(sm + L::X + e * BR * 128, &mx, 64 * e, it.h, row, &B.x_full);
              tma_load_3d(sm + L::Y + e * BR * 128, &my, 64 * e, it.h, row, &B.x_full);
            }
          }
        }
        const int group = a.hq / a.hkv, len = DKV ? it.q.Lq : it.q.Lk;
        for (int i = 0; i < c.cnt; ++i) {
          ok = mbar_wait(&B.st_empty[stage], (round & 1) ^ 1);
          if (!ok) break;
          const int c0 = c.col0(i), head = DKV ? it.h * group + c.group_head(i) : it.h / group;
          const int left = len - c0;  // rows of this sequence in the tiles
          unsigned char* dst = sm + L::ST + stage * 2 * L::COLS;
          uint64_t* bar = left < BC ? &B.aux : &B.st_full[stage];
          if (lane == 0) {
            mbar_expect_tx(bar, 2 * L::COLS);
            const int row = (DKV ? it.q.q0 : it.q.k0) + c0;
            for (int e = 0; e < D / 64; ++e) {
              tma_load_3d(dst + e * BC * 128, &mu, 64 * e, head, row, bar);
              tma_load_3d(dst + L::COLS + e * BC * 128, &mw, 64 * e, head, row, bar);
            }
          }
          if (DKV) {
            float* v = reinterpret_cast<float*>(sm + L::VEC) + stage * 2 * BC;
            const float* src = vec + (int64_t)head * a.Tq + it.q.q0 + c0;
            for (int e = lane; e < BC; e += 32)
              if (e < left) {
                cp_async4(v + e, src + e);
                cp_async4(v + BC + e, src + (int64_t)a.hq * a.Tq + e);
              }
            cp_async_arrive(&B.st_full[stage]);
          }
          if (left < BC) {  // the rows past the sequence's end are another's: zeros instead
            ok = mbar_wait(&B.aux, aux & 1);
            ++aux;
            if (!ok) break;
            const int per = (BC - left) * 8;
            for (int e = lane; e < per * 2 * (D / 64); e += 32)
              *reinterpret_cast<uint4*>(dst + (e / per) * BC * 128 + left * 128 + (e % per) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.st_full[stage]);
          }
          if (++stage == STAGES) stage = 0, ++round;
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
      const uint64_t dU = desc_k_sw128(smem_u32(sm + L::ST)), dUt = desc_mn_sw128(smem_u32(sm + L::ST), BC * 128);
      constexpr int STEP = L::COLS / 16;  // of a descriptor, from U to W of a stage
      uint32_t n = 0, xn = 0, an = 0, stage = 0, round = 0;
      uint32_t buf = 0, bn = 0, np[2] = {0, 0};  // S, T buffer and its use; P, dS
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
          ok = warp_wait(&B.st_full[stage], round & 1);
          if (scores) {
            ok = ok && warp_wait(&B.s_free[buf], (bn & 1) ^ 1);  // the buffer's last S, T are in registers
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
              const uint64_t u = dU + stage * (2 * STEP);
              if (DKV) {
                mma_rows<D, BR, BC>(tm + 128 * buf, dX, u, iS);
                mma_rows<D, BR, BC>(tm + 128 * buf + 64, dY, u + STEP, iS);
              } else {
                mma_ts_rows<D, BC>(tm + 128 * buf, tm + M::X, u, iS);
                mma_ts_rows<D, BC>(tm + 128 * buf + 64, tm + M::Y, u + STEP, iS);
              }
              mma_commit(&B.s_full[i & 1]);
              if (i + 1 == cnt) mma_commit(&B.x_empty);
            }
            if (++buf == M::ST_BUFS) buf = 0, ++bn;
          } else {
            const int b = i & 1;
            ok = ok && warp_wait(&B.p_full[b], np[b] & 1);
            ++np[b];
            if (i == 0) {  // the last item's results have left TMEM
              ok = ok && warp_wait(&B.acc_empty, (an & 1) ^ 1);
              ++an;
            }
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
              const uint64_t u = dUt + stage * (2 * STEP);
              mma_ts_cols<BC>(tm + M::ACC, tm + M::PD + M::PD_STEP * b, u, iA, i > 0);
              if (DKV) mma_ts_cols<BC>(tm + M::ACC + D, tm + M::PD + M::PD_STEP * b + 32, u + STEP, iA, i > 0);
              mma_commit(&B.p_free[b]);
              mma_commit(&B.st_empty[stage]);
              if (i + 1 == cnt) mma_commit(&B.acc_full);
            }
          }
          if (++stage == STAGES) stage = 0, ++round;
        }
      }
    }
  } else {
    // -------------------------------------------------------------------- rows ----
    regs_more<kRowRegs>();
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tP = tmem_lane_addr(tm + M::PD + M::PD_STEP * wg, warp, 0);
    const float sc = __fmul_rn(a.scale, kLog2e);
    const float2 sc2 = make_float2(sc, sc);
    uint32_t n = 0, ns = 0, an = 0, xn = 0;
    uint32_t stage = 0, round = 0, blk = 0;  // stage of the item's block 0, and the S, T buffer's block count
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
        // Group 0 brings Q's rows to TMEM, group 1 dO's, with which it forms delta = do . o.
        const int64_t r = (int64_t)(it.q.q0 + it.row0 + row) * a.hq + it.h;
        const uint4* xp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(wg ? a.dout : a.q) + r * D);
        uint4 x[D / 8];
#pragma unroll
        for (int e = 0; e < D / 8; ++e) x[e] = live ? xp[e] : make_uint4(0, 0, 0, 0);
        float dl = 0.f, ls = INFINITY;
        float* sh = reinterpret_cast<float*>(sm + L::VEC);
        if (wg) {
          if (live) {
            const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(a.out) + r * D;
            float x0 = 0.f, x1 = 0.f;
#pragma unroll
            for (int e = 0; e < D / 8; ++e) {
              float y[8];
              load8(o + 8 * e, y);
              const uint32_t g[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                x0 = __fmaf_rn(__uint_as_float(g[k] << 16), y[2 * k], x0);
                x1 = __fmaf_rn(__uint_as_float(g[k] & 0xffff0000u), y[2 * k + 1], x1);
              }
            }
            dl = __fadd_rn(x0, x1);
            const float l = a.lse[r];
            if (l != -INFINITY) ls = __fmul_rn(l, kLog2e);  // a row that sees nothing: P = exp2(-inf) = 0
            float* v = vec + (int64_t)it.h * a.Tq + it.q.q0 + it.row0 + row;
            v[0] = ls;
            v[(int64_t)a.hq * a.Tq] = dl;
          }
          ok = mbar_wait(&B.vec_free, (n & 1));  // group 0 has the last item's (n counts from 1 here)
          if (!ok) break;
          sh[row] = ls;
          sh[BR + row] = dl;
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.vec_full);
        }
        if (c.cnt) {
          ok = mbar_wait(&B.x_empty, (xn & 1) ^ 1);  // the last item's scores are done
          ++xn;
          if (!ok) break;
          const uint32_t tX = tmem_lane_addr(tm + (wg ? M::Y : M::X), warp, 0);
#pragma unroll
          for (int e = 0; e < D / 8; e += 4) tmem_st16u(tX + 4 * e, reinterpret_cast<const uint32_t*>(&x[e]));
          tmem_st_wait();
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.x_full);
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
      for (int i = wg; i < c.cnt; i += 2) {
        const int c0 = c.col0(i);
        uint32_t st = stage + i, sr = round + st / STAGES;
        st %= STAGES;
        if (DKV) {
          ok = mbar_wait(&B.st_full[st], sr & 1);  // the vectors
          if (!ok) break;
        }
        ok = mbar_wait(&B.s_full[wg], ns & 1);
        ++ns;
        if (!ok) break;
        fence_after_sync();
        // which entries are visible, where not all are
        bool cut;
        uint32_t see[2];
        if (DKV) {
          const int p0 = c0 + c.off;  // position of column 0
          cut = it.row0 + BR - 1 > p0 || c0 + BC > it.q.Lq ||
                (a.window > 0 && p0 + BC - 1 - it.row0 >= a.window && it.row0 + BR > a.sinks);
          const int end = (a.window > 0 && at >= a.sinks) ? min(it.q.Lq - c0, at + a.window - p0) : it.q.Lq - c0;
#pragma unroll
          for (int g = 0; g < 2; ++g) see[g] = ~below(at - p0 - 32 * g) & below(end - 32 * g);
        } else {
          const int p0 = it.row0 + c.off;
          cut = c0 + BC - 1 > p0 || (a.window > 0 && p0 + BR - 1 - c0 >= a.window && c0 + BC > a.sinks);
          const int lo = a.window > 0 ? at - a.window + 1 : 0;
#pragma unroll
          for (int g = 0; g < 2; ++g)
            see[g] = below(at + 1 - c0 - 32 * g) & (~below(lo - c0 - 32 * g) | below(a.sinks - c0 - 32 * g));
        }
        if (!cut) see[0] = see[1] = ~0u;
        float s[BC], t[BC];
        const uint32_t tS = tmem_lane_addr(tm + 128 * ((blk + i) % M::ST_BUFS), warp, 0);
        tmem_ld64(tS, s);
        tmem_ld64(tS + 64, t);
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.s_free[(blk + i) % M::ST_BUFS]);  // S, T are in registers
        if (ns > 1) {  // the group's last P and dS have been read
          ok = mbar_wait(&B.p_free[wg], ns & 1);
          if (!ok) break;
        }
        const float4* lv = reinterpret_cast<const float4*>(sm + L::VEC) + st * (2 * BC / 4);
        const float4* dv = lv + BC / 4;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
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
          tmem_st16u(tP + 16 * g, pd);
          if (DKV) tmem_st16u(tP + 32 + 16 * g, pp);
        }
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&B.p_full[wg]);
          if (DKV) mbar_arrive(&B.st_empty[st]);
        }
      }
      if (!ok) break;
      blk += c.cnt;
      stage += c.cnt;
      round += stage / STAGES;
      stage %= STAGES;
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
    // something gave up: copies that were issued land before the memory is given back
    if (warp == kLoadWarp && lane == 0)
      for (int i = 0; i < STAGES; ++i) mbar_wait(&B.st_full[i], 0, 1u << 12);
  }
  __syncthreads();
  if (warp == kScoreWarp) tmem_dealloc(tm, 512);
}

template <int D, bool DKV>
bool bwd_tc(const WindowAttn& a, cudaStream_t st) {
  CUtensorMap mx, my, mu, mw;
  const bool ok = DKV ? make_rows_map(&mx, a.k, a.Tk, a.hkv, D, BR, a.hdr) && make_rows_map(&my, a.v, a.Tk, a.hkv, D, BR, a.hdr) &&
                            make_rows_map(&mu, a.q, a.Tq, a.hq, D, BC, a.hdr) && make_rows_map(&mw, a.dout, a.Tq, a.hq, D, BC, a.hdr)
                      : make_rows_map(&mx, a.q, a.Tq, a.hq, D, BR, a.hdr) && make_rows_map(&my, a.dout, a.Tq, a.hq, D, BR, a.hdr) &&
                            make_rows_map(&mu, a.k, a.Tk, a.hkv, D, BC, a.hdr) && make_rows_map(&mw, a.v, a.Tk, a.hkv, D, BC, a.hdr);
  if (!ok) return false;
  // dk, dv: N more items, the sequences' first blocks ahead of the others
  const int64_t blocks = item_count(DKV ? a.Tk : a.Tq, BR, a.N);
  const int64_t work = DKV ? (blocks + a.N) * a.hkv : blocks * a.hq;
  static std::atomic<uint64_t> ready{0};
  ensure_smem(k_window_bwd_tc<D, DKV>, (Smem<D, DKV>::BYTES), ready);
  k_window_bwd_tc<D, DKV><<<(unsigned)(work < kSms ? work : kSms), kThreads, (Smem<D, DKV>::BYTES), st>>>(
      a, blocks, work, a.hdr->pad + (DKV ? 1 : 0), a.delta, mx, my, mu, mw);
  return true;
}

}  // namespace

bool launch_window_dq_tc(const WindowAttn& a, cudaStream_t st) {
  // the error word and the two item counters
  if (cudaMemsetAsync(a.hdr, 0, sizeof(WsHeader), st) != cudaSuccess) return false;
  return a.d == 128 ? bwd_tc<128, false>(a, st) : bwd_tc<64, false>(a, st);
}
bool launch_window_dkv_tc(const WindowAttn& a, cudaStream_t st) {
  return a.d == 128 ? bwd_tc<128, true>(a, st) : bwd_tc<64, true>(a, st);
}

}  // namespace gdn
