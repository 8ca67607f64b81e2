// attn_host.cu -- the C ABI of the attention-layer operators (include/gdn_cpr.h): argument
// checks and workspace sizes; the kernels are in attn_tokens.cu, attn_decode.cu,
// attn_window.cu and attn_window_tc.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn.h"
#include "hooks.h"

namespace {
using namespace gdn;

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool ok_ptr(const void* p, size_t a) { return p != nullptr && aligned(p, a); }
inline bool ok_ws(const void* ws, size_t have, size_t need) { return ws && aligned(ws, kAlign) && have >= need; }
inline bool ok_dtype(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }
inline bool ok_d(int d) { return d == 32 || d == 64 || d == 128; }
inline char* at(void* ws, size_t off) { return static_cast<char*>(ws) + off; }

// log2 of a page size the cache may have, or -1
int page_shift_of(int32_t page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

gdn_status check_norm(const gdn_cpr_norm_rope* c) {
  if (!c) return GDN_ERR_INVALID_ARG;
  if (c->tokens < 0 || c->h_q < 0 || c->h_k < 0 || c->h_q + (int64_t)c->h_k <= 0 || c->rot < 0 || c->table_rows < 0)
    return GDN_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f) || !isfinite(c->eps)) return GDN_ERR_INVALID_ARG;
  if (c->h_q > 65535 || c->h_k > 65535 || !ok_d(c->d)) return GDN_ERR_UNSUPPORTED;
  // blocks are numbered in 31 bits
  if ((int64_t)c->tokens * (c->h_q + 2 * (int64_t)c->h_k) > (int64_t)INT32_MAX) return GDN_ERR_UNSUPPORTED;
  if (c->rot > c->d || c->rot % 8 != 0) return GDN_ERR_UNSUPPORTED;
  if (c->norm != GDN_NORM_NONE && c->norm != GDN_NORM_RMS && c->norm != GDN_NORM_L2) return GDN_ERR_UNSUPPORTED;
  if (c->layout != GDN_ROPE_HALF && c->layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_UNSUPPORTED;
  if (!ok_dtype(c->in_dtype) || !ok_dtype(c->out_dtype) || !ok_dtype(c->grad_dtype)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// a token's rows: the stride holds its heads and keeps every row on a 16-byte boundary
bool ok_stride(int64_t stride, int heads, const gdn_cpr_norm_rope* c) {
  return stride >= (int64_t)heads * c->d && stride % (c->in_dtype == GDN_BF16 ? 8 : 4) == 0;
}

gdn_status check_tables(const gdn_cpr_norm_rope* c, const float* cos, const float* sin, const int32_t* pos) {
  if (c->rot == 0 || c->tokens == 0) return GDN_OK;
  if (c->table_rows < 1) return GDN_ERR_INVALID_ARG;  // a token outside the tables still reads their row 0
  return ok_ptr(cos, 16) && ok_ptr(sin, 16) && ok_ptr(pos, 4) ? GDN_OK : GDN_ERR_INVALID_ARG;
}

NormRope norm_args(const gdn_cpr_norm_rope* c, const void* q, const void* k, const float* wq, const float* wk,
                   const float* cos, const float* sin, const int32_t* pos) {
  NormRope a{};
  a.T = c->tokens;
  a.hq = c->h_q;
  a.hk = c->h_k;
  a.rot = c->rot;
  a.table_rows = c->table_rows;
  a.norm = c->norm;
  a.layout = c->layout;
  a.eps = c->eps;
  a.q_stride = c->q_stride;
  a.k_stride = c->k_stride;
  a.v_stride = c->v_stride;
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.cos = cos;
  a.sin = sin;
  a.pos = pos;
  return a;
}

gdn_status check_attn(const gdn_cpr_attn* a) {
  if (!a) return GDN_ERR_INVALID_ARG;
  if (a->h_q <= 0 || a->h_kv <= 0 || a->window < 0 || a->sinks < 0) return GDN_ERR_INVALID_ARG;
  if (!(a->scale >= 0.f) || !isfinite(a->scale)) return GDN_ERR_INVALID_ARG;
  if (a->h_q % a->h_kv != 0 || a->h_q > 65535 || !ok_d(a->d) || !ok_dtype(a->dtype)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

float scale_of(const gdn_cpr_attn* a) { return a->scale > 0.f ? a->scale : 1.f / sqrtf((float)a->d); }

// Decode workspace: header | runs' accumulators [N, hq, splits, d] | their (m, l)
size_t decode_bytes(const gdn_cpr_attn* a, int32_t N, int splits) {
  const size_t records = splits > 1 ? (size_t)N * a->h_q * splits : 0;
  return align_up(GDN_CPR_ATTN_HEADER_BYTES + records * (a->d + 2) * sizeof(float));
}

int decode_splits(const gdn_cpr_attn* a, int32_t max_len) {
  return paged_decode_max_splits(visible_keys(max_len, a->window, a->sinks), a->h_kv);
}

// An empty call sets its error word too.  It queues nothing else, so it also passes where there is no
// device, and memory that the device does not know is left alone.
gdn_status empty_call(void* ws, cudaStream_t st) {
  cudaPointerAttributes p{};
  if (cudaPointerGetAttributes(&p, ws) != cudaSuccess || p.type == cudaMemoryTypeUnregistered) {
    cudaGetLastError();
    return GDN_OK;
  }
  return cudaMemsetAsync(ws, 0, sizeof(WsHeader), st) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status finish() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// Rows of a packed batch of window_attn: position + window stays inside 32 bits.
constexpr int32_t kMaxRows = 1 << 30;

const char* const kNormStages[] = {"norm and rotation", nullptr};
const char* const kMapStages[] = {"page map", nullptr};
const char* const kPagedStages[] = {"paged decode attention", nullptr};
const char* const kWindowStages[] = {"window attention", nullptr};
const char* const kWindowBwdStages[] = {"window attention dq", "window attention dk, dv", nullptr};

gdn_status window_args(const gdn_cpr_attn* attn, int32_t N, int32_t Tq, int32_t Tk, const int32_t* cu_q,
                       const int32_t* cu_k, const void* q, const void* k, const void* v, WindowAttn* w) {
  gdn_status rc = check_attn(attn);
  if (rc != GDN_OK) return rc;
  if (N < 0 || Tq < 0 || Tk < 0 || (N == 0 && (Tq || Tk))) return GDN_ERR_INVALID_ARG;
  if (Tq > kMaxRows || Tk > kMaxRows) return GDN_ERR_UNSUPPORTED;
  if (N > 0 && (!ok_ptr(cu_q, 4) || !ok_ptr(cu_k, 4))) return GDN_ERR_INVALID_ARG;
  if (Tq > 0 && !ok_ptr(q, 16)) return GDN_ERR_INVALID_ARG;
  if (Tk > 0 && (!ok_ptr(k, 16) || !ok_ptr(v, 16))) return GDN_ERR_INVALID_ARG;
  *w = WindowAttn{};
  w->N = N;
  w->Tq = Tq;
  w->Tk = Tk;
  w->hq = attn->h_q;
  w->hkv = attn->h_kv;
  w->d = attn->d;
  w->window = attn->window < kMaxRows ? attn->window : 0;  // as far as any sequence reaches
  w->sinks = attn->sinks;
  w->scale = scale_of(attn);
  w->cu_q = cu_q;
  w->cu_k = cu_k;
  w->q = q;
  w->k = k;
  w->v = v;
  return GDN_OK;
}

bool window_on_tensor_cores(const gdn_cpr_attn* a) { return a->dtype == GDN_BF16 && a->d != 32; }

size_t window_bytes(const gdn_cpr_attn* a, int32_t Tq, bool backward) {
  return align_up(GDN_CPR_ATTN_HEADER_BYTES + (backward ? 2 * (size_t)Tq * a->h_q * sizeof(float) : 0));
}

}  // namespace

extern "C" {

gdn_status gdn_cpr_qk_norm_rope(const gdn_cpr_norm_rope* cfg, const void* q, const void* k, const void* v,
                                const float* q_weight, const float* k_weight, const float* cos, const float* sin,
                                const int32_t* positions, void* q_out, void* k_out, void* k_pages, void* v_pages,
                                int32_t num_pages, int32_t page_size, const int32_t* slot_map, gdn_stream_t stream) {
  NvtxRange nvtx("gdn_cpr_qk_norm_rope");
  gdn_status rc = check_norm(cfg);
  if (rc != GDN_OK) return rc;
  const int T = cfg->tokens;
  if (cfg->h_q && !ok_stride(cfg->q_stride, cfg->h_q, cfg)) return GDN_ERR_INVALID_ARG;
  if (cfg->h_k && !ok_stride(cfg->k_stride, cfg->h_k, cfg)) return GDN_ERR_INVALID_ARG;
  if (T > 0 && ((cfg->h_q && !ok_ptr(q, 16)) || (cfg->h_k && !ok_ptr(k, 16)))) return GDN_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(q_out, 16) || !aligned(k_out, 16))
    return GDN_ERR_INVALID_ARG;
  rc = check_tables(cfg, cos, sin, positions);
  if (rc != GDN_OK) return rc;
  NormRope a = norm_args(cfg, q, k, q_weight, k_weight, cos, sin, positions);
  if (k_pages || v_pages) {
    const int shift = page_shift_of(page_size);
    if (num_pages < 0 || page_size <= 0) return GDN_ERR_INVALID_ARG;
    if (shift < 0) return GDN_ERR_UNSUPPORTED;
    if (!ok_ptr(k_pages, 16) || !ok_ptr(v_pages, 16) || (T > 0 && (!ok_ptr(v, 16) || !ok_ptr(slot_map, 4))))
      return GDN_ERR_INVALID_ARG;
    if (!ok_stride(cfg->v_stride, cfg->h_k, cfg)) return GDN_ERR_INVALID_ARG;
    a.v = v;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.page_shift = shift;
    a.slots = (int64_t)num_pages << shift;
    a.slot_map = slot_map;
  }
  if (T == 0) return GDN_OK;
  a.q_out = q_out;
  a.k_out = k_out;
  Stages stg(stream, kNormStages);
  launch_norm_rope(a, cfg->d, cfg->in_dtype == GDN_BF16, cfg->out_dtype == GDN_BF16, stream);
  stg.mark(1);
  return finish();
}

gdn_status gdn_cpr_qk_norm_rope_workspace_size(const gdn_cpr_norm_rope* cfg, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  const gdn_status rc = check_norm(cfg);
  if (rc != GDN_OK) return rc;
  // one row of d sums per block: at most kNormBwdBlocks, or one per run of heads (of 8 or more)
  const size_t runs = (size_t)(cfg->h_q + 3) / 4 + (size_t)(cfg->h_k + 3) / 4;
  *bytes = align_up((runs > kNormBwdBlocks ? runs : kNormBwdBlocks) * cfg->d * sizeof(float));
  return GDN_OK;
}

gdn_status gdn_cpr_qk_norm_rope_bwd(const gdn_cpr_norm_rope* cfg, const void* q, const void* k, const float* q_weight,
                                    const float* k_weight, const float* cos, const float* sin,
                                    const int32_t* positions, const void* dq_out, const void* dk_out, void* dq,
                                    void* dk, float* dq_weight, float* dk_weight, void* ws, size_t ws_bytes,
                                    gdn_stream_t stream) {
  NvtxRange nvtx("gdn_cpr_qk_norm_rope_bwd");
  gdn_status rc = check_norm(cfg);
  if (rc != GDN_OK) return rc;
  const int T = cfg->tokens;
  if (cfg->h_q && !ok_stride(cfg->q_stride, cfg->h_q, cfg)) return GDN_ERR_INVALID_ARG;
  if (cfg->h_k && !ok_stride(cfg->k_stride, cfg->h_k, cfg)) return GDN_ERR_INVALID_ARG;
  if (T > 0 && cfg->h_q && (!ok_ptr(q, 16) || !ok_ptr(dq_out, 16) || !ok_ptr(dq, 16))) return GDN_ERR_INVALID_ARG;
  if (T > 0 && cfg->h_k && (!ok_ptr(k, 16) || !ok_ptr(dk_out, 16) || !ok_ptr(dk, 16))) return GDN_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return GDN_ERR_INVALID_ARG;
  if ((dq_weight == nullptr) != (dk_weight == nullptr)) return GDN_ERR_INVALID_ARG;
  if (dq_weight && (!aligned(dq_weight, 4) || !aligned(dk_weight, 4))) return GDN_ERR_INVALID_ARG;
  rc = check_tables(cfg, cos, sin, positions);
  if (rc != GDN_OK) return rc;
  NormRope a = norm_args(cfg, q, k, q_weight, k_weight, cos, sin, positions);
  if (dq_weight) {
    size_t need = 0;
    gdn_cpr_qk_norm_rope_workspace_size(cfg, &need);
    if (!ok_ws(ws, ws_bytes, need)) return GDN_ERR_WORKSPACE;
    a.partial = static_cast<float*>(ws);
    a.dwq = dq_weight;
    a.dwk = dk_weight;
  }
  if (T == 0) {
    if (dq_weight && (cudaMemsetAsync(dq_weight, 0, cfg->d * sizeof(float), stream) != cudaSuccess ||
                      cudaMemsetAsync(dk_weight, 0, cfg->d * sizeof(float), stream) != cudaSuccess))
      return GDN_ERR_CUDA;
    return GDN_OK;
  }
  a.gq = dq_out;
  a.gk = dk_out;
  a.dq = dq;
  a.dk = dk;
  Stages stg(stream, kNormStages);
  stg.mark(launch_norm_rope_bwd(a, cfg->d, cfg->in_dtype == GDN_BF16, cfg->grad_dtype == GDN_BF16, stream));
  return finish();
}

gdn_status gdn_cpr_page_map(int32_t num_seqs, int32_t total_tokens, int32_t page_size, int32_t max_blocks,
                            int32_t num_free, const int32_t* lens, const int32_t* new_lens, const int32_t* free_pages,
                            int32_t* block_table, int32_t* seq_lens, int32_t* cu_seqlens, int32_t* positions,
                            int32_t* slot_map, int32_t* pages_used, void* ws, size_t ws_bytes, gdn_stream_t stream) {
  NvtxRange nvtx("gdn_cpr_page_map");
  if (num_seqs < 0 || total_tokens < 0 || page_size <= 0 || max_blocks < 0 || num_free < 0)
    return GDN_ERR_INVALID_ARG;
  const int shift = page_shift_of(page_size);
  if (shift < 0 || num_seqs > kPageMapMaxSeqs) return GDN_ERR_UNSUPPORTED;
  if (!ok_ptr(cu_seqlens, 4) || !ok_ptr(pages_used, 4)) return GDN_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!ok_ptr(lens, 4) || !ok_ptr(new_lens, 4) || !ok_ptr(seq_lens, 4))) return GDN_ERR_INVALID_ARG;
  if (num_seqs > 0 && max_blocks > 0 && !ok_ptr(block_table, 4)) return GDN_ERR_INVALID_ARG;
  if (num_free > 0 && !ok_ptr(free_pages, 4)) return GDN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!ok_ptr(positions, 16) || !ok_ptr(slot_map, 16))) return GDN_ERR_INVALID_ARG;
  if (!ok_ws(ws, ws_bytes, GDN_CPR_ATTN_HEADER_BYTES)) return GDN_ERR_WORKSPACE;
  PageMap a{};
  a.N = num_seqs;
  a.T = total_tokens;
  a.page_shift = shift;
  a.max_blocks = max_blocks;
  a.num_free = num_free;
  a.lens = lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.cu = cu_seqlens;
  a.positions = positions;
  a.slot_map = slot_map;
  a.pages_used = pages_used;
  a.hdr = static_cast<WsHeader*>(ws);
  Stages stg(stream, kMapStages);
  launch_page_map(a, stream);
  stg.mark(1);
  return finish();
}

gdn_status gdn_cpr_paged_decode_workspace_size(const gdn_cpr_attn* attn, int32_t num_seqs, int32_t max_len,
                                               size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  const gdn_status rc = check_attn(attn);
  if (rc != GDN_OK) return rc;
  if (num_seqs < 0 || max_len < 0) return GDN_ERR_INVALID_ARG;
  *bytes = decode_bytes(attn, num_seqs, decode_splits(attn, max_len));
  return GDN_OK;
}

gdn_status gdn_cpr_paged_decode(const gdn_cpr_attn* attn, int32_t num_seqs, int32_t max_len, const void* q,
                                const void* k_pages, const void* v_pages, int32_t num_pages, int32_t page_size,
                                const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens, void* out,
                                float* lse, void* ws, size_t ws_bytes, gdn_stream_t stream) {
  NvtxRange nvtx("gdn_cpr_paged_decode");
  gdn_status rc = check_attn(attn);
  if (rc != GDN_OK) return rc;
  if (num_seqs < 0 || max_len < 0 || num_pages < 0 || page_size <= 0 || max_blocks < 0) return GDN_ERR_INVALID_ARG;
  const int shift = page_shift_of(page_size);
  if (shift < 0 || num_seqs > 65535) return GDN_ERR_UNSUPPORTED;
  // the kernels keep a key's row (page, head, offset) in 32 bits
  if ((((int64_t)num_pages * attn->h_kv) << shift) >= (int64_t)UINT32_MAX) return GDN_ERR_UNSUPPORTED;
  if (num_seqs > 0 && (!ok_ptr(q, 16) || !ok_ptr(out, 16) || !ok_ptr(seq_lens, 4) || !aligned(lse, 4)))
    return GDN_ERR_INVALID_ARG;
  if (num_seqs > 0 && num_pages > 0 && (!ok_ptr(k_pages, 16) || !ok_ptr(v_pages, 16))) return GDN_ERR_INVALID_ARG;
  if (num_seqs > 0 && max_blocks > 0 && !ok_ptr(block_table, 4)) return GDN_ERR_INVALID_ARG;
  const int splits = decode_splits(attn, max_len);
  // runs are numbered in 32 bits (at most 16 query heads of a key head to one)
  const int64_t parts = (attn->h_q / attn->h_kv + 15) / 16;
  if ((double)num_seqs * attn->h_kv * parts * splits >= (double)(1 << 30)) return GDN_ERR_UNSUPPORTED;
  if (!ok_ws(ws, ws_bytes, decode_bytes(attn, num_seqs, splits))) return GDN_ERR_WORKSPACE;
  if (num_seqs == 0) return empty_call(ws, stream);
  PagedDecode a{};
  a.N = num_seqs;
  a.hq = attn->h_q;
  a.hkv = attn->h_kv;
  a.d = attn->d;
  a.window = attn->window;
  a.sinks = attn->sinks;
  a.max_len = max_len;
  a.scale = scale_of(attn);
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.num_pages = num_pages;
  a.page_shift = shift;
  a.max_blocks = max_blocks;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.partial = reinterpret_cast<float*>(at(ws, GDN_CPR_ATTN_HEADER_BYTES));
  a.max_splits = splits;
  a.hdr = static_cast<WsHeader*>(ws);
  Stages stg(stream, kPagedStages);
  stg.mark(launch_paged_decode(a, attn->dtype == GDN_BF16, stream));
  return finish();
}

gdn_status gdn_cpr_window_attn_workspace_size(const gdn_cpr_attn* attn, int32_t total_q, int32_t backward,
                                              size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  const gdn_status rc = check_attn(attn);
  if (rc != GDN_OK) return rc;
  if (total_q < 0) return GDN_ERR_INVALID_ARG;
  *bytes = window_bytes(attn, total_q, backward != 0);
  return GDN_OK;
}

gdn_status gdn_cpr_window_attn(const gdn_cpr_attn* attn, int32_t num_seqs, int32_t total_q, int32_t total_k,
                               const int32_t* cu_q, const int32_t* cu_k, const void* q, const void* k, const void* v,
                               void* out, float* lse, void* ws, size_t ws_bytes, gdn_stream_t stream) {
  NvtxRange nvtx("gdn_cpr_window_attn");
  WindowAttn w;
  const gdn_status rc = window_args(attn, num_seqs, total_q, total_k, cu_q, cu_k, q, k, v, &w);
  if (rc != GDN_OK) return rc;
  if (total_q > 0 && (!ok_ptr(out, 16) || !ok_ptr(lse, 4))) return GDN_ERR_INVALID_ARG;
  if (!ok_ws(ws, ws_bytes, window_bytes(attn, total_q, false))) return GDN_ERR_WORKSPACE;
  if (num_seqs == 0) return empty_call(ws, stream);
  w.out = out;
  w.lse = lse;
  w.hdr = static_cast<WsHeader*>(ws);
  w.fault_wait = take_wait_fault(window_on_tensor_cores(attn));
  Stages stg(stream, kWindowStages);
  if (!launch_window_attn(w, attn->dtype == GDN_BF16, stream)) return GDN_ERR_CUDA;
  stg.mark(1);
  return finish();
}

gdn_status gdn_cpr_window_attn_bwd(const gdn_cpr_attn* attn, int32_t num_seqs, int32_t total_q, int32_t total_k,
                                   const int32_t* cu_q, const int32_t* cu_k, const void* q, const void* k,
                                   const void* v, const void* out, const float* lse, const void* dout, void* dq,
                                   void* dk, void* dv, void* ws, size_t ws_bytes, gdn_stream_t stream) {
  NvtxRange nvtx("gdn_cpr_window_attn_bwd");
  WindowAttn w;
  const gdn_status rc = window_args(attn, num_seqs, total_q, total_k, cu_q, cu_k, q, k, v, &w);
  if (rc != GDN_OK) return rc;
  if (total_q > 0 && (!ok_ptr(out, 16) || !ok_ptr(lse, 4) || !ok_ptr(dout, 16) || !ok_ptr(dq, 16)))
    return GDN_ERR_INVALID_ARG;
  if (total_k > 0 && (!ok_ptr(dk, 16) || !ok_ptr(dv, 16))) return GDN_ERR_INVALID_ARG;
  if (!ok_ws(ws, ws_bytes, window_bytes(attn, total_q, true))) return GDN_ERR_WORKSPACE;
  if (num_seqs == 0) return empty_call(ws, stream);
  w.out = const_cast<void*>(out);
  w.lse = const_cast<float*>(lse);
  w.dout = dout;
  w.dq = dq;
  w.dk = dk;
  w.dv = dv;
  w.delta = reinterpret_cast<float*>(at(ws, GDN_CPR_ATTN_HEADER_BYTES));
  w.hdr = static_cast<WsHeader*>(ws);
  w.fault_wait = take_wait_fault(window_on_tensor_cores(attn));
  Stages stg(stream, kWindowBwdStages);
  const bool bf16 = attn->dtype == GDN_BF16;
  w.few = bf16 ? few_positions(w.window, w.sinks) : 0;
  if (!launch_window_dq(w, bf16, stream)) return GDN_ERR_CUDA;
  stg.mark(bf16 ? 2 : 1);
  if (!launch_window_dkv(w, bf16, stream)) return GDN_ERR_CUDA;
  stg.mark(1);
  return finish();
}

}  // extern "C"
