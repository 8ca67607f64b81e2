/*
 * gdn_cpr.h -- C ABI of the CPR Gated DeltaNet library (sm_103a, one GPU).
 *
 * The operator (Gated DeltaNet; IsoExec page "IsoExec: SkyRLにおけるトレーナーと推論の
 * ミスマッチを解消する", section "Chunkwise-Parallel Recurrent (CPR) Gated DeltaNet"), per
 * (sequence, value head) with an fp32 state S of d_v x d_k:
 *
 *     S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,      o_t = S_t q_t.
 *
 * CPR, as that section describes it, keeps this recurrence as the main computation but
 * evaluates it in parallel across chunks of C tokens, and resynchronises the decode
 * state every C tokens.  Concretely, in this library:
 *   - a boundary pass computes the state S^(j) before every chunk j (chunks aligned to
 *     each sequence's own first token) with the chunk (WY/UT) form, sequentially in j;
 *   - every chunk then runs the token recurrence from its own S^(j), all chunks at once;
 *   - decode runs the same token step on a running state and, whenever a chunk's C-th
 *     token has been appended, replaces that running state by the next boundary state,
 *     computed by the same boundary code on the cached chunk.
 * Every mode uses one token-step routine and one boundary routine with fixed reduction
 * orders, so prefill, trainer forward and decode give bit-identical o and states, for any
 * batch size, packing or slot assignment.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layouts (row-major, densely packed; T = total tokens, N = sequences or decode slots):
 *     q, k        [T, H_qk, d_k]   in_dtype
 *     v           [T, H_v,  d_v]   in_dtype
 *     g, beta     [T, H_v]         fp32 (g is the log decay: the step multiplies S by exp(g))
 *     o           [T, H_v,  d_v]   out_dtype
 *     states      [N, H_v, d_v, d_k] fp32 (row i of S is value dim i; o = S q)
 *     cu_seqlens  [N + 1] int32, cu_seqlens[0] = 0, non-decreasing, cu_seqlens[N] = T
 * Grouped heads: value head h reads query/key head h / (H_v / H_qk).  No scale is applied
 * to q.  Sequences of length 0 are allowed (state_out = state_in, bit for bit).
 *
 * Supported configurations ("claims"; anything else returns GDN_ERR_UNSUPPORTED before any
 * work is queued, in the spirit of the IsoExec contract's topology claims on the
 * hegai.media page, section "Что именно объединяет IsoExec"):
 *     d_k == d_v in {32, 64, 128};  chunk C in {16, 32, 64};  H_v % H_qk == 0;
 *     in_dtype in {GDN_F32, GDN_BF16};  out_dtype in {GDN_F32, GDN_BF16};
 *     every tensor pointer 16-byte aligned (g, beta: 4-byte).
 *
 * Ownership: the caller allocates and owns every buffer, including the workspace.  The
 * library allocates no device memory and keeps no mutable global state apart from the
 * optional per-thread hooks (gdn_cpr_set_profile, gdn_cpr_test_wait_timeout) and the
 * built-in scratch array of gdn_cpr_decode_step_noalloc.
 *
 * Execution: every call only queues work on `stream` and returns; nothing synchronises
 * except gdn_cpr_get_device_error.  Inputs must stay valid until the stream reaches the
 * queued work.  cu_seqlens_host must describe the same values as cu_seqlens_dev; it is
 * read on the host during the call (grid and workspace sizing) and not kept.
 *
 * Errors: argument errors are returned synchronously and nothing is queued.  Errors that
 * only the device can see (device cu_seqlens disagreeing with the host copy, a decode
 * slot out of range, a bounded wait that gave up) are recorded in an error word inside the
 * workspace; the affected kernels then skip their work (they never read or write out of
 * bounds), and gdn_cpr_get_device_error reports the code.  Each call clears the word
 * when it starts.  No kernel traps or asserts.
 */
#ifndef GDN_CPR_H
#define GDN_CPR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *gdn_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad sizes, bad cu_seqlens_host */
    GDN_ERR_UNSUPPORTED = 2, /* outside the supported configurations listed above */
    GDN_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed */
    GDN_ERR_WORKSPACE = 4,   /* workspace NULL, misaligned or smaller than required */
    GDN_ERR_DEVICE = 5       /* returned by gdn_cpr_get_device_error when the word is set */
} gdn_status;

/* Codes stored in the device error word (read back by gdn_cpr_get_device_error). */
typedef enum {
    GDN_DEVERR_NONE = 0,
    GDN_DEVERR_CU_SEQLENS = 1, /* device cu_seqlens disagree with cu_seqlens_host */
    GDN_DEVERR_SLOT = 2,       /* decode slot index outside [0, cache.slots) */
    GDN_DEVERR_POS = 3,        /* negative cache position */
    GDN_DEVERR_TIMEOUT = 4,    /* a bounded on-device wait gave up */
    GDN_DEVERR_BOUNDS = 5,     /* bounds-checked builds only (GDN_CHECKED): a work item's index
                                  range fell outside its buffer; the item was skipped */
    GDN_DEVERR_POS_HOST = 6,   /* gdn_cpr_decode_step_pos: the host positions said no token
                                  completes a chunk, the cache says one does; step skipped */
    GDN_DEVERR_PAGES = 7       /* page operators: free list too short, block table too narrow,
                                  or a page index outside the cache */
} gdn_device_error;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

typedef enum {
    GDN_MODE_PREFILL = 0, /* gdn_cpr_prefill */
    GDN_MODE_DECODE = 1,  /* gdn_cpr_decode_step */
    GDN_MODE_FWD = 2,     /* gdn_cpr_fwd */
    GDN_MODE_BWD = 3,     /* gdn_cpr_bwd */
    GDN_MODE_CONTINUE = 4 /* gdn_cpr_prefill_continue (upper bound over cache positions) */
} gdn_mode;

typedef struct {
    int32_t num_seqs;     /* N: sequences (prefill/fwd/bwd) or tokens this step (decode) */
    int32_t total_tokens; /* T: cu_seqlens[N] (prefill/fwd/bwd); N for decode */
    int32_t h_qk;         /* query/key heads */
    int32_t h_v;          /* value heads (state heads) */
    int32_t d_k;          /* key dim */
    int32_t d_v;          /* value dim */
    int32_t chunk;        /* C */
    gdn_dtype in_dtype;   /* q, k, v */
    gdn_dtype out_dtype;  /* o */
} gdn_cpr_shape;

/* Decode cache: everything needed to continue a sequence bit-exactly (also the full
 * checkpoint of a decoding sequence: copy it out and back to resume).  All arrays are
 * caller-owned device memory, indexed by slot.
 *   s_run     [slots, H_v, d_v, d_k] fp32   running state (recurrent since the last boundary),
 *                                             held scaled: the state is c_run * s_run
 *   c_run     [slots, H_v] fp32           its scale (1 right after a boundary; see token_step)
 *   s_bnd     [slots, H_v, d_v, d_k] fp32   boundary state before the current chunk
 *   tail_k    [slots, C, H_qk, d_k]  in_dtype  keys of the current, unfinished chunk
 *   tail_v    [slots, C, H_v,  d_v]  in_dtype  values of the current chunk
 *   tail_g    [slots, C, H_v]        fp32
 *   tail_beta [slots, C, H_v]        fp32
 *   pos       [slots] int32          tokens consumed so far by the slot's sequence          */
typedef struct {
    float *s_run;
    float *c_run;
    float *s_bnd;
    void *tail_k;
    void *tail_v;
    float *tail_g;
    float *tail_beta;
    int32_t *pos;
    int32_t slots;
} gdn_cpr_cache;

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int gdn_cpr_version(void);

/* Static, human-readable name of a status code. */
const char *gdn_cpr_status_string(gdn_status s);

/* Bytes of workspace the given mode needs for this shape.  cu_seqlens_host [N+1] is
 * required for PREFILL, FWD and BWD (the size depends on the number of chunks,
 * sum over sequences of ceil(L/C)) and ignored for DECODE.  The workspace must be
 * 256-byte aligned.  Returns GDN_ERR_INVALID_ARG / GDN_ERR_UNSUPPORTED like the calls. */
gdn_status gdn_cpr_workspace_size(const gdn_cpr_shape *shape, gdn_mode mode,
                                  const int32_t *cu_seqlens_host, size_t *bytes);

/* Prefill (rollout prefill; IsoExec page section "Chunkwise-Parallel Recurrent (CPR)
 * Gated DeltaNet": the recurrence evaluated in parallel across chunks).
 *   q, k, v, g, beta    inputs, layouts above (device)
 *   state_in            [N, H_v, d_v, d_k] fp32 or NULL for zero (device)
 *   cu_seqlens_dev/host the same N+1 offsets, on the device and on the host
 *   o                   output [T, H_v, d_v] in out_dtype (device)
 *   state_out           NULL or [N, H_v, d_v, d_k]: the state decode continues from --
 *                       the boundary state S^(L/C) if L % C == 0, else the token
 *                       recurrence from S^(floor(L/C)) through the last L % C tokens
 *   cache_out           NULL or a decode cache to initialise for these sequences:
 *                       s_run = state_out, s_bnd = S^(floor(L/C)), tail = the last L % C
 *                       tokens, pos = L, at slot slot_of_seq[n] (NULL: slot n)
 *   slot_of_seq         NULL or [N] int32 device array of distinct slots
 *   ws, ws_bytes        workspace of gdn_cpr_workspace_size(GDN_MODE_PREFILL) bytes  */
gdn_status gdn_cpr_prefill(const gdn_cpr_shape *shape, const void *q, const void *k,
                           const void *v, const float *g, const float *beta,
                           const float *state_in, const int32_t *cu_seqlens_dev,
                           const int32_t *cu_seqlens_host, void *o, float *state_out,
                           const gdn_cpr_cache *cache_out, const int32_t *slot_of_seq, void *ws,
                           size_t ws_bytes, gdn_stream_t stream);

/* One decode token for each of N slots (rollout decode; IsoExec page section
 * "Chunkwise-Parallel Recurrent (CPR) Gated DeltaNet": the hidden state is resynchronised
 * every C tokens).  shape->num_seqs = shape->total_tokens = N.
 *   q, k [N, H_qk, d_k], v [N, H_v, d_v], g, beta [N, H_v]: this step's token per slot
 *   slot [N] int32 device: distinct cache slots (out of range -> device error, skipped)
 *   cache               updated in place: s_run stepped, token appended to the tail, pos+1;
 *                       when pos+1 is a multiple of C the boundary state is advanced over
 *                       the completed chunk and s_run is replaced by it
 *   o [N, H_v, d_v]     output
 * The launch configuration depends only on N and the shape, and the resync decision is
 * taken on the device from pos, so a step can be captured in a CUDA graph once the
 * workspace and pointers are fixed.                                                     */
gdn_status gdn_cpr_decode_step(const gdn_cpr_shape *shape, const void *q, const void *k,
                               const void *v, const float *g, const float *beta,
                               const int32_t *slot, const gdn_cpr_cache *cache, void *o,
                               void *ws, size_t ws_bytes, gdn_stream_t stream);

/* gdn_cpr_decode_step for callers that know the slots' positions on the host (a serving
 * scheduler tracks every sequence's length): pos_host [N] is the host copy of
 * cache->pos[slot[n]] before this step, read during the call and not kept.  When no token of
 * the step completes a chunk ((pos_host[n] + 1) % C != 0 for every n), the resynchronisation
 * kernels are not launched at all -- two launches fewer per step; otherwise the call is
 * exactly gdn_cpr_decode_step.  Results and bits are those of gdn_cpr_decode_step.  The
 * claim is checked on the device: if a slot's cache position does complete a chunk after
 * all, the whole step is skipped (nothing in the cache changes, o is not written) and the
 * workspace's error word reads GDN_DEVERR_POS_HOST.  A negative pos_host entry returns
 * GDN_ERR_INVALID_ARG.  The launch sequence depends on pos_host, so a CUDA graph captured
 * with it is valid only for steps at those positions.                                     */
gdn_status gdn_cpr_decode_step_pos(const gdn_cpr_shape *shape, const void *q, const void *k,
                                   const void *v, const float *g, const float *beta,
                                   const int32_t *slot, const int32_t *pos_host,
                                   const gdn_cpr_cache *cache, void *o, void *ws, size_t ws_bytes,
                                   gdn_stream_t stream);

/* Trainer forward (case "trainer_fwd" next to "engine_prefill" on the IsoExec page,
 * section on contract structure).  Identical arithmetic to gdn_cpr_prefill -- o and
 * state_out are bit-identical -- and additionally saves the boundary states:
 *   saved_bnd [sum_s ceil(L_s/C), H_v, d_v, d_k] fp32: the state before every chunk, chunks
 *             numbered in sequence order (chunk 0 of a sequence holds its state_in).     */
gdn_status gdn_cpr_fwd(const gdn_cpr_shape *shape, const void *q, const void *k, const void *v,
                       const float *g, const float *beta, const float *state_in,
                       const int32_t *cu_seqlens_dev, const int32_t *cu_seqlens_host, void *o,
                       float *state_out, float *saved_bnd, void *ws, size_t ws_bytes,
                       gdn_stream_t stream);

/* Trainer backward (IsoExec page, CPR timing table row "Trainer Fwd+Bwd").  Gradient of
 * loss = <dO, o> + <dstate_out, state_out> with respect to every input, where o and
 * state_out are gdn_cpr_fwd's outputs.  Uses saved_bnd from gdn_cpr_fwd on the same
 * inputs.  Reverse chain over chunks for the boundary adjoints, then every chunk in
 * parallel; grouped-head dq/dk are summed over the value heads of a group in ascending
 * order; no atomics, so results are deterministic.
 *   dO [T, H_v, d_v] out_dtype; dstate_out NULL (= 0) or [N, H_v, d_v, d_k] fp32
 *   dq, dk [T, H_qk, d_k] fp32; dv [T, H_v, d_v] fp32; dg, dbeta [T, H_v] fp32
 *   dstate_in NULL or [N, H_v, d_v, d_k] fp32                                            */
gdn_status gdn_cpr_bwd(const gdn_cpr_shape *shape, const void *q, const void *k, const void *v,
                       const float *g, const float *beta, const float *state_in,
                       const int32_t *cu_seqlens_dev, const int32_t *cu_seqlens_host,
                       const float *saved_bnd, const void *dO, const float *dstate_out,
                       float *dq, float *dk, float *dv, float *dg, float *dbeta,
                       float *dstate_in, void *ws, size_t ws_bytes, gdn_stream_t stream);

/* Prefill continued from a decode cache at any position: chunked prefill, and decode of
 * several tokens per sequence at once (the IsoExec page's CPR section: decode continues the
 * same recurrence and resynchronises every C tokens; this extends a cached sequence by any
 * number of tokens with the bits of one prefill of the whole sequence).  Sequence i appends
 * L_i = cu_seqlens[i+1] - cu_seqlens[i] tokens to cache slot slot_dev[i], whose position
 * pos_host[i] (host copy of cache->pos[slot_dev[i]]; checked on the device, a mismatch sets
 * GDN_DEVERR_CU_SEQLENS and nothing runs) may lie inside a chunk.  The r_i = pos_host[i] % C
 * tokens of the slot's tail are replayed with the new ones from the slot's boundary state,
 * so that every output and the updated cache are bit-identical to a single gdn_cpr_prefill
 * of the whole sequence (and to gdn_cpr_decode_step token by token).
 *   q, k, v, g, beta, o  the new tokens only, laid out as for gdn_cpr_prefill
 *   slot_dev [N] int32 device, distinct slots; cache  updated in place: s_run, s_bnd, tail,
 *                        pos += L_i
 *   state_out            NULL or [N, H_v, d_v, d_k]: the state after the last token
 *   ws, ws_bytes         gdn_cpr_workspace_size(GDN_MODE_CONTINUE, cu_seqlens_host) bytes
 * Argument errors (NULL or misaligned pointers, negative positions) are returned; a slot
 * out of range on the device sets GDN_DEVERR_SLOT.                                        */
gdn_status gdn_cpr_prefill_continue(const gdn_cpr_shape *shape, const void *q, const void *k,
                                    const void *v, const float *g, const float *beta,
                                    const int32_t *cu_seqlens_dev, const int32_t *cu_seqlens_host,
                                    const int32_t *slot_dev, const int32_t *pos_host,
                                    const gdn_cpr_cache *cache, void *o, float *state_out, void *ws,
                                    size_t ws_bytes, gdn_stream_t stream);

/* The explicit running state of decode cache slots (the state decode continues from, as
 * gdn_cpr_prefill returns it in state_out): out[i] = c_run[s] * s_run[s] for s = slots_dev[i],
 * every value head, one round-to-nearest fp32 product per element -- the same product the
 * kernels use when a scaled running state leaves them as state_out, so a cache read back
 * here equals the state_out of the same sequence bit for bit.  (IsoExec page, section
 * "Chunkwise-Parallel Recurrent (CPR) Gated DeltaNet": decode continues the recurrence on a
 * running state; the cache holds it as c_run * s_run, see gdn_cpr_cache.)
 *   shape      only h_v, d_k = d_v (and the configuration checks) are used
 *   cache      the decode cache to read (device)
 *   slots_dev  [n] int32 device slot indices, or NULL for slots 0 .. n-1 (n <= cache->slots)
 *   out        [n, H_v, d_v, d_k] fp32 device, 16-byte aligned
 * Queues one kernel on `stream`.  A slot index outside [0, cache->slots) on the device gives
 * an all-NaN block for that entry.  Argument errors are returned and nothing is queued. */
gdn_status gdn_cpr_running_state(const gdn_cpr_shape *shape, const gdn_cpr_cache *cache,
                                 const int32_t *slots_dev, int32_t n, float *out,
                                 gdn_stream_t stream);

/* Numerical-policy identity (IsoExec pages, section on the structure of the execution
 * contract, item "Identities": SHA-256 digests by which trainer and rollout engine check
 * that they run the same verified numerical policy).  Writes into digest[32] the SHA-256
 * (FIPS 180-4) of a canonical text listing every choice that decides the bits of this
 * library's results for the given shape: d_k, d_v, chunk length, input and output dtypes,
 * the boundary path (tensor cores with split-bf16 operands, or fp32 SIMT), the reduction
 * orders of the token step, the triangular solve and the cumulative sum, the exponential,
 * the rounding of the output and the library version.  The number of sequences, tokens
 * and heads do not enter it: shapes whose results are bit-identical share a digest.
 * When text is non-NULL it also receives that text, NUL-terminated and truncated to
 * text_len bytes.  Host only, no GPU work.  Returns GDN_ERR_INVALID_ARG for a NULL shape
 * or digest and GDN_ERR_UNSUPPORTED / GDN_ERR_INVALID_ARG for shapes the calls reject.
 * This library's own addition: the pages name the digests but define no content.     */
gdn_status gdn_cpr_policy_digest(const gdn_cpr_shape *shape, unsigned char digest[32], char *text,
                                 size_t text_len);

/* Optional profiling hook (per calling thread; NULL disables it, the default).  While set,
 * every entry point called from this thread records events[i] (cudaEvent_t handles created
 * by the caller) on its stream at its stage boundaries -- events[0] before its first
 * kernel, events[s] after stage s -- for as many stages as it has, up to n_events, and
 * adds the number of kernels it launched to *kernels.  Stages:
 *   prefill / fwd : 1 work list, 2 boundary pre-pass, 3 boundary chain, 4 intra-chunk
 *                   recurrence, 5 cache tail (prefill with a cache only)
 *   decode_step   : 1 token step, 2 resync (pre-pass and boundary step), 3 position advance
 *   bwd           : see gdn_cpr_bwd's stages in the implementation notes
 * The structure must stay valid while set.  Has no effect on results.                   */
typedef struct {
    void *events[16];   /* cudaEvent_t */
    int32_t n_events;   /* how many of events[] are valid */
    int32_t stages;     /* set by each call: how many stage events it recorded (incl. [0]) */
    int64_t kernels;    /* incremented by each call by the kernels it launched */
} gdn_cpr_profile;

void gdn_cpr_set_profile(gdn_cpr_profile *profile);

/* Size of the built-in device scratch used by gdn_cpr_decode_step_noalloc (64 MiB). */
#define GDN_CPR_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

/* gdn_cpr_decode_step without a caller-provided workspace, for callers that cannot
 * allocate device memory (a serving loop whose memory is reserved up front by another
 * allocator, code that must not call cudaMalloc while other GPU work is captured or
 * replayed, or a plain C host with no device allocator).  The IsoExec pages have no
 * counterpart: this is a deployment convenience, not part of CPR.
 *   Arguments, results and bits are exactly those of gdn_cpr_decode_step; only the
 *   workspace differs.  It lives in one file-scope device array of
 *   GDN_CPR_NOALLOC_SCRATCH_BYTES that every GPU which loads this library's module holds
 *   until the process exits.  The call itself allocates nothing (no cudaMalloc/cudaFree).
 *   Limit: the decode workspace of the shape (gdn_cpr_workspace_size with
 *   GDN_MODE_DECODE) must fit the array -- about 1000 (token, value head) pairs per step at
 *   d = 128, C = 64 (e.g. 31 slots x 32 heads); larger requests return GDN_ERR_WORKSPACE
 *   and queue nothing.
 *   The first call on a device looks up the array's device address (with that device
 *   current); make that first call before capturing any stream into a CUDA graph.  The
 *   address is kept with the identity of the context it belongs to; after a device reset
 *   the next call looks it up again (and is again a first call in that sense).
 *   Device-side errors of these calls (a slot out of range, ...) are recorded in the
 *   array's own error word: read them with gdn_cpr_noalloc_device_error.
 *   Every call on a device shares the array and leaves its contents behind; the step
 *   clears what must start at zero.  Calls that overlap on the GPU (other streams, other
 *   threads, concurrent graph replays) race on the array: serialise them.               */
gdn_status gdn_cpr_decode_step_noalloc(const gdn_cpr_shape *shape, const void *q, const void *k,
                                       const void *v, const float *g, const float *beta,
                                       const int32_t *slot, const gdn_cpr_cache *cache, void *o,
                                       gdn_stream_t stream);

/* Synchronises `stream`, then reads the device error word of the built-in scratch array
 * of the current device, which gdn_cpr_decode_step_noalloc uses as its workspace: the
 * device-side error (slot out of range, negative position, a bounded wait that gave up) of
 * the last no-alloc call on this device, as gdn_cpr_get_device_error reports it for a
 * caller-provided workspace.  Returns GDN_OK when the word is clear, GDN_ERR_DEVICE with
 * *code set when it is not, GDN_ERR_CUDA if the sync or read fails.  Allocates nothing.  */
gdn_status gdn_cpr_noalloc_device_error(gdn_stream_t stream, int32_t *code);

/* Test hook of the failure path (per calling thread; off by default): the next `calls`
 * prefill or trainer-forward calls from this thread whose boundary pass runs on tensor
 * cores make one CTA of the boundary chain wait, before it issues any copy or MMA, on a
 * barrier phase that nothing completes.  Its bounded wait (a short poll limit here) gives
 * up, the CTA records GDN_DEVERR_TIMEOUT in the workspace's error word, frees its tensor
 * memory and exits, so gdn_cpr_get_device_error reports the timeout and the context stays
 * usable.  The outputs of such a call are not valid.  calls <= 0 switches it off.
 * gdn_cpr_window_attn and gdn_cpr_window_attn_bwd calls on tensor cores (bf16, d = 64 or 128) count too:
 * there every CTA (of both gradient kernels) waits so, and gives up, with a copy under way. */
void gdn_cpr_test_wait_timeout(int32_t calls);

/* Synchronises `stream`, then reads the device error word of `ws` (the workspace of the
 * last call queued with it) into *code (a gdn_device_error).  Returns GDN_OK when the
 * word is clear, GDN_ERR_DEVICE when it is set, GDN_ERR_CUDA if the sync or copy fails. */
gdn_status gdn_cpr_get_device_error(const void *ws, gdn_stream_t stream, int32_t *code);

/* =====================================================================================
 * Attention-layer operators
 *
 * A hybrid model interleaves Gated DeltaNet layers with softmax-attention layers.  These are
 * the operators such layers need beside the recurrence above (this library's own addition;
 * the pages describe CPR only): the per-head norms and rotation of queries and keys, the
 * paged cache's bookkeeping, decode attention over that cache, and sliding-window attention
 * for prefill and training with its gradient.  The conventions above hold (caller-owned
 * memory, work only queued on `stream`, argument errors returned before anything is queued,
 * fixed reduction orders and no atomics in any arithmetic) with these additions:
 *
 * Layouts:  q, out [T, H_q, d];  k, v [T, H_kv, d];  query head h reads key head
 * h / (H_q / H_kv).  Cache pages: k_pages, v_pages [pages, H_kv, page_size, d] -- the rows of
 * one head of a page are contiguous.  block_table [N, max_blocks] int32: page of positions
 * b * page_size .. of request n.  A slot is page * page_size + offset.
 * Claims: d in {32, 64, 128}; dtypes fp32 and bf16; H_q % H_kv == 0; page_size a power of two
 * in [16, 256]; tensors 16-byte aligned.
 *
 * Visibility: a query at position p of its request sees key j when j <= p and (window == 0 or
 * p - j < window or j < sinks).  A query that sees no key gives a row of zeros (and a
 * log-sum-exp of -infinity), and its gradient is zero.
 *
 * Results for a request depend on that request alone: not on the batch it is in, its place in
 * the packing, the pages it lies on, or what lies in other requests' rows or in the unused
 * part of a page (infinities and NaN there included).
 * ===================================================================================== */
typedef enum { GDN_NORM_NONE = 0, GDN_NORM_RMS = 1, GDN_NORM_L2 = 2 } gdn_norm;
typedef enum { GDN_ROPE_HALF = 0, GDN_ROPE_INTERLEAVED = 1 } gdn_rope_layout;

typedef struct {
    int32_t tokens;      /* T */
    int32_t h_q, h_k;    /* heads of q and of k (and v); T (h_q + 2 h_k) < 2^31 */
    int32_t d;
    int32_t rot;         /* rotated entries at the front of every head: 0 or a multiple of 8, <= d */
    int32_t table_rows;  /* rows of cos and sin; at least 1 where tokens are rotated */
    gdn_norm norm;
    gdn_rope_layout layout;
    float eps;
    gdn_dtype in_dtype;   /* q, k, v, and the gradients dq, dk */
    gdn_dtype out_dtype;  /* q_out, k_out and the cache */
    gdn_dtype grad_dtype; /* dq_out, dk_out (backward) */
    int64_t q_stride, k_stride, v_stride; /* elements from one token of q, k, v to the next, so that
                                             they may be parts of one projection's rows; multiples
                                             of 16 bytes.  Everything else is dense. */
} gdn_cpr_norm_rope;

/* Norm and rotation of queries and keys, one pass:  y = R(pos) (x * r * w) per (token, head),
 *   r = 1, 1 / sqrt(mean x^2 + eps) (RMS) or 1 / sqrt(sum x^2 + eps) (L2; what gdn_cpr_prefill
 *   and gdn_cpr_fwd expect of q and k);  w [d] fp32 or NULL (ones);
 *   R turns the pairs (x_i, x_{i + rot/2}) (half) or (x_{2i}, x_{2i+1}) (interleaved), i < rot/2,
 *   by (cos, sin)[pos][i]:  (a, b) -> (a c - b s, b c + a s).
 *   q_weight, k_weight  [d] fp32 or NULL
 *   cos, sin            [table_rows, rot / 2] fp32, positions [T] int32 (all NULL if rot == 0);
 *                       a token whose position lies outside the tables gets rows of NaN
 *   q_out, k_out        [T, H, d]; either may be NULL (that output is not wanted)
 *   k_pages, v_pages    NULL, or the paged cache: k_out's rows and v's rows (unchanged but for
 *                       the conversion to out_dtype) are written at slot_map [T] int32; a slot
 *                       outside [0, num_pages * page_size) is skipped (-1: a token not kept)  */
gdn_status gdn_cpr_qk_norm_rope(const gdn_cpr_norm_rope *cfg, const void *q, const void *k,
                                const void *v, const float *q_weight, const float *k_weight,
                                const float *cos, const float *sin, const int32_t *positions,
                                void *q_out, void *k_out, void *k_pages, void *v_pages,
                                int32_t num_pages, int32_t page_size, const int32_t *slot_map,
                                gdn_stream_t stream);

/* Its gradient.  With g = R^T dy and g' = g w:  dx = r g' - c r^3 (x . g') x, c = 1 / d (RMS),
 * 1 (L2) or 0;  dw = sum over tokens and heads of g x r, in a fixed order (fp32).
 *   dq_out, dk_out  [T, H, d] in grad_dtype;  dq, dk [T, H, d] in in_dtype
 *   dq_weight, dk_weight  [d] fp32, or both NULL; then no workspace is needed
 *   A token whose position lies outside the tables gives NaN in dq and dk and is left out of
 *   the weights' gradients.                                                                 */
gdn_status gdn_cpr_qk_norm_rope_bwd(const gdn_cpr_norm_rope *cfg, const void *q, const void *k,
                                    const float *q_weight, const float *k_weight, const float *cos,
                                    const float *sin, const int32_t *positions, const void *dq_out,
                                    const void *dk_out, void *dq, void *dk, float *dq_weight,
                                    float *dk_weight, void *ws, size_t ws_bytes,
                                    gdn_stream_t stream);
gdn_status gdn_cpr_qk_norm_rope_workspace_size(const gdn_cpr_norm_rope *cfg, size_t *bytes);

/* The paged cache's bookkeeping for one step, on the device, from request lengths.  Request n
 * has lens[n] cached tokens and appends new_lens[n]; it owns ceil(lens[n] / page_size) pages,
 * listed at the front of its block-table row, and takes those it lacks from free_pages, in
 * request order from the list's front.
 *   lens, new_lens [N] int32; free_pages [num_free] int32
 *   block_table [N, max_blocks] int32   updated: the new pages' entries, nothing else
 *   seq_lens [N] int32                  lens + new_lens
 *   cu_seqlens [N + 1] int32            offsets of the new tokens, packed
 *   positions, slot_map [total_tokens] int32  of every new token; total_tokens = sum new_lens
 *   pages_used [1] int32                how many entries of free_pages were taken
 * Nothing is taken off the list here, so a call may be repeated.  If total_tokens is not the
 * sum (GDN_DEVERR_CU_SEQLENS), a length is negative or their sum does not fit 32 bits
 * (GDN_DEVERR_POS), or the free list or a block-table row is too short (GDN_DEVERR_PAGES), the
 * error word says so, positions and slot_map are -1, seq_lens and cu_seqlens are zeros,
 * pages_used is 0 and the block table keeps its contents.  A page whose index is negative or
 * whose slots do not fit 32 bits sets GDN_DEVERR_PAGES too, and its tokens' slots are -1.
 * N <= 8192.
 *   ws: GDN_CPR_ATTN_HEADER_BYTES, 256-byte aligned (the error word)                         */
#define GDN_CPR_ATTN_HEADER_BYTES 256u
gdn_status gdn_cpr_page_map(int32_t num_seqs, int32_t total_tokens, int32_t page_size,
                            int32_t max_blocks, int32_t num_free, const int32_t *lens,
                            const int32_t *new_lens, const int32_t *free_pages,
                            int32_t *block_table, int32_t *seq_lens, int32_t *cu_seqlens,
                            int32_t *positions, int32_t *slot_map, int32_t *pages_used, void *ws,
                            size_t ws_bytes, gdn_stream_t stream);

typedef struct {
    int32_t h_q, h_kv, d;
    int32_t window; /* keys a query sees behind it, itself included; 0 = all */
    int32_t sinks;  /* first keys that stay visible outside the window */
    float scale;    /* of the scores; 0 = 1 / sqrt(d) */
    gdn_dtype dtype; /* q, k, v, out and their gradients */
} gdn_cpr_attn;

/* Attention of one new token per request over the paged cache: q [N, H_q, d] is the token at
 * position seq_lens[n] - 1, whose key and value are already in the cache.  seq_lens[n] = 0
 * gives zeros.  The visible keys are split over their count and joined in a fixed order.
 *   seq_lens [N] int32; max_len >= every seq_lens (sizes the grid and, without a window, the
 *   workspace: about H_q max_len / 512 records of d + 2 floats a request; a longer or negative
 *   length sets GDN_DEVERR_POS and gives NaN for that request); a page index outside
 *   [0, num_pages) sets GDN_DEVERR_PAGES, NaN likewise
 *   out [N, H_q, d];  lse NULL or [N, H_q] fp32: the log-sum-exp of the scaled scores
 *   num_pages * H_kv * page_size < 2^32 - 1; N <= 65535; fewer than 2^30 runs at max_len over
 *   the batch (N H_kv ceil(H_q / H_kv / 16) max(1, max_len / 512), or by the visible keys)
 *   ws: gdn_cpr_paged_decode_workspace_size bytes; its error word is set by every call      */
gdn_status gdn_cpr_paged_decode(const gdn_cpr_attn *attn, int32_t num_seqs, int32_t max_len,
                                const void *q, const void *k_pages, const void *v_pages,
                                int32_t num_pages, int32_t page_size, const int32_t *block_table,
                                int32_t max_blocks, const int32_t *seq_lens, void *out, float *lse,
                                void *ws, size_t ws_bytes, gdn_stream_t stream);
gdn_status gdn_cpr_paged_decode_workspace_size(const gdn_cpr_attn *attn, int32_t num_seqs,
                                               int32_t max_len, size_t *bytes);

/* Causal attention over packed sequences with a sliding window and first keys that stay
 * visible (prefill and trainer forward).  Sequence n has queries cu_q[n] .. and keys cu_k[n]
 * ..; the last query is at the last key's position, so fewer queries than keys continue a
 * sequence, and with more the first rows see nothing.
 *   total_q, total_k  rows of q and of k, v: cu_q[N], cu_k[N]; at most 2^30
 *   cu_q, cu_k        [N + 1] int32 on the device only; a table that is not non-decreasing from
 *                     0 to its total sets GDN_DEVERR_CU_SEQLENS (outputs are then not valid)
 *   out [total_q, H_q, d];  lse [total_q, H_q] fp32, natural logarithm
 *   ws: gdn_cpr_window_attn_workspace_size bytes; its error word is set by every call       */
gdn_status gdn_cpr_window_attn(const gdn_cpr_attn *attn, int32_t num_seqs, int32_t total_q,
                               int32_t total_k, const int32_t *cu_q, const int32_t *cu_k,
                               const void *q, const void *k, const void *v, void *out, float *lse,
                               void *ws, size_t ws_bytes, gdn_stream_t stream);

/* Its gradient, from the forward's out and lse.  dq [total_q, H_q, d]; dk, dv [total_k, H_kv,
 * d], summed over a group's heads in a fixed order; deterministic.
 * In both a masked key or value of the same sequence may take part with weight 0, so an infinity or
 * NaN there can reach rows that do not see it; other sequences' rows never do.             */
gdn_status gdn_cpr_window_attn_bwd(const gdn_cpr_attn *attn, int32_t num_seqs, int32_t total_q,
                                   int32_t total_k, const int32_t *cu_q, const int32_t *cu_k,
                                   const void *q, const void *k, const void *v, const void *out,
                                   const float *lse, const void *dout, void *dq, void *dk, void *dv,
                                   void *ws, size_t ws_bytes, gdn_stream_t stream);
gdn_status gdn_cpr_window_attn_workspace_size(const gdn_cpr_attn *attn, int32_t total_q,
                                              int32_t backward, size_t *bytes);

/* =====================================================================================
 * 8-bit cache
 *
 * The paged cache with keys and values in 8 bits: half the memory of bf16 pages, and half the
 * bytes of a decode step.  A block is `block` consecutive tokens of one key head, x [block, d]; it
 * is held as 8-bit codes c and one fp32 scale s and stands for c s:
 *   GDN_INT8  s = max|x| / 127, c = 127 x / max|x| to the nearest whole number, ties to even
 *   GDN_E4M3  s = the least power of two 2^e with max|x| <= 448 2^e, c = x / s to the nearest e4m3
 *             value, ties to even
 * A block whose max|x| lies below 2^-100 is held as zeros with s = 0; one that holds an infinity or
 * a NaN as zeros with s = NaN, so that all of it reads as NaN.  (In e4m3 a value of 1.9375 2^127 or
 * more rounds to 2^128, which reads as an infinity.)
 *
 * Only whole blocks are held in 8 bits.  The rows of a request's unfinished block wait, as they
 * came, in its tail: of seq_len tokens the first seq_len / block * block are in the pages, the
 * others in rows 0 .. of tail[slot].  So every block is rounded once, from the values that were
 * appended, and what the cache holds does not depend on how the tokens were split over calls.
 *
 * Layouts:  k_pages, v_pages [num_pages, h_kv, page_size, d] 8 bits;  k_scale, v_scale [num_pages,
 * h_kv, page_size / block] fp32;  k_tail, v_tail [slots, h_kv, block, d] in dtype.  Request n has
 * the tail slot[n] (NULL: n); slots of one call are distinct.  block_table, seq_lens and the
 * conventions of the attention-layer operators above apply.
 * Claims: theirs, and block in {16, 32, 64, 128}, block <= page_size; num_pages * h_kv * page_size
 * and slots * h_kv * block below 2^32 - 1; h_kv <= 65535, N <= 65535.
 * ===================================================================================== */
typedef enum { GDN_INT8 = 0, GDN_E4M3 = 1 } gdn_code;

typedef struct {
    int32_t num_pages, page_size, block, slots, h_kv, d;
    gdn_code code;
    gdn_dtype dtype; /* of the tails, of what is appended, and of q and out in decode */
    void *k_pages, *v_pages;
    float *k_scale, *v_scale;
    void *k_tail, *v_tail;
} gdn_cpr_quant_cache;

/* New keys and values into the cache.  Request n appends the tokens cu_seqlens[n] .. of k and v; its
 * length afterwards is seq_lens[n] (what gdn_cpr_page_map gives).  Every block that they complete is
 * written to the page of the block table that covers it; the rows of an unfinished block go to the tail.
 *   k, v        [total_tokens, h_kv, d] in dtype; k_stride, v_stride elements from one token to the
 *               next (multiples of 16 bytes)
 *   cu_seqlens  [N + 1] int32, seq_lens [N] int32, block_table [N, max_blocks] int32
 *   Skipped, and reported by the error word: a request whose offsets are not 0 <= cu_seqlens[n] <=
 *   cu_seqlens[n + 1] <= total_tokens, or all offsets if cu_seqlens does not run from 0 to
 *   total_tokens (GDN_DEVERR_CU_SEQLENS; where its own offsets fit, a request may have been written);
 *   a request whose length is negative or less than what it appends (GDN_DEVERR_POS); one whose
 *   slot lies outside [0, slots) (GDN_DEVERR_SLOT); a block whose page lies outside the cache or the
 *   block table (GDN_DEVERR_PAGES).  A request that appends nothing is left alone.
 *   ws: GDN_CPR_ATTN_HEADER_BYTES, 256-byte aligned (the error word, set by every call), or NULL:
 *   what is wrong is skipped as above and not reported, and the call is one kernel            */
gdn_status gdn_cpr_quant_append(const gdn_cpr_quant_cache *cache, int32_t num_seqs,
                                int32_t total_tokens, const void *k, const void *v,
                                int64_t k_stride, int64_t v_stride, const int32_t *cu_seqlens,
                                const int32_t *seq_lens, const int32_t *block_table,
                                int32_t max_blocks, const int32_t *slot, void *ws, size_t ws_bytes,
                                gdn_stream_t stream);

/* Cached keys and values back into packed rows, as gdn_cpr_window_attn takes them for a prefill that
 * continues requests: of request n its last cu_seqlens[n + 1] - cu_seqlens[n] positions.
 *   k, v        [total_tokens, h_kv, d] in out_dtype
 *   Rows of a request whose length is negative or less than the rows asked for (GDN_DEVERR_POS), rows
 *   in a tail whose slot lies outside [0, slots) (GDN_DEVERR_SLOT) and rows on a page outside the cache
 *   or the block table (GDN_DEVERR_PAGES) are NaN.  Offsets that do not fit (GDN_DEVERR_CU_SEQLENS): as
 *   above, and the outputs are not valid.
 *   ws: GDN_CPR_ATTN_HEADER_BYTES, 256-byte aligned (the error word, set by every call), or NULL:
 *   what is wrong is skipped as above and not reported, and the call is one kernel            */
gdn_status gdn_cpr_quant_read(const gdn_cpr_quant_cache *cache, int32_t num_seqs,
                              int32_t total_tokens, const int32_t *cu_seqlens,
                              const int32_t *seq_lens, const int32_t *block_table,
                              int32_t max_blocks, const int32_t *slot, gdn_dtype out_dtype, void *k,
                              void *v, void *ws, size_t ws_bytes, gdn_stream_t stream);

/* gdn_cpr_paged_decode over the 8-bit cache: q [N, H_q, d] is the token at position seq_lens[n] - 1,
 * whose key and value have been appended.  Keys and values are what the cache holds them as; windows,
 * first tokens, scale, lse and errors as there.  attn and cache agree in h_kv, d and dtype.
 *   slot        NULL or [N] int32: the requests' tails; one outside [0, slots) sets GDN_DEVERR_SLOT and
 *               gives NaN for a request whose tail holds tokens
 *   A visible key that is not finite gives NaN in its request's rows, a visible value at least in its
 *   column's entries (infinities or NaN); in a block, where all of it reads as NaN, either gives NaN
 *   if any key of the block is visible.  Masked keys of a block may take part with weight 0.
 *   ws: gdn_cpr_quant_decode_workspace_size bytes; its error word is set by every call        */
gdn_status gdn_cpr_quant_decode(const gdn_cpr_attn *attn, const gdn_cpr_quant_cache *cache,
                                int32_t num_seqs, int32_t max_len, const void *q,
                                const int32_t *block_table, int32_t max_blocks,
                                const int32_t *seq_lens, const int32_t *slot, void *out, float *lse,
                                void *ws, size_t ws_bytes, gdn_stream_t stream);
gdn_status gdn_cpr_quant_decode_workspace_size(const gdn_cpr_attn *attn, int32_t num_seqs,
                                               int32_t max_len, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* GDN_CPR_H */
