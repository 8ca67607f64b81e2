"""Attention-layer operators for hybrid models, beside the recurrence in api.py: norms and
rotation of queries and keys, the paged cache's bookkeeping, decode attention over it, and
sliding-window attention with its gradient.  A thin binding like api.py: tensors supply memory
and the current stream, every step runs in the kernels of libgdn_cpr.so, and a refused call
raises api.GdnError.  What only the device can see (a length past max_len, a page outside the cache,
a cu_seqlens table that does not fit) is in the error word of the workspace: pass `ws`
(api.alloc_workspace) and read api.device_error(ws); a call that makes its own workspace does not
keep it.  Shapes, masks and errors: include/gdn_cpr.h.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import api
from .api import GdnError, _dt

NORMS = {"none": 0, "rms": 1, "l2": 2}
LAYOUTS = {"half": 0, "interleaved": 1}
HEADER_BYTES = 256


class NormRopeStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "h_q", "h_k", "d", "rot", "table_rows")] + [
        ("norm", ctypes.c_int), ("layout", ctypes.c_int), ("eps", ctypes.c_float), ("in_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64)]


class AttnStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("h_q", "h_kv", "d", "window", "sinks")] + [
        ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class PagedCache:
    """Key-value cache in pages: k, v [pages, H_kv, page_size, d]."""

    def __init__(self, pages, page_size, h_kv, d, dtype=torch.bfloat16, device="cuda"):
        self._set(torch.zeros((pages, h_kv, page_size, d), dtype=dtype, device=device),
                  torch.zeros((pages, h_kv, page_size, d), dtype=dtype, device=device))

    @classmethod
    def wrap(cls, k, v):
        """A cache over existing page tensors."""
        c = cls.__new__(cls)
        c._set(k, v)
        return c

    def _set(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v pages are [pages, H_kv, page_size, d], alike in shape and dtype")
        self.k, self.v = k, v
        self.pages, self.h_kv, self.page_size, self.d = k.shape

    def pointers(self):
        k, v = self.k, self.v
        return _want(k, v.shape, v.dtype, "k pages"), _want(v, k.shape, k.dtype, "v pages")


def rope_tables(rows, rot, base=10000.0, scale=1.0, device="cuda"):
    """cos and sin [rows, rot / 2] fp32 of the angles (p / scale) base^(-2 i / rot), formed in 64
    bits.  scale > 1 compresses positions for contexts longer than the model was trained on."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] / scale * freq[None]
    return ang.cos().float().to(device), ang.sin().float().to(device)


# The calls below run once or more per layer of a decode step, so the wrappers keep their own cost
# low: one check per tensor that the caller gives, the raw stream handle, one allocation where several results
# go together; descriptions of shapes and their workspace sizes are kept by their values.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _check(fn, rc):
    if rc:
        raise GdnError(fn, rc)


def _want(x, shape, dtype, name):
    """Pointer of a contiguous GPU tensor of that shape and dtype."""
    if x.dtype is not dtype or x.shape != shape or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name} is {x.dtype} {tuple(x.shape)} on {x.device}"
                         f"{'' if x.is_contiguous() else ', not contiguous'}; expected {dtype} {tuple(shape)} on the GPU")
    return x.data_ptr()


def _opt(x, shape, dtype, name):
    return None if x is None else _want(x, shape, dtype, name)


def _clip(x):
    """A window, a count of first tokens or a bound on lengths, in 32 bits: lengths have no more, so anything
    past them means the same; negative ones stay so, for the library to refuse."""
    return max(-1, min(int(x), 2 ** 31 - 1))


def _rows(x, heads, d, name):
    """(pointer, token stride) of [T, heads, d] whose heads are dense; tokens may be strided."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or not x.is_cuda:
        raise ValueError(f"{name} is {tuple(x.shape)} on {x.device}, expected [T, {heads}, {d}] on the GPU")
    tokens, head, entry = x.stride()
    if (entry != 1 or (head != d and heads > 1)) and x.numel():
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return x.data_ptr(), (tokens if shape[0] > 1 else heads * d)


def _bytes(fn, *args):
    n = ctypes.c_size_t(0)
    _check(fn, getattr(api.load(), fn)(*args, ctypes.byref(n)))
    return n.value


def _workspace(x, nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device=x.device)


@functools.lru_cache(maxsize=1024)
def _norm_rope_desc(T, hq, hk, d, rot, rows, norm, layout, eps, in_dtype, out_dtype, grad_dtype, qs, ks, vs):
    return NormRopeStruct(T, hq, hk, d, rot, rows, NORMS[norm], LAYOUTS[layout], eps, _dt(in_dtype), _dt(out_dtype),
                          _dt(grad_dtype), qs, ks, vs)


def _norm_rope_struct(q, k, v, norm, eps, cos, sin, positions, layout, out_dtype, grad_dtype):
    T, hq, d = q.shape
    hk = k.shape[1]
    if k.shape[0] != T or k.dtype != q.dtype or (v is not None and v.dtype != q.dtype):
        raise ValueError("q, k and v have the same tokens and dtype")
    rot = rows = 0
    cp = sp = pp = None
    if cos is not None:
        rot, rows = 2 * cos.shape[1], cos.shape[0]
        cp, sp = _want(cos, cos.shape, torch.float32, "cos"), _want(sin, cos.shape, torch.float32, "sin")
        pp = _want(positions, (T,), torch.int32, "positions")
    qp, qs = _rows(q, hq, d, "q")
    kp, ks = _rows(k, hk, d, "k")
    vp, vs = (None, hk * d) if v is None else _rows(v, hk, d, "v")
    if v is not None and v.shape[0] != T:
        raise ValueError("q, k and v have the same tokens and dtype")
    return _norm_rope_desc(T, hq, hk, d, rot, rows, norm, layout, eps, q.dtype, out_dtype, grad_dtype, qs, ks, vs), \
        qp, kp, vp, cp, sp, pp


def qk_norm_rope(q, k, v=None, *, norm="rms", q_weight=None, k_weight=None, eps=1e-6, cos=None, sin=None,
                 positions=None, layout="half", out_dtype=None, cache: PagedCache | None = None, slot_map=None,
                 want_q=True, want_k=True, q_out=None, k_out=None):
    """gdn_cpr_qk_norm_rope: norms of q [T, Hq, d] and k [T, Hk, d] per head and the rotation by
    cos, sin [rows, rot / 2] at positions [T].  With a cache, k's results and v go to the cache
    at slot_map [T] as well.  Returns (q_out, k_out); want_q / want_k leave one out."""
    od = out_dtype or (cache.k.dtype if cache is not None else q.dtype)
    st, qp, kp, vp, cp, sp, pp = _norm_rope_struct(q, k, v, norm, eps, cos, sin, positions, layout, od, od)
    T, hq, hk, d = st.tokens, st.h_q, st.h_k, st.d
    if q_out is not None:
        qo = _want(q_out, (T, hq, d), od, "q_out")
    else:
        q_out = torch.empty((T, hq, d), dtype=od, device=q.device) if want_q else None
        qo = q_out.data_ptr() if want_q else None
    if k_out is not None:
        ko = _want(k_out, (T, hk, d), od, "k_out")
    else:
        k_out = torch.empty((T, hk, d), dtype=od, device=q.device) if want_k else None
        ko = k_out.data_ptr() if want_k else None
    kc = vc = slots = None
    pages = page = 0
    if cache is not None:
        if cache.h_kv != hk or cache.d != d or cache.k.dtype != od or v is None:
            raise ValueError("the cache holds heads, size and dtype of k_out, and needs v")
        (kc, vc), pages, page = cache.pointers(), cache.pages, cache.page_size
        slots = _want(slot_map, (T,), torch.int32, "slot_map")
    _check("gdn_cpr_qk_norm_rope", api.load().gdn_cpr_qk_norm_rope(
        ctypes.byref(st), qp, kp, vp, _opt(q_weight, (d,), torch.float32, "q_weight"),
        _opt(k_weight, (d,), torch.float32, "k_weight"), cp, sp, pp, qo, ko, kc, vc, pages, page,
        slots, _raw_stream(q.device.index)))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, dq_out, dk_out, *, norm="rms", q_weight=None, k_weight=None, eps=1e-6, cos=None, sin=None,
                     positions=None, layout="half", ws=None):
    """gdn_cpr_qk_norm_rope_bwd.  Returns dict dq, dk (q's dtype) and, when a weight is given,
    dq_weight, dk_weight [d] fp32."""
    gd = dq_out.dtype
    st, qp, kp, _, cp, sp, pp = _norm_rope_struct(q, k, None, norm, eps, cos, sin, positions, layout, q.dtype, gd)
    T, hq, hk, d = st.tokens, st.h_q, st.h_k, st.d
    dev = q.device
    dq, dk = torch.empty((T, hq, d), dtype=q.dtype, device=dev), torch.empty((T, hk, d), dtype=q.dtype, device=dev)
    out = dict(dq=dq, dk=dk, dq_weight=None, dk_weight=None)
    dwq = dwk = wp = None
    nbytes = 0
    if q_weight is not None or k_weight is not None:
        out["dq_weight"], out["dk_weight"] = torch.empty((2, d), dtype=torch.float32, device=dev).unbind()
        dwq, dwk = out["dq_weight"].data_ptr(), out["dk_weight"].data_ptr()
        if ws is None:
            ws = _workspace(q, _bytes("gdn_cpr_qk_norm_rope_workspace_size", ctypes.byref(st)))
        wp, nbytes = ws.data_ptr(), ws.numel()
    _check("gdn_cpr_qk_norm_rope_bwd", api.load().gdn_cpr_qk_norm_rope_bwd(
        ctypes.byref(st), qp, kp, _opt(q_weight, (d,), torch.float32, "q_weight"),
        _opt(k_weight, (d,), torch.float32, "k_weight"), cp, sp, pp, _want(dq_out, (T, hq, d), gd, "dq_out"),
        _want(dk_out, (T, hk, d), gd, "dk_out"), dq.data_ptr(), dk.data_ptr(), dwq, dwk, wp, nbytes,
        _raw_stream(dev.index)))
    return out


def page_map(lens, new_lens, free_pages, block_table, page_size, total_tokens):
    """gdn_cpr_page_map: extends block_table [N, max_blocks] (in place) for new_lens [N] tokens
    after lens [N] cached ones with pages from the front of free_pages.  Returns dict seq_lens,
    cu_seqlens, positions, slot_map, pages_used, and ws, whose error word says what was wrong
    (api.device_error)."""
    N, T = lens.numel(), int(total_tokens)
    if not 0 <= T < 2 ** 31:
        raise ValueError(f"total_tokens is {T}: not a count that fits 32 bits")
    if page_size >= 2 ** 31:
        page_size = -1
    i32 = torch.int32
    # one allocation: the header, then the results, positions and slots on 16-byte boundaries
    pad = -T % 4
    buf = torch.empty(HEADER_BYTES // 4 + 2 * (T + pad) + 2 * N + 2, dtype=i32, device=lens.device)
    if pad:
        ws, pos, _, slots, _, seq, cu, used = buf.split_with_sizes([HEADER_BYTES // 4, T, pad, T, pad, N, N + 1, 1])
    else:
        ws, pos, slots, seq, cu, used = buf.split_with_sizes([HEADER_BYTES // 4, T, T, N, N + 1, 1])
    at = buf.data_ptr()
    a_pos = at + HEADER_BYTES
    a_slots = a_pos + 4 * (T + pad)
    a_seq = a_slots + 4 * (T + pad)
    if block_table.dim() != 2 or block_table.shape[0] != N:
        raise ValueError("block_table is [N, max_blocks]")
    _check("gdn_cpr_page_map", api.load().gdn_cpr_page_map(
        N, T, page_size, block_table.shape[1], free_pages.numel(), _want(lens, (N,), i32, "lens"),
        _want(new_lens, (N,), i32, "new_lens"), _want(free_pages, free_pages.shape, i32, "free_pages"),
        _want(block_table, block_table.shape, i32, "block_table"), a_seq, a_seq + 4 * N, a_pos, a_slots,
        a_seq + 8 * N + 4, at, HEADER_BYTES, _raw_stream(lens.device.index)))
    return dict(seq_lens=seq, cu_seqlens=cu, positions=pos, slot_map=slots, pages_used=used, ws=ws)


@functools.lru_cache(maxsize=1024)
def _attn_struct(hq, hkv, d, window, sinks, scale, dtype):
    return AttnStruct(hq, hkv, d, _clip(window), _clip(sinks), scale or 0.0, _dt(dtype))


@functools.lru_cache(maxsize=4096)
def _attn_bytes(fn, hq, hkv, d, window, sinks, scale, dtype, *args):
    return _bytes(fn, ctypes.byref(_attn_struct(hq, hkv, d, window, sinks, scale, dtype)), *args)


def paged_decode(q, cache: PagedCache, block_table, seq_lens, *, window=0, sinks=0, scale=None, max_len=None, out=None,
                 want_lse=False, ws=None):
    """gdn_cpr_paged_decode: attention of one token per request, q [N, Hq, d], over the cache's
    first seq_lens[n] tokens.  max_len bounds seq_lens (default: what block_table can hold).
    Returns out [N, Hq, d], or (out, lse) with want_lse."""
    shape, dtype, device = q.shape, q.dtype, q.device
    N, hq, d = shape
    if cache.d != d or cache.k.dtype is not dtype:
        raise ValueError("q and the cache have the same d and dtype")
    table = block_table.shape
    if len(table) != 2 or table[0] != N:
        raise ValueError("block_table is [N, max_blocks]")
    blocks = table[1]
    if max_len is None:
        max_len = blocks * cache.page_size
    if not 0 <= max_len < 2 ** 31:
        max_len = _clip(max_len)
    desc = (hq, cache.h_kv, d, window, sinks, scale, dtype)
    qp = _want(q, shape, dtype, "q")
    if out is None:
        out = torch.empty_like(q)
        op = out.data_ptr()
    else:
        op = _want(out, shape, dtype, "out")
    lse = torch.empty((N, hq), dtype=torch.float32, device=device) if want_lse else None
    if ws is None:
        ws = _workspace(q, _attn_bytes("gdn_cpr_paged_decode_workspace_size", *desc, N, max_len))
    kp, vp = cache.pointers()
    _check("gdn_cpr_paged_decode", api.load().gdn_cpr_paged_decode(
        ctypes.byref(_attn_struct(*desc)), N, max_len, qp, kp, vp, cache.pages, cache.page_size,
        _want(block_table, table, torch.int32, "block_table"), blocks,
        _want(seq_lens, (N,), torch.int32, "seq_lens"), op,
        None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(device.index)))
    return (out, lse) if want_lse else out


def _window_setup(q, k, v, cu_q, cu_k, window, sinks, scale, backward, ws):
    Tq, hq, d = q.shape
    Tk, hkv, _ = k.shape
    N = cu_q.numel() - 1
    cu_k = cu_q if cu_k is None else cu_k
    dtype, shape = q.dtype, (Tk, hkv, d)
    desc = (hq, hkv, d, window, sinks, scale, dtype)
    offsets = _want(cu_q, (N + 1,), torch.int32, "cu_seqlens")
    args = (ctypes.byref(_attn_struct(*desc)), N, Tq, Tk, offsets,
            offsets if cu_k is cu_q else _want(cu_k, (N + 1,), torch.int32, "cu_seqlens_k"),
            _want(q, q.shape, dtype, "q"), _want(k, shape, dtype, "k"), _want(v, shape, dtype, "v"))
    if ws is None:
        ws = _workspace(q, _attn_bytes("gdn_cpr_window_attn_workspace_size", *desc, Tq, int(backward)))
    return args, ws


def window_attn(q, k, v, cu_seqlens, *, cu_seqlens_k=None, window=0, sinks=0, scale=None, out=None, lse=None, ws=None):
    """gdn_cpr_window_attn: causal attention over packed sequences, q [Tq, Hq, d], k, v
    [Tk, Hkv, d]; a query sees the last `window` keys (0: all) and the first `sinks`.
    cu_seqlens_k (default cu_seqlens) gives sequences more keys than queries.  Returns
    (out [Tq, Hq, d], lse [Tq, Hq] fp32)."""
    args, ws = _window_setup(q, k, v, cu_seqlens, cu_seqlens_k, window, sinks, scale, False, ws)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    _check("gdn_cpr_window_attn", api.load().gdn_cpr_window_attn(
        *args, _want(out, q.shape, q.dtype, "out"), _want(lse, q.shape[:2], torch.float32, "lse"), ws.data_ptr(),
        ws.numel(), _raw_stream(q.device.index)))
    return out, lse


def window_attn_bwd(q, k, v, out, lse, dout, cu_seqlens, *, cu_seqlens_k=None, window=0, sinks=0, scale=None, ws=None):
    """gdn_cpr_window_attn_bwd from window_attn's out and lse.  Returns dict dq, dk, dv in q's dtype."""
    args, ws = _window_setup(q, k, v, cu_seqlens, cu_seqlens_k, window, sinks, scale, True, ws)
    g = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
    _check("gdn_cpr_window_attn_bwd", api.load().gdn_cpr_window_attn_bwd(
        *args, _want(out, q.shape, q.dtype, "out"), _want(lse, q.shape[:2], torch.float32, "lse"),
        _want(dout, q.shape, q.dtype, "dout"), g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(),
        ws.data_ptr(), ws.numel(), _raw_stream(q.device.index)))
    return g
