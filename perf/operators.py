"""Cases of the attention-layer operators (gated_deltanet_cpr_gb300.attn) and their plain forms.

A hybrid model interleaves Gated DeltaNet layers with softmax-attention layers.  The
operators measured here are the ones such a model needs beside the recurrence:

  norm_rope  norms of queries and keys per head with the position rotation in the same pass,
             writing keys and values into a paged cache when one is given; its gradient
  page_map   block tables, slot maps, positions and packed offsets from request lengths
  decode     attention of one new token per request over a paged key-value cache
  attn       attention over packed sequences with a sliding window and a few first tokens that
             stay visible; its gradient

`own` chooses between the plain form (elementary torch operations in 32 bits) and the
library's calls.  `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------------- cases ----
def listed():
    return [
        # prefill of the repository's prefill workload (4 x 4096 tokens): RMS norm with weights,
        # half-layout rotation of half the head, keys and values written to the paged cache
        dict(name="norm_rope prefill", op="norm_rope", tokens=16384, hq=32, hk=8, d=128, rot=64, norm="rms",
             layout="half", weights=True, dtype="bf16", grad="", page=64),
        # one new token for each of a few requests: what counts is the latency
        dict(name="norm_rope decode", op="norm_rope", tokens=4, hq=16, hk=2, d=128, rot=128, norm="rms",
             layout="interleaved", weights=True, dtype="bf16", grad="", page=16),
        # training: the L2 norm that the Gated DeltaNet layers put on their queries and keys
        # (16 heads each, no rotation), forward and backward from gdn_cpr_bwd's fp32 gradients
        dict(name="norm_rope train l2", op="norm_rope", tokens=16384, hq=16, hk=16, d=128, rot=0, norm="l2",
             layout="half", weights=False, dtype="bf16", grad="f32", page=0),
        # one decode step of the repository's decode workload: 256 requests, a token each
        dict(name="page_map decode", op="page_map", requests=256, old_lo=2048, old_hi=2176, new_lo=1, new_hi=1, page=64),
        # a batch of new requests as in the long-context workload: 64 log-uniform lengths
        dict(name="page_map prefill", op="page_map", requests=64, old_lo=0, old_hi=0, new_lo=128, new_hi=32768, page=16),
        # a few short requests: latency of one layer's decode attention
        dict(name="decode few", op="decode", requests=4, len_lo=300, len_hi=1100, hq=16, hk=2, d=128, page=16,
             window=0, sinks=0, dtype="bf16"),
        # the decode workload: 256 requests around 2048 tokens, bound by the cache's bytes
        dict(name="decode many", op="decode", requests=256, len_lo=2048, len_hi=2176, hq=32, hk=8, d=128, page=64,
             window=0, sinks=0, dtype="bf16"),
        # few long and ragged requests, small heads: the split over the length carries it
        dict(name="decode long", op="decode", requests=7, len_lo=3000, len_hi=131072, hq=12, hk=4, d=64, page=32,
             window=0, sinks=0, dtype="bf16"),
        # sliding-window layer in 32 bits: last 1000 tokens and 4 first ones
        dict(name="decode window f32", op="decode", requests=48, len_lo=200, len_hi=32768, hq=8, hk=4, d=128, page=16,
             window=1000, sinks=4, dtype="f32"),
        # prefill of one long sequence through a sliding-window layer
        dict(name="attn prefill long", op="attn", seqs=1, q_lo=32768, q_hi=32768, past=0, hq=16, hk=4, d=128,
             window=4096, sinks=4, dtype="bf16", train=False),
        # training on the trainer workload's packed sequences (lengths in [512, 8192])
        dict(name="attn train packed", op="attn", seqs=8, q_lo=512, q_hi=8192, past=0, hq=16, hk=4, d=128,
             window=2048, sinks=8, dtype="bf16", train=True),
        # short ragged sequences in 32 bits, as in the repository's smallest configurations
        dict(name="attn train small f32", op="attn", seqs=7, q_lo=20, q_hi=300, past=0, hq=4, hk=2, d=64,
             window=100, sinks=3, dtype="f32", train=True),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "page_map", "decode", "decode", "attn", "attn"])
    while True:
        d = rng.choice([32, 64, 128, 128])
        hk = rng.choice([1, 2, 3, 4, 8])
        hq = hk * rng.choice([1, 2, 3, 4, 5, 8])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "norm_rope":
            c = dict(op=op, tokens=_logu(rng, 1, 40000), hq=hq, hk=hk, d=d, rot=rng.choice([0, d // 4, d // 2, d]),
                     norm=rng.choice(["rms", "l2", "none"]), layout=rng.choice(["half", "interleaved"]),
                     weights=rng.random() < 0.5, dtype=dtype, grad=rng.choice(["", dtype, "f32"]),
                     page=rng.choice([16, 32, 64]))
            if c["grad"]:
                c["page"] = 0
        elif op == "page_map":
            lo = _logu(rng, 1, 2000)
            old = rng.choice([0, _logu(rng, 1, 30000)])
            c = dict(op=op, requests=_logu(rng, 1, 3000), old_lo=old // 3, old_hi=old,
                     new_lo=rng.choice([0, 1, lo]), new_hi=lo, page=rng.choice([16, 32, 64, 128]))
            if c["requests"] * c["new_hi"] > 400000:
                continue
        elif op == "decode":
            hi = _logu(rng, 1, 131072)
            c = dict(op=op, requests=_logu(rng, 1, 300), len_lo=rng.choice([0, 1, max(1, hi // 2)]), len_hi=hi, hq=hq,
                     hk=hk, d=d, page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, _logu(rng, 1, 8192)]),
                     sinks=rng.choice([0, 1, 4, 16]), dtype=dtype)
            if c["requests"] * hi * hk * d > 3e8:
                continue
        else:
            hi = _logu(rng, 1, 32768)
            c = dict(op=op, seqs=_logu(rng, 1, 16), q_lo=rng.choice([1, max(1, hi // 4)]), q_hi=hi,
                     past=rng.choice([0, 0, _logu(rng, 1, 4000)]), hq=hq, hk=hk, d=d,
                     window=rng.choice([0, _logu(rng, 1, 8192)]), sinks=rng.choice([0, 1, 4, 16, 70]), dtype=dtype,
                     train=rng.random() < 0.5)
            span = min(hi + c["past"], c["window"] or 1 << 30)
            # what the plain form keeps for every query, head and reachable key has to fit too
            if c["seqs"] * hi * span * hq * (2.5 if c["train"] else 1) * (4 if dtype == "f32" else 1) > 1.2e9:
                continue
        return c


# ------------------------------------------------------------------------ inputs ----
def _lengths(n, lo, hi, seed):
    """n whole numbers in [lo, hi]: log-uniform where the range spans more than twenty-fold."""
    r = np.random.default_rng(seed)
    if hi > 20 * max(lo, 1):
        x = np.exp(r.uniform(np.log(max(lo, 0.5)), np.log(hi + 0.49), n)).round().astype(np.int64)
        return np.clip(x, lo, hi)
    return r.integers(lo, hi + 1, n)


def _case_lengths(case, seed):
    if case["op"] == "page_map":
        n = case["requests"]
        return _lengths(n, case["old_lo"], case["old_hi"], seed), _lengths(n, case["new_lo"], case["new_hi"], seed + 1)
    if case["op"] == "decode":
        return _lengths(case["requests"], case["len_lo"], case["len_hi"], seed)
    q = _lengths(case["seqs"], case["q_lo"], case["q_hi"], seed)
    past = _lengths(case["seqs"], 0, case["past"], seed + 1) if case["past"] else np.zeros_like(q)
    return q, q + past


# work() and exact() have no inputs in hand for the shape of a case: lengths come from a seed of
# their own, so that every seed of a case does the same work on other values
SHAPE_SEED = 20


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def randn(*shape, dtype="f32"):
        return torch.randn(shape, generator=gen, device=dev).to(DT[dtype])

    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)

    s = dict(case)
    if case["op"] == "norm_rope":
        T, hq, hk, d, rot = case["tokens"], case["hq"], case["hk"], case["d"], case["rot"]
        dt = case["dtype"]
        s["q"], s["k"], s["v"] = randn(T, hq, d, dtype=dt), randn(T, hk, d, dtype=dt), randn(T, hk, d, dtype=dt)
        s["wq"] = 1 + 0.1 * randn(d) if case["weights"] else None
        s["wk"] = 1 + 0.1 * randn(d) if case["weights"] else None
        s["cos"] = s["sin"] = s["pos"] = None
        if rot:
            top = 4096
            freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
            ang = torch.tensor(np.arange(top)[:, None] * freq[None], device=dev)
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            s["pos"] = ((torch.arange(T, device=dev) + torch.randint(top, (1,), generator=gen, device=dev)) % top).int()
        if case["page"]:
            pages = -(-T // case["page"]) + 3
            s["k_pages"] = torch.zeros((pages, hk, case["page"], d), dtype=DT[dt], device=dev)
            s["v_pages"] = torch.zeros_like(s["k_pages"])
            order = torch.randperm(pages, generator=gen, device=dev)
            t = torch.arange(T, device=dev)
            s["slots"] = (order[t // case["page"]] * case["page"] + t % case["page"]).int()
        if case["grad"]:
            s["dq"], s["dk"] = randn(T, hq, d, dtype=case["grad"]), randn(T, hk, d, dtype=case["grad"])
    elif case["op"] == "page_map":
        old, new = _case_lengths(case, SHAPE_SEED)
        p = np.random.default_rng(int(seed))
        order = p.permutation(len(old))
        old, new = old[order], new[order]
        s["old"], s["new"], s["total"] = ints(old), ints(new), int(new.sum())
        width = int((-(-(old + new) // case["page"])).max()) + 2
        have = -(-old // case["page"])
        need = int((-(-(old + new) // case["page"]) - have).sum())
        ids = p.permutation(int(have.sum()) + need + 5)
        table = np.full((len(old), width), -1, dtype=np.int64)
        for n, at in enumerate(_offsets(have)[:-1]):
            table[n, :have[n]] = ids[at:at + have[n]]
        s["table"], s["free"] = ints(table), ints(ids[int(have.sum()):])
    elif case["op"] == "decode":
        lens = np.random.default_rng(int(seed)).permutation(_case_lengths(case, SHAPE_SEED))
        hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
        blocks = -(-lens // page)
        pages = int(blocks.sum()) + 3
        s["q"] = randn(len(lens), hq, d, dtype=case["dtype"])
        s["k_pages"] = randn(pages, hk, page, d, dtype=case["dtype"])
        s["v_pages"] = randn(pages, hk, page, d, dtype=case["dtype"])
        ids = np.random.default_rng(int(seed) + 1).permutation(pages)
        table = np.zeros((len(lens), max(1, int(blocks.max()))), dtype=np.int64)
        for n, at in enumerate(_offsets(blocks)[:-1]):
            table[n, :blocks[n]] = ids[at:at + blocks[n]]
        s["table"], s["lens"], s["max_len"] = ints(table), ints(lens), int(lens.max())
    else:
        ql, kl = _case_lengths(case, SHAPE_SEED)
        order = np.random.default_rng(int(seed)).permutation(len(ql))
        ql, kl = ql[order], kl[order]
        hq, hk, d, dt = case["hq"], case["hk"], case["d"], case["dtype"]
        s["cu_q"], s["cu_k"], s["ql"], s["kl"] = ints(_offsets(ql)), ints(_offsets(kl)), ints(ql), ints(kl)
        s["n_q"], s["n_k"], s["longest"] = int(ql.sum()), int(kl.sum()), int(kl.max())
        s["blocks"] = int((-(-ql // _block(case))).sum())
        s["q"] = randn(s["n_q"], hq, d, dtype=dt)
        s["k"], s["v"] = randn(s["n_k"], hk, d, dtype=dt), randn(s["n_k"], hk, d, dtype=dt)
        if case["train"]:
            s["dout"] = randn(s["n_q"], hq, d, dtype=dt)
    return s


# --------------------------------------------------------------- the library's calls ----
def _own(s):
    from gated_deltanet_cpr_gb300 import attn

    if s["op"] == "norm_rope":
        kw = dict(norm=s["norm"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS, cos=s["cos"], sin=s["sin"],
                  positions=s["pos"], layout=s["layout"])
        if s["page"]:
            cache = attn.PagedCache.wrap(s["k_pages"], s["v_pages"])
            q, k = attn.qk_norm_rope(s["q"], s["k"], s["v"], cache=cache, slot_map=s["slots"], **kw)
            return {"q": q, "k": k, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        q, k = attn.qk_norm_rope(s["q"], s["k"], **kw)
        out = {"q": q, "k": k}
        if s["grad"]:
            g = attn.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], **kw)
            out.update(dq=g["dq"], dk=g["dk"])
            if s["wq"] is not None:
                out.update(dwq=g["dq_weight"], dwk=g["dk_weight"])
        return out
    if s["op"] == "page_map":
        m = attn.page_map(s["old"], s["new"], s["free"], s["table"], s["page"], s["total"])
        return {"table": s["table"], **{n: m[n] for n in ("seq_lens", "cu_seqlens", "positions", "slot_map", "pages_used")}}
    if s["op"] == "decode":
        cache = attn.PagedCache.wrap(s["k_pages"], s["v_pages"])
        return attn.paged_decode(s["q"], cache, s["table"], s["lens"], window=s["window"], sinks=s["sinks"],
                                 max_len=s["max_len"])
    kw = dict(cu_seqlens_k=s["cu_k"], window=s["window"], sinks=s["sinks"])
    out, lse = attn.window_attn(s["q"], s["k"], s["v"], s["cu_q"], **kw)
    if not s["train"]:
        return {"out": out, "lse": lse}
    g = attn.window_attn_bwd(s["q"], s["k"], s["v"], out, lse, s["dout"], s["cu_q"], **kw)
    return {"out": out, "lse": lse, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}


# ------------------------------------------------------------------- plain forms ----
def _rotate(y, s, sign):
    """Rotates the first rot entries of every head by sign * the position's angles."""
    rot = s["rot"]
    if not rot:
        return y
    cos, sin = s["cos"][s["pos"].long()][:, None], sign * s["sin"][s["pos"].long()][:, None]
    head, rest = y[..., :rot], y[..., rot:]
    if s["layout"] == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _inverse_norm(x, norm):
    if norm == "none":
        return torch.ones_like(x[..., :1])
    sq = (x * x).mean(-1, keepdim=True) if norm == "rms" else (x * x).sum(-1, keepdim=True)
    return torch.rsqrt(sq + EPS)


def _norm_rope(x, w, s):
    x = x.float()
    y = x * _inverse_norm(x, s["norm"])
    return _rotate(y if w is None else y * w, s, 1.0)


def _norm_rope_grad(x, w, dy, s):
    """dx and dw of y = rotate(x r w), r = (c sum x^2 + eps)^(-1/2)."""
    x, g = x.float(), _rotate(dy.float(), s, -1.0)
    r = _inverse_norm(x, s["norm"])
    dw = None if w is None else (g * x * r).sum((0, 1))
    g = g if w is None else g * w
    c = {"rms": 1.0 / x.shape[-1], "l2": 1.0, "none": 0.0}[s["norm"]]
    return r * g - (c * r * r * r * (g * x).sum(-1, keepdim=True)) * x, dw


def _plain_norm_rope(s):
    dt = DT[s["dtype"]]
    q, k = _norm_rope(s["q"], s["wq"], s).to(dt), _norm_rope(s["k"], s["wk"], s).to(dt)
    out = {"q": q, "k": k}
    if s["page"]:
        page, off = s["slots"].long() // s["page"], s["slots"].long() % s["page"]
        s["k_pages"][page, :, off] = k
        s["v_pages"][page, :, off] = s["v"]
        out.update(k_pages=s["k_pages"], v_pages=s["v_pages"])
    if s["grad"]:
        dq, dwq = _norm_rope_grad(s["q"], s["wq"], s["dq"], s)
        dk, dwk = _norm_rope_grad(s["k"], s["wk"], s["dk"], s)
        out.update(dq=dq.to(dt), dk=dk.to(dt))
        if dwq is not None:
            out.update(dwq=dwq, dwk=dwk)
    return out


def _plain_page_map(s):
    page, table = s["page"], s["table"]
    old, new = s["old"].long(), s["new"].long()
    lens = old + new
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    have, want = (old + page - 1) // page, (lens + page - 1) // page
    first = torch.nn.functional.pad((want - have).cumsum(0), (1, 0))  # of the free list, for every request
    col = torch.arange(table.shape[1], device=table.device)[None]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (first[:-1, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][at], table))
    t = torch.arange(s["total"], device=table.device)
    n = torch.searchsorted(cu, t, right=True) - 1
    pos = old[n] + t - cu[n]
    slots = table[n, pos // page].long() * page + pos % page
    return {"table": table, "seq_lens": lens.int(), "cu_seqlens": cu.int(), "positions": pos.int(),
            "slot_map": slots.int(), "pages_used": first[-1:].int()}


def _plain_decode(s):
    q, hk, page = s["q"].float(), s["hk"], s["page"]
    n, hq, d = q.shape
    lens = s["lens"].long()[:, None]
    if s["window"] and s["window"] + s["sinks"] < s["max_len"]:
        # the first tokens and the last ones; a first token that the window shows too counts once
        last = lens - s["window"] + torch.arange(s["window"], device=q.device)[None]
        head = torch.arange(s["sinks"], device=q.device)[None].expand(n, -1)
        at = torch.cat([head, last], 1)
        seen = torch.cat([head < lens - s["window"], last >= 0], 1) & (at < lens)
    else:
        at = torch.arange(s["max_len"], device=q.device)[None].expand(n, -1)
        seen = at < lens
        if s["window"]:
            seen = seen & ((at >= lens - s["window"]) | (at < s["sinks"]))
    at = torch.where(seen, at, 0)
    pages = torch.where(seen, s["table"].long().gather(1, at // page), 0)
    k = s["k_pages"][pages, :, at % page].float()  # [n, keys, hk, d]
    v = torch.where(seen[:, :, None, None], s["v_pages"][pages, :, at % page].float(), 0)
    x = torch.einsum("nhgd,nkhd->nhgk", q.view(n, hk, hq // hk, d), k) / math.sqrt(d)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    l = e.sum(-1, keepdim=True)
    o = torch.einsum("nhgk,nkhd->nhgd", e, v) / torch.where(l > 0, l, 1.0)
    return o.reshape(n, hq, d).to(s["q"].dtype)


def _block(case):
    """Query rows of one block of the plain attention."""
    return 256 if case["q_hi"] > 512 else 32


def _plain_attn(s):
    """Blocks of queries against the keys that their windows reach, plus the first keys."""
    hk, d, B = s["hk"], s["d"], _block(s)
    g, dev = s["hq"] // hk, s["q"].device
    ql, kl, cu_q, cu_k = s["ql"].long(), s["kl"].long(), s["cu_q"].long(), s["cu_k"].long()
    window = min(s["window"] or s["longest"], s["longest"])
    per = (ql + B - 1) // B
    seq = torch.repeat_interleave(torch.arange(len(per), device=dev), per, output_size=s["blocks"])
    row0 = (torch.arange(s["blocks"], device=dev) - (per.cumsum(0) - per)[seq]) * B
    row = row0[:, None] + torch.arange(B, device=dev)[None]
    pos = row + (kl - ql)[seq][:, None]  # the position of each query among its keys
    live = row < ql[seq][:, None]
    qi = torch.where(live, row + cu_q[seq][:, None], 0)
    near = (row0 + (kl - ql)[seq])[:, None] - window + 1 + torch.arange(window + B - 1, device=dev)[None]
    first = torch.arange(s["sinks"], device=dev)[None].expand(len(seq), -1)
    kp = torch.cat([near, first], 1)  # key positions of each block
    far = pos[:, :, None] - kp[:, None]
    inside = (far >= 0) & (far < window) & (kp >= 0)[:, None]
    inside[:, :, window + B - 1:] = far[:, :, window + B - 1:] >= window  # a first key that the window shows too counts once
    inside &= live[:, :, None]
    inside &= (kp < kl[seq][:, None])[:, None]
    ki = (kp.clamp(min=0).minimum((kl[seq][:, None] - 1).clamp(min=0)) + cu_k[seq][:, None]).clamp(max=s["n_k"] - 1)
    q = s["q"].float()[qi].view(-1, B, hk, g, d)
    k, v = s["k"].float()[ki], s["v"].float()[ki]  # [blocks, keys, hk, d]
    scale = 1 / math.sqrt(d)
    x = torch.einsum("nbhgd,nkhd->nhgbk", q, k).mul_(scale)
    x.masked_fill_(~inside[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(torch.isfinite(m), m, 0.0)).exp_()
    l = p.sum(-1, keepdim=True)
    lse = m + torch.log(l)  # -inf where nothing is visible
    p /= torch.where(l > 0, l, 1.0)
    o = torch.einsum("nhgbk,nkhd->nbhgd", p, v)
    dt = s["q"].dtype
    keep = live.reshape(-1)
    out = o.reshape(-1, s["hq"], d)[keep]
    res = {"out": out.to(dt), "lse": lse[..., 0].permute(0, 3, 1, 2).reshape(-1, s["hq"])[keep]}
    if not s["train"]:
        return res
    do = s["dout"].float()[qi].view(-1, B, hk, g, d) * live[:, :, None, None, None]
    zero = torch.zeros((s["n_k"], hk, d), device=dev)
    dv = zero.index_add(0, ki.reshape(-1), torch.einsum("nhgbk,nbhgd->nkhd", p, do).reshape(-1, hk, d))
    ds = torch.einsum("nbhgd,nkhd->nhgbk", do, v)
    ds -= (do * o).sum(-1).permute(0, 2, 3, 1)[..., None]
    ds *= p
    ds *= scale
    dq = torch.einsum("nhgbk,nkhd->nbhgd", ds, k).reshape(-1, s["hq"], d)[keep]
    dk = zero.index_add(0, ki.reshape(-1), torch.einsum("nhgbk,nbhgd->nkhd", ds, q).reshape(-1, hk, d))
    res.update(dq=dq.to(dt), dk=dk.to(dt), dv=dv.to(dt))
    return res


def run(state):
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "page_map": _plain_page_map, "decode": _plain_decode,
            "attn": _plain_attn}[state["op"]](state)


# -------------------------------------------------------------------------- work ----
def _visible(ql, kl, window, sinks):
    """Query-key pairs that one head of these sequences sees."""
    total = 0
    for a, b in zip(ql.tolist(), kl.tolist()):
        pos = np.arange(b - a, b)
        n = pos + 1
        if window:
            n = np.minimum(n, window) + np.minimum(sinks, np.maximum(n - window, 0))
        total += int(np.maximum(n, 0).sum())
    return total


def work(case):
    if case["op"] == "norm_rope":
        T, hq, hk, d, e = case["tokens"], case["hq"], case["hk"], case["d"], SIZE[case["dtype"]]
        x = T * (hq + hk) * d
        b = 2 * x * e + (T * case["rot"] * 4 if case["rot"] else 0)
        f = x * 8
        if case["page"]:
            b += T * hk * d * e * 3  # keys to the cache, values read and written
        if case["grad"]:
            b += x * SIZE[case["grad"]] + x * e
            f += x * 16
        return {"bytes": b, "flops": f}
    if case["op"] == "page_map":
        old, new = _case_lengths(case, SHAPE_SEED)
        fresh = int((-(-(old + new) // case["page"]) - -(-old // case["page"])).sum())
        return {"bytes": 4 * (8 * len(old) + 2 * fresh + 2 * int(new.sum())), "flops": 10 * int(new.sum())}
    e = SIZE[case["dtype"]]
    if case["op"] == "decode":
        lens = _case_lengths(case, SHAPE_SEED)
        pairs = _visible((lens > 0).astype(np.int64), lens, case["window"], case["sinks"])
        qo = 2 * len(lens) * case["hq"] * case["d"] * e
        return {"bytes": qo + 2 * pairs * case["hk"] * case["d"] * e, "flops": 4 * pairs * case["hq"] * case["d"]}
    ql, kl = _case_lengths(case, SHAPE_SEED)
    pairs = _visible(ql, kl, case["window"], case["sinks"])
    nq, nk = int(ql.sum()) * case["hq"] * case["d"] * e, int(kl.sum()) * case["hk"] * case["d"] * e
    b = 2 * nq + 2 * nk + 4 * int(ql.sum()) * case["hq"]
    f = 4 * pairs * case["hq"] * case["d"]
    if case["train"]:
        b += 2 * nq + 2 * nk
        f = f // 4 * 14
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------- exact ----
def exact(case, seed):
    """The outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "page_map":
        return None
    d = case["d"]
    D = torch.float64
    if case["op"] == "norm_rope":
        out = {}
        T, rot = case["tokens"], case["rot"]
        # the rotation as a d x d matrix per token, in pieces of tokens
        if rot:
            i = torch.arange(rot // 2, device="cuda")
            a, b = (i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            ws = torch.ones(d, dtype=D, device="cuda") if w is None else w.to(D)
            y, dx, dw = [], [], torch.zeros(d, dtype=D, device="cuda")
            for t0 in range(0, T, 4096):
                t = slice(t0, min(T, t0 + 4096))
                x = s[name][t].to(D)
                if case["norm"] == "none":
                    r = torch.ones_like(x[..., 0])
                else:
                    r = (x.pow(2).sum(-1) * (1.0 / d if case["norm"] == "rms" else 1.0) + EPS).pow(-0.5)
                z = x * r[..., None] * ws
                u = z.clone()
                if rot:
                    c, sn = s["cos"].to(D)[s["pos"][t].long()][:, None], s["sin"].to(D)[s["pos"][t].long()][:, None]
                    u[..., a], u[..., b] = z[..., a] * c - z[..., b] * sn, z[..., a] * sn + z[..., b] * c
                y.append(u)
                if case["grad"]:
                    gy = s["d" + name][t].to(D)
                    g = gy.clone()
                    if rot:
                        g[..., a], g[..., b] = gy[..., a] * c + gy[..., b] * sn, gy[..., b] * c - gy[..., a] * sn
                    dw += (g * x * r[..., None]).sum((0, 1))
                    g = g * ws
                    n = {"rms": 1.0 / d, "l2": 1.0, "none": 0.0}[case["norm"]]
                    dx.append(g * r[..., None] - x * (n * r.pow(3) * (g * x).sum(-1))[..., None])
            out[name] = torch.cat(y)
            if case["grad"]:
                out["d" + name] = torch.cat(dx)
                if w is not None:
                    out["dw" + name] = dw
        if case["page"]:
            for name, val in (("k_pages", out["k"]), ("v_pages", s["v"].to(D))):
                flat = torch.zeros_like(s[name], dtype=D).transpose(1, 2).reshape(-1, case["hk"], d)
                flat[s["slots"].long()] = val
                out[name] = flat.view(-1, case["page"], case["hk"], d).transpose(1, 2).contiguous()
        return out
    g = case["hq"] // case["hk"]

    def softmax_rows(x, seen):
        x = torch.where(seen, x, -math.inf)
        lse = torch.logsumexp(x, -1)
        p = torch.where(seen, torch.exp(x - torch.where(lse.isfinite(), lse, 0.0)[..., None]), 0.0)
        return p, lse

    if case["op"] == "decode":
        out = torch.zeros(s["q"].shape, dtype=D, device="cuda")
        for n, L in enumerate(s["lens"].tolist()):
            if L == 0:
                continue
            ids = s["table"][n, :-(-L // case["page"])].long()
            k = s["k_pages"][ids].transpose(1, 2).reshape(-1, case["hk"], d)[:L].to(D)
            v = s["v_pages"][ids].transpose(1, 2).reshape(-1, case["hk"], d)[:L].to(D)
            j = torch.arange(L, device="cuda")
            seen = (j < case["sinks"]) | (L - 1 - j < case["window"]) if case["window"] else j >= 0
            x = torch.einsum("hgd,khd->hgk", s["q"][n].to(D).view(case["hk"], g, d), k) / math.sqrt(d)
            p, _ = softmax_rows(x, seen)
            out[n] = torch.einsum("hgk,khd->hgd", p, v).reshape(-1, d)
        return out
    if work(case)["flops"] > 1.7e12:
        return None
    hq = case["hq"]
    out = torch.zeros(s["q"].shape, dtype=D, device="cuda")
    lse = torch.full((s["n_q"], hq), -math.inf, dtype=D, device="cuda")
    grads = {"dq": torch.zeros_like(out), "dk": torch.zeros(s["k"].shape, dtype=D, device="cuda"),
             "dv": torch.zeros(s["v"].shape, dtype=D, device="cuda")}
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for n in range(len(cq) - 1):
        Lq, Lk = cq[n + 1] - cq[n], ck[n + 1] - ck[n]
        for r0 in range(0, Lq, 1024):
            rows = torch.arange(r0, min(Lq, r0 + 1024), device="cuda")
            pos = rows + Lk - Lq
            lo = max(0, int(pos[0]) - case["window"] + 1) if case["window"] else 0
            cols = torch.arange(0, max(0, int(pos[-1]) + 1), device="cuda")
            cols = cols[(cols >= lo) | (cols < case["sinks"])]
            if not len(cols):
                continue
            dist = pos[:, None] - cols[None]
            seen = dist >= 0
            if case["window"]:
                seen &= (dist < case["window"]) | (cols < case["sinks"])[None]
            q = s["q"][cq[n] + rows].to(D).transpose(0, 1)
            k, v = (s[m][ck[n] + cols].to(D).transpose(0, 1).repeat_interleave(g, 0) for m in ("k", "v"))
            p, e = softmax_rows(q @ k.transpose(1, 2) / math.sqrt(d), seen[None])
            o = p @ v
            out[cq[n] + rows], lse[cq[n] + rows] = o.transpose(0, 1), e.transpose(0, 1)
            if case["train"]:
                do = s["dout"][cq[n] + rows].to(D).transpose(0, 1)
                ds = p * (do @ v.transpose(1, 2) - (do * o).sum(-1, keepdim=True)) / math.sqrt(d)
                grads["dq"][cq[n] + rows] = (ds @ k).transpose(0, 1)
                for m, y in (("dk", ds.transpose(1, 2) @ q), ("dv", p.transpose(1, 2) @ do)):
                    grads[m][ck[n] + cols] += y.view(case["hk"], g, len(cols), d).sum(1).transpose(0, 1)
    return {"out": out, "lse": lse, **(grads if case["train"] else {})}
