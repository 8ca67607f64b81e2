"""Cases of the 8-bit cache's operators (gated_deltanet_cpr_gb300.attn) and their plain forms.

The attention layers of a hybrid model keep their keys and values in pages.  Held in 8 bits, with a scale for
each block of tokens and key head, a cache takes half the memory, and a decode step half the bytes:

  append  new keys and values into the cache: every block that they complete is rounded to 8 bits once, from the
          values as they came, and the rows of an unfinished block wait in a tail in the inputs' type; what was
          written is read back, as a prefill does whose queries see what later steps will see
  read    cached keys and values back into packed rows, for prefill attention that continues requests
  decode  attention of one new token per request over such a cache

A block x [block, d] of one head is held as codes c and a scale s; it stands for c s:
  int8  s = max|x| / 127,                         c = x 127 / max|x| to the nearest whole number, ties to even
  e4m3  s = the least power of two 2^e with max|x| <= 448 2^e,  c = x / s to the nearest e4m3 value, ties to even
A block whose largest value lies below 2^-100 is held as zeros (s = 0).

`own` chooses between the plain form (elementary torch operations) and the library's calls.  `exact` gives the
same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------- cases ----
def listed():
    return [
        # the repository's prefill workload (4 x 4096 tokens): prompts into an empty cache, and back
        dict(name="append prefill", op="append", requests=4, old_lo=0, old_hi=0, new_lo=4096, new_hi=4096, hk=8, d=128,
             page=64, block=16, fmt="int8", dtype="bf16"),
        # one decode step of the repository's decode workload: 256 requests, a token each
        dict(name="append decode", op="append", requests=256, old_lo=2048, old_hi=2176, new_lo=1, new_hi=1, hk=8, d=128,
             page=64, block=16, fmt="int8", dtype="bf16"),
        # ragged chunks after earlier ones, small heads, floating codes
        dict(name="append chunks e4m3", op="append", requests=23, old_lo=0, old_hi=9000, new_lo=1, new_hi=1500, hk=4,
             d=64, page=32, block=32, fmt="e4m3", dtype="bf16"),
        # a few short prompts in 32 bits, as in the repository's smallest configurations
        dict(name="append small f32", op="append", requests=5, old_lo=0, old_hi=0, new_lo=20, new_hi=300, hk=2, d=32,
             page=16, block=16, fmt="int8", dtype="f32"),
        # requests of the long-context workload, 64 log-uniform lengths, read whole to be continued
        dict(name="read long", op="read", requests=64, len_lo=128, len_hi=32768, last=0, hk=4, d=128, page=64, block=64,
             fmt="int8", dtype="bf16"),
        # the last keys of a few requests for a sliding-window layer: what counts is the latency
        dict(name="read few e4m3", op="read", requests=4, len_lo=300, len_hi=1100, last=256, hk=2, d=128, page=16,
             block=16, fmt="e4m3", dtype="bf16"),
        # a few short requests: latency of one layer's decode attention
        dict(name="decode few", op="decode", requests=4, len_lo=300, len_hi=1100, hq=16, hk=2, d=128, page=16, block=16,
             window=0, sinks=0, fmt="int8", dtype="bf16"),
        # the decode workload: 256 requests around 2048 tokens, bound by the cache's bytes
        dict(name="decode many", op="decode", requests=256, len_lo=2048, len_hi=2176, hq=32, hk=8, d=128, page=64,
             block=16, window=0, sinks=0, fmt="int8", dtype="bf16"),
        # the same in floating codes and larger blocks
        dict(name="decode many e4m3", op="decode", requests=256, len_lo=2048, len_hi=2176, hq=32, hk=8, d=128, page=64,
             block=64, window=0, sinks=0, fmt="e4m3", dtype="bf16"),
        # few long and ragged requests, small heads: the split over the length carries it
        dict(name="decode long", op="decode", requests=7, len_lo=3000, len_hi=131072, hq=12, hk=4, d=64, page=32,
             block=32, window=0, sinks=0, fmt="int8", dtype="bf16"),
        # 16 query heads to a key head, the widest group that one pass takes
        dict(name="decode wide e4m3", op="decode", requests=33, len_lo=500, len_hi=16384, hq=32, hk=2, d=128, page=128,
             block=128, window=0, sinks=0, fmt="e4m3", dtype="bf16"),
        # sliding-window layer in 32 bits: last 1000 tokens and 4 first ones
        dict(name="decode window f32", op="decode", requests=48, len_lo=200, len_hi=32768, hq=8, hk=4, d=128, page=16,
             block=16, window=1000, sinks=4, fmt="int8", dtype="f32"),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "decode", "decode", "decode"])
    while True:
        page = rng.choice([16, 32, 64, 128, 256])
        c = dict(op=op, requests=_logu(rng, 1, 300), hk=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([32, 64, 128, 128]),
                 page=page, block=rng.choice([b for b in (16, 32, 64, 128) if b <= page]),
                 fmt=rng.choice(["int8", "e4m3"]), dtype=rng.choice(["bf16", "bf16", "f32"]))
        hi = _logu(rng, 1, 100000)
        if op == "append":
            old, hi = rng.choice([0, _logu(rng, 1, 20000)]), min(hi, 20000)
            c.update(old_lo=old // 3, old_hi=old, new_lo=rng.choice([0, 1, hi]), new_hi=rng.choice([1, hi]))
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
            if c["requests"] * (old + c["new_hi"]) * c["hk"] * c["d"] > 3e8 or c["requests"] * c["new_hi"] * c["hk"] * c["d"] > 1.6e7:
                continue
        else:
            c.update(len_lo=rng.choice([0, 1, max(1, hi // 2)]), len_hi=hi)
            if op == "read":
                c["last"] = rng.choice([0, 0, _logu(rng, 1, 8192)])
            else:
                c.update(hq=c["hk"] * rng.choice([1, 2, 3, 4, 5, 8, 12]), window=rng.choice([0, 0, _logu(rng, 1, 8192)]),
                         sinks=rng.choice([0, 1, 4, 16]))
            if c["requests"] * hi * c["hk"] * c["d"] > (1.9e8 if op == "read" else 3e8):
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


# work() has no inputs in hand for the shape of a case: lengths come from a seed of their own, so that every seed
# of a case does the same work on other values
SHAPE_SEED = 20


def _case_lengths(case):
    """(cached before the call, appended, read back at the end) per request."""
    n = case["requests"]
    if case["op"] != "append":
        lens = _lengths(n, case["len_lo"], case["len_hi"], SHAPE_SEED)
        back = np.minimum(lens, case["last"]) if case.get("last") else lens
        return lens, np.zeros_like(lens), back
    old, new = (_lengths(n, case[m + "_lo"], case[m + "_hi"], SHAPE_SEED + k) for k, m in enumerate(("old", "new")))
    # chunks of a prompt begin with a block, so that a call may be repeated: a chunk that completes a block and
    # begins another replaces what the tail held
    old = np.where(new > 1, old // case["block"] * case["block"], old)
    # what is read back: the new tokens' blocks from their first token on
    back = np.where(new > 0, old + new - old // case["block"] * case["block"], 0)
    return old, new, back


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _amax(x):
    """Largest magnitude of every block [..., block, d], in 32 bits."""
    return x.float().abs().amax((-1, -2), keepdim=True)


def _quantise(x, fmt):
    """Codes and scales of blocks x [..., block, d], in 64 bits: the quotients lie next to ties."""
    m = _amax(x).double()
    some = m >= 2.0 ** -100
    m = torch.where(some, m, 1.0)
    if fmt == "int8":
        s = m / 127
        c = torch.where(some, torch.round(x.double() * 127 / m), 0.0).to(torch.int8)
    else:
        f, e = torch.frexp(m / 448)  # m / 448 = f 2^e with f in [1/2, 1); m has 24 bits, so f is 1/2 only where it is exact
        s = torch.ldexp(torch.ones_like(m), torch.where(f == 0.5, e - 1, e))
        c = torch.where(some, x.double() / s, 0.0).float().to(torch.float8_e4m3fn)
    return c, torch.where(some, s, 0.0).float()[..., 0, 0]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    perm = np.random.default_rng(int(seed))
    s = dict(case)
    hk, d, page, B, fmt, dt = case["hk"], case["d"], case["page"], case["block"], case["fmt"], DT[case["dtype"]]
    order = perm.permutation(case["requests"])
    old, new, back = (x[order] for x in _case_lengths(case))
    lens = old + new

    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)

    blocks = -(-lens // page)
    pages, N = int(blocks.sum()) + 3, len(lens)
    ids = perm.permutation(pages)
    table = np.full((N, max(1, int(blocks.max()))), -1, dtype=np.int64)
    for n, at in enumerate(_offsets(blocks)[:-1]):
        table[n, :blocks[n]] = ids[at:at + blocks[n]]
    s["table"], s["lens"], s["cu"], s["max_len"] = ints(table), ints(lens), ints(_offsets(new)), int(lens.max())
    slots = perm.permutation(N + 2)
    s["slots"] = ints(slots[:N])
    s["spare_page"], s["spare_slot"] = int(ids[-1]), int(slots[-1])  # nobody's
    s["cu_back"], s["back"], s["new"] = ints(_offsets(back)), int(back.sum()), int(new.sum())

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    # the blocks that new tokens touch
    s["touched"] = int(np.where(new > 0, -(-lens // B) - old // B, 0).sum())
    for m in ("k", "v"):
        size = torch.exp(0.5 * randn(hk, 1, d))  # channels of a head differ, as they do in a layer's keys and values
        s[m + "_pages"] = torch.empty((pages, hk, page, d), dtype=CODE[fmt], device=dev)
        s[m + "_scale"] = torch.empty((pages, hk, page // B), dtype=torch.float32, device=dev)
        step = max(1, (1 << 26) // (hk * page * d))
        for p in range(0, pages, step):  # piece by piece, for the memory's sake
            x = (randn(min(step, pages - p), hk, page, d) * size).to(dt)
            c, sc = _quantise(x.view(-1, hk, page // B, B, d), fmt)
            s[m + "_pages"][p:p + step].view(torch.uint8).copy_(c.view(torch.uint8).view(-1, hk, page, d))
            s[m + "_scale"][p:p + step] = sc
        s[m + "_tail"] = (randn(N + 2, hk, B, d) * size).to(dt)
        if case["op"] == "append":
            # part of a projection's rows, so tokens are strided
            s[m] = (randn(s["new"], 2 * hk, d) * size.squeeze(1).repeat(2, 1)).to(dt)[:, :hk]
    if case["op"] == "decode":
        s["q"] = randn(N, case["hq"], d).to(dt)
    return s


# --------------------------------------------------------------- the library's calls ----
def _own(s):
    from gated_deltanet_cpr_gb300 import attn

    cache = attn.QuantCache.wrap(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"])
    if s["op"] == "decode":
        return attn.quant_decode(s["q"], cache, s["table"], s["lens"], slots=s["slots"], window=s["window"],
                                 sinks=s["sinks"], max_len=s["max_len"])
    if s["op"] == "append":
        attn.quant_append(s["k"], s["v"], cache, s["table"], s["lens"], s["cu"], slots=s["slots"])
    k, v = attn.quant_read(cache, s["table"], s["lens"], s["cu_back"], s["back"], slots=s["slots"])
    return _with_state(s, k, v)


def _with_state(s, k, v):
    if s["op"] == "read":
        return {"k": k, "v": v}
    return {"k": k, "v": v, **{m: s[m] for m in ("k_scale", "v_scale", "k_tail", "v_tail")}}


# ------------------------------------------------------------------- plain forms ----
def _rows(s, m, n, pos):
    """Rows of request n at positions pos (arrays of the same shape): [..., hk, d] in 32 bits."""
    page, B = s["page"], s["block"]
    lens = s["lens"].long()[n]
    waits = pos >= lens - lens % B
    p = s["table"].long()[n, pos // page]
    p, off = torch.where(waits, 0, p), pos % page
    c = s[m + "_pages"].view(torch.uint8)[p, :, off].view(CODE[s["fmt"]]).float() * s[m + "_scale"][p, :, off // B][..., None]
    t = s[m + "_tail"][s["slots"].long()[n], :, pos % B].float()
    return torch.where(waits[..., None, None], t, c)


def _plain_append(s):
    B, page, dev = s["block"], s["page"], s["k"].device
    lens, cu, slots = s["lens"].long(), s["cu"].long(), s["slots"].long()
    new = cu[1:] - cu[:-1]
    old = lens - new
    per = torch.where(new > 0, (lens + B - 1) // B - old // B, 0)  # touched blocks of every request
    n = torch.repeat_interleave(torch.arange(len(lens), device=dev), per, output_size=s["touched"])
    b = old[n] // B + torch.arange(s["touched"], device=dev) - (per.cumsum(0) - per)[n]
    pos = b[:, None] * B + torch.arange(B, device=dev)[None]
    fresh = (pos >= old[n][:, None]) & (pos < lens[n][:, None])
    at = torch.where(fresh, pos + (cu[:-1] - old)[n][:, None], 0)
    whole = (b + 1) * B <= lens[n]
    # blocks that are not whole go to a page that nobody owns, rows that are not new to a slot of that kind
    p = torch.where(whole, s["table"].long()[n, torch.where(whole, b * B // page, 0)], s["spare_page"])
    j = torch.where(whole, b % (page // B), 0)
    waits = fresh & ~whole[:, None]
    slot = torch.where(waits, slots[n][:, None], s["spare_slot"])
    for m in ("k", "v"):
        x = s[m][at].float()  # [blocks, B, hk, d]
        tail = s[m + "_tail"]
        held = tail[slots[n]].transpose(1, 2).float()
        x = torch.where(fresh[..., None, None], x, held).transpose(1, 2)  # [blocks, hk, B, d]
        c, sc = _quantise(x, s["fmt"])
        pages = s[m + "_pages"].view(torch.uint8).view(-1, s["hk"], page // B, B, s["d"])
        keep = (pages[s["spare_page"], :, 0].clone(), s[m + "_scale"][s["spare_page"], :, 0].clone(), tail[s["spare_slot"]].clone())
        pages[p, :, j] = c.view(torch.uint8)
        s[m + "_scale"][p, :, j] = sc
        tail[slot, :, torch.arange(B, device=dev)[None].expand_as(slot)] = x.transpose(1, 2).to(tail.dtype)
        pages[s["spare_page"], :, 0], s[m + "_scale"][s["spare_page"], :, 0], tail[s["spare_slot"]] = keep


def _plain_read(s):
    lens, cu = s["lens"].long(), s["cu_back"].long()
    n = torch.repeat_interleave(torch.arange(len(lens), device=lens.device), cu[1:] - cu[:-1], output_size=s["back"])
    pos = lens[n] - cu[1:][n] + torch.arange(s["back"], device=lens.device)
    return tuple(_rows(s, m, n, pos).to(DT[s["dtype"]]) for m in ("k", "v"))


def _plain_decode(s):
    q, hk = s["q"].float(), s["hk"]
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
    row = torch.arange(n, device=q.device)[:, None].expand_as(at)
    x = torch.einsum("nhgd,nkhd->nhgk", q.view(n, hk, hq // hk, d), _rows(s, "k", row, at)) / math.sqrt(d)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    l = e.sum(-1, keepdim=True)
    o = torch.einsum("nhgk,nkhd->nhgd", e, _rows(s, "v", row, at)) / torch.where(l > 0, l, 1.0)
    return o.reshape(n, hq, d).to(s["q"].dtype)


def run(state):
    if own:
        return _own(state)
    if state["op"] == "decode":
        return _plain_decode(state)
    if state["op"] == "append":
        _plain_append(state)
    return _with_state(state, *_plain_read(state))


# -------------------------------------------------------------------------- work ----
def work(case):
    hk, d, e, B = case["hk"], case["d"], SIZE[case["dtype"]], case["block"]
    old, new, back = _case_lengths(case)
    lens = old + new
    tail = lens % B
    if case["op"] == "decode":
        w, f = case["window"], np.minimum(case["sinks"], lens)
        seen = lens if not w else np.where(lens <= w, lens, w + np.minimum(f, np.maximum(lens - w, 0)))
        held = np.maximum(seen - tail, 0)
        b = 2 * hk * (int(held.sum()) * (d + 4 / B) + int((seen - held).sum()) * d * e)
        return {"bytes": int(b) + 2 * len(lens) * case["hq"] * d * e, "flops": 4 * int(seen.sum()) * case["hq"] * d}
    # rows read back from 8 bits and from the tails, and written
    held = int(np.maximum(back - tail, 0).sum())
    b = 2 * hk * (held * (d + 4 / B) + (int(back.sum()) - held) * d * e + int(back.sum()) * d * e)
    f = 2 * hk * d * int(back.sum())
    if case["op"] == "append":
        waits = int(np.minimum(new, tail).sum())
        done = int(np.where(new > 0, lens // B - old // B, 0).sum())  # blocks completed
        from_tail = int(np.where((new > 0) & (lens // B > old // B), old % B, 0).sum())
        b += 2 * hk * (int(new.sum()) * d * e + waits * d * e + from_tail * d * e + done * (B * d + 4))
        f += 4 * hk * d * B * done
    return {"bytes": max(1, int(b)), "flops": f}


# ------------------------------------------------------------------------- exact ----
def _exact_block(x, fmt):
    """Values that the blocks x [blocks, hk, B, d] (64 bits) are held as, and their scales."""
    m = x.abs().flatten(2).amax(2)[..., None, None]
    empty = m < 2.0 ** -100
    one = torch.where(empty, 1.0, m)
    if fmt == "int8":
        scale = one / 127
        y = torch.round(x * 127 / one) * scale.float().to(torch.float64)
    else:
        # the least power of two, by comparison: an estimate by logarithm, put right by one either way
        e = torch.ceil(torch.log2(one / 448))
        e = torch.where(one > 448 * torch.exp2(e), e + 1, e)
        e = torch.where(one <= 448 * torch.exp2(e - 1), e - 1, e)
        scale = torch.exp2(e)
        z = x / scale
        # four significant bits, a least step of 2^-9
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
        y = torch.round(z / step) * step * scale
    return torch.where(empty, 0.0, y), torch.where(empty, 0.0, scale)[..., 0, 0]


def exact(case, seed):
    """The outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    D = torch.float64
    hk, d, B, page = case["hk"], case["d"], case["block"], case["page"]
    lens, table, slots, cu, cb = (s[m].tolist() for m in ("lens", "table", "slots", "cu", "cu_back"))
    out = {m: s[m].to(D) for m in ("k_scale", "v_scale", "k_tail", "v_tail")} if case["op"] == "append" else {}

    def rows(m, n, first):
        """Positions first .. lens[n] of request n, after the append: [rows, hk, d]."""
        L = lens[n]
        new = cu[n + 1] - cu[n]
        old, b0 = L - new, first // B
        held = (L // B if new == 0 else old // B) * B  # whole blocks from before
        parts = []
        if held > b0 * B:
            # whole pages first, then the rows wanted
            p = torch.tensor(table[n][b0 * B // page:-(-held // page)], dtype=torch.int64, device="cuda")
            c = s[m + "_pages"].view(torch.uint8)[p].view(CODE[case["fmt"]]).to(torch.float32).to(D)
            c = c.view(len(p), hk, page // B, B, d) * s[m + "_scale"][p].to(D)[..., None, None]
            c = c.view(len(p), hk, page, d).transpose(1, 2).reshape(-1, hk, d)
            start = b0 * B // page * page
            parts.append(c[b0 * B - start:held - start])
        if new == 0:
            parts.append(s[m + "_tail"][slots[n], :, :L - held].to(D).transpose(0, 1))
        else:
            x = torch.cat([s[m + "_tail"][slots[n], :, :old - held].to(D).transpose(0, 1), s[m][cu[n]:cu[n + 1]].to(D)])
            whole = len(x) // B
            y, sc = _exact_block(x[:whole * B].view(whole, B, hk, d).transpose(1, 2), case["fmt"])
            parts.append(y.transpose(1, 2).reshape(-1, hk, d))
            parts.append(x[whole * B:])
            for j in range(whole):
                at = held // B + j
                out[m + "_scale"][table[n][at * B // page], :, at % (page // B)] = sc[j]
            skip = old - held if whole == 0 else 0  # rows that the tail had
            out[m + "_tail"][slots[n], :, skip:len(x) - whole * B] = x[whole * B + skip:].transpose(0, 1)
        return torch.cat(parts)[first - b0 * B:]

    if case["op"] != "decode":
        for m in ("k", "v"):
            out[m] = torch.cat([rows(m, n, lens[n] - (cb[n + 1] - cb[n])) for n in range(len(lens))])
        return out
    w, f = case["window"], case["sinks"]
    o = torch.zeros(s["q"].shape, dtype=D, device="cuda")
    for n, L in enumerate(lens):
        if L == 0:
            continue
        k, v = rows("k", n, 0), rows("v", n, 0)
        if w and L > w:
            j = torch.arange(L, device="cuda")
            j = j[(j < f) | (j >= L - w)]
            k, v = k[j], v[j]
        x = torch.einsum("hgd,khd->hgk", s["q"][n].to(D).view(hk, -1, d), k) * d ** -0.5
        o[n] = torch.einsum("hgk,khd->hgd", torch.softmax(x, -1), v).reshape(-1, d)
    return o
