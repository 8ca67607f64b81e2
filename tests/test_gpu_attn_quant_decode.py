"""Decode attention over the 8-bit cache against plain attention in 64 bits over what the cache holds.

Tolerances: attn_ref's, with u = 2^-8 in bf16, for the output's rounding and for the probabilities', which are
f16 (2^-11); q, scaled by a power of two, and the codes are exact there.  In fp32 q, the probabilities and the tail's
rows are sums of two f16, off by 2^-22 at most, and the product of two rests is left out, 2^-22 again: 2^-22
for the probabilities, and 3 * 2^-22 = 12 * 2^-24 of the terms' absolute sum for a score, by which its probability and the
log-sum-exp are off as well.  f16's least step is 2^-24, and p 2^14 (relative to its run's largest, 1 at most) is held: however
small p is, it is off by 2^-25 2^-14 = 2^-39 at least, so that an output whose large probabilities meet values of exactly 0
is off by up to 2^-39 sum |v|."""
import pytest
import torch

import attn_ref as A
from test_gpu_attn_quant_rows import BF, F32, Store, attn, expect, ints, offsets, rows  # noqa: F401

pytestmark = pytest.mark.gpu


def reference(q, k, v, L, dtype, window=0, sinks=0, scale=None):
    """The last token of L over rows k, v."""
    u, more = 2.0 ** -8, 0.0
    if dtype == F32 and L:
        g = q.shape[1] // k.shape[1]
        size = torch.einsum("hgd,khd->hgk", q[0].double().abs().view(-1, g, q.shape[2]), k.double().abs())
        more = 12 * A.EPS * float(size.max()) * (scale or q.shape[2] ** -0.5)
        u = 2.0 ** -22 + more
    r = A.attention(q, k, v, torch.tensor([L - 1]), window, sinks, scale, u=u)
    r["tol"]["lse"] += more
    if L:
        r["tol"]["out"] += 2.0 ** -39 * v.double().abs().sum(0).repeat_interleave(q.shape[1] // k.shape[1], 0)[None]
    return r


def filled(attn, gdn, lens, hk, d, page, block, code, dtype, seed=0):
    s = Store(attn, gdn, lens, hk, d, page, block, code, dtype, seed)
    ks, vs = rows(lens, hk, d, dtype, seed + 1), rows(lens, hk, d, dtype, seed + 2)
    s.append(ks, vs, lens)
    return s, ks, vs


def check(attn, gdn, lens, hq, hk, d, page, block, code, dtype, window=0, sinks=0, scale=None, max_len=None, seed=0):
    s, ks, vs = filled(attn, gdn, lens, hk, d, page, block, code, dtype, seed)
    q = rows([len(lens)], hq, d, dtype, seed + 3)[0]
    ws = gdn.alloc_workspace(64 << 20, "cuda")
    out, lse = attn.quant_decode(q.cuda(), s.cache, s.table, ints(lens), slots=s.slots, window=window, sinks=sinks,
                                 scale=scale, max_len=max_len, want_lse=True, ws=ws)
    assert gdn.device_error(ws) == 0
    for i, L in enumerate(lens):
        r = reference(q[i:i + 1], expect(ks[i], block, code, F32), expect(vs[i], block, code, F32), L, dtype, window, sinks, scale)
        assert A.worst(out[i:i + 1], r["out"], r["tol"]["out"]) <= 1, (i, L)
        assert A.worst(lse[i:i + 1], r["lse"], r["tol"]["lse"]) <= 1, (i, L)
    return s, q, out


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page,block", [(32, 16, 16), (64, 32, 16), (128, 16, 16), (128, 64, 64), (64, 128, 128), (32, 64, 32)])
def test_ragged_lengths(attn, gdn, d, page, block, dtype, code):
    """Empty, single, odd lengths, block, page and run boundaries, several runs."""
    check(attn, gdn, [0, 1, 2, 15, 16, 17, 31, 127, 128, 129, 300, 0, 1031], 8, 2, d, page, block, code, dtype)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (5, 1), (12, 4), (16, 2), (9, 1), (16, 1), (17, 1), (40, 1), (32, 2)])
def test_grouped_heads(attn, gdn, hq, hk, dtype, code):
    check(attn, gdn, [33, 1, 200], hq, hk, 64, 32, 32, code, dtype)
    check(attn, gdn, [130, 257], hq, hk, 128, 64, 16, code, dtype)


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (100, 4), (100, 200), (0, 5), (33, 17), (500, 0),
                                          (5000, 1), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_window_and_first_tokens(attn, gdn, window, sinks, dtype, block):
    check(attn, gdn, [0, 1, 5, 63, 64, 65, 99, 100, 101, 104, 128, 133, 640], 4, 2, 128, 64, block, "int8", dtype, window, sinks)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_and_every_page_size(attn, gdn, dtype):
    """Lengths in each range of the split rule."""
    for page, block in ((16, 16), (32, 16), (64, 32), (128, 128), (256, 64)):
        check(attn, gdn, [2048, 2049, 9000], 4, 1, 64, page, block, "int8", dtype, seed=page)
    check(attn, gdn, [20000, 3], 2, 1, 32, 64, 16, "e4m3", dtype, scale=0.3)


def test_large_and_small_values(attn, gdn):
    """Scores of some hundreds, where the running maximum has to move; queries, keys and values far from 1 in size."""
    for dtype in (BF, F32):
        check(attn, gdn, [500, 64, 1, 77], 4, 2, 64, 16, 16, "int8", dtype, scale=6.0)
        s, ks, vs = filled(attn, gdn, [333, 40], 2, 128, 32, 32, "e4m3", dtype)
        for fq, fk, fv in ((1e20, 1e-20, 1e15), (1e-15, 1e15, 1e-25), (1e-3, 1e3, 1e30)):
            q = (rows([2], 4, 128, dtype, 9)[0].float() * fq).to(dtype)
            k, v = [(x.float() * fk).to(dtype) for x in ks], [(x.float() * fv).to(dtype) for x in vs]
            s.append(k, v, [333, 40])
            out = attn.quant_decode(q.cuda(), s.cache, s.table, ints([333, 40]), slots=s.slots)
            for i, L in enumerate([333, 40]):
                r = reference(q[i:i + 1], expect(k[i], 32, "e4m3", F32), expect(v[i], 32, "e4m3", F32), L, dtype)
                assert A.worst(out[i:i + 1], r["out"], r["tol"]["out"]) <= 1


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_large_row(attn, gdn, dtype):
    """One key and one value far larger than the others: other blocks keep their own scales."""
    lens = [100, 260]
    s = Store(attn, gdn, lens, 1, 64, 16, 16, "int8", dtype)
    ks, vs = rows(lens, 1, 64, dtype, 1), rows(lens, 1, 64, dtype, 2)
    for n, at in ((0, 3), (1, 258)):
        vs[n][at] *= 1e6
        ks[n][at] *= -30
    s.append(ks, vs, lens)
    q = rows([2], 3, 64, dtype, 3)[0]
    out = attn.quant_decode(q.cuda(), s.cache, s.table, ints(lens), slots=s.slots)
    for i, L in enumerate(lens):
        r = reference(q[i:i + 1], expect(ks[i], 16, "int8", F32), expect(vs[i], 16, "int8", F32), L, dtype)
        assert A.worst(out[i:i + 1], r["out"], r["tol"]["out"]) <= 1


@pytest.mark.parametrize("dtype,d,code", [(BF, 128, "int8"), (BF, 64, "e4m3"), (F32, 128, "e4m3"), (BF, 32, "int8")])
def test_batch_pages_and_bounds_do_not_change_bits(attn, gdn, dtype, d, code):
    """More runs than warps beside a long request, the same bits whatever max_len says, alone, and on other pages."""
    lens = [(37 * i) % 211 for i in range(250)] + [3000, 700, 9000, 1]
    s, q, out = check(attn, gdn, lens, 8, 4, d, 16, 16, code, dtype, seed=3)
    n = ints(lens)
    assert torch.equal(out, attn.quant_decode(q.cuda(), s.cache, s.table, n, slots=s.slots, max_len=100000))
    for i in (5, 249, 250, 251, 252):
        one = attn.quant_decode(q[i:i + 1].cuda(), s.cache, s.table[i:i + 1].contiguous(), n[i:i + 1], slots=s.slots[i:i + 1],
                                max_len=lens[i])
        assert torch.equal(one, out[i:i + 1]), i
    few = [7, 250, 251]
    s2 = Store(attn, gdn, [lens[i] for i in few], 4, d, 64, 16, code, dtype, 11)
    ks, vs = rows(lens, 4, d, dtype, 4), rows(lens, 4, d, dtype, 5)
    s2.append([ks[i] for i in few], [vs[i] for i in few], [lens[i] for i in few])
    again = attn.quant_decode(q[few].cuda(), s2.cache, s2.table, ints([lens[i] for i in few]), slots=s2.slots)
    assert torch.equal(again, out[few])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_is_not_visible_changes_nothing(attn, gdn, dtype):
    """Rows past a tail's end, other slots, other pages, other scales, and masked rows of a tail: junk of every kind."""
    lens, block = [200, 37, 64, 130], 32
    s, ks, vs = filled(attn, gdn, lens, 2, 64, 32, block, "int8", dtype)
    q = rows([4], 4, 64, dtype, 7)[0].cuda()
    kw = dict(slots=s.slots, window=3, sinks=1)
    ref = attn.quant_decode(q, s.cache, s.table, ints(lens), **kw), attn.quant_decode(q, s.cache, s.table, ints(lens), slots=s.slots)
    c = s.cache
    mine = set(s.slots.tolist())
    for junk in (float("nan"), float("inf"), -float("inf"), 3e38):
        for t in (c.k_tail, c.v_tail):
            for x in range(c.slots):
                t[x, :, (lens[s.slots.tolist().index(x)] % block if x in mine else 0):] = junk
        for t in (c.k_scale, c.v_scale):
            t[s.free] = junk
            for n, L in enumerate(lens):  # the page whose block is unfinished
                if L % block:
                    t[int(s.table[n, L // 32])] = junk
        assert torch.equal(attn.quant_decode(q, c, s.table, ints(lens), **kw), ref[0])
        assert torch.equal(attn.quant_decode(q, c, s.table, ints(lens), slots=s.slots), ref[1])
    # masked rows of request 0's tail: it holds rows 192 .. 199, of which the window shows the last three
    for t in (c.k_tail, c.v_tail):
        t[int(s.slots[0]), :, :5] = float("nan")
    assert torch.equal(attn.quant_decode(q, c, s.table, ints(lens), **kw), ref[0])


def test_values_that_are_not_finite(attn, gdn):
    """They give NaN in the rows of their request and key head, a value that waits in the tail at least in its own
    column, and nothing changes elsewhere."""
    lens = [100, 90, 40]
    for at, where in ((5, "k"), (5, "v"), (99, "k"), (97, "v")):
        for bad in (float("nan"), float("inf")):
            for dtype in (BF, F32):
                s, ks, vs = filled(attn, gdn, lens, 2, 64, 16, 16, "e4m3", dtype)
                q = rows([3], 4, 64, dtype, 7)[0].cuda()
                ref = attn.quant_decode(q, s.cache, s.table, ints(lens), slots=s.slots)
                (ks if where == "k" else vs)[0][at, 1, 3] = bad
                s.append(ks, vs, lens)
                out = attn.quant_decode(q, s.cache, s.table, ints(lens), slots=s.slots)
                lost = out[0, 2:, 3:4].isfinite().logical_not() if (at, where) == (97, "v") else out[0, 2:].isnan()
                assert lost.all() and torch.equal(out[0, :2], ref[0, :2]) and torch.equal(out[1:], ref[1:])
    q[1, 0, 5] = float("inf")
    out = attn.quant_decode(q, s.cache, s.table, ints(lens), slots=s.slots)
    assert out[1, 0].isnan().all() and torch.equal(out[1, 1:], ref[1, 1:]) and torch.equal(out[2], ref[2])


def test_bad_lengths_slots_and_pages_are_reported(attn, gdn):
    for lens in ([50, 60, 70], [400, 300, 905]):
        s, ks, vs = filled(attn, gdn, lens, 2, 64, 16, 16, "int8", BF)
        q, n = rows([3], 4, 64, BF, 7)[0].cuda(), ints(lens)
        ws = gdn.alloc_workspace(1 << 22, "cuda")
        call = lambda t=s.table, n=n, sl=s.slots: attn.quant_decode(q, s.cache, t, n, slots=sl, max_len=1000, ws=ws)  # noqa: E731
        ref = call().clone()
        assert gdn.device_error(ws) == 0
        for length in (-3, 1001):
            bad = n.clone()
            bad[1] = length
            out = call(n=bad)
            assert gdn.device_error(ws) == 3
            assert out[1].isnan().all() and torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
        for page in (-1, s.cache.pages, 2 ** 31 - 1):
            t = s.table.clone()
            t[2, 1] = page
            out = call(t=t)
            assert gdn.device_error(ws) == 7
            assert out[2].isnan().all() and torch.equal(out[0], ref[0])
        for slot in (-1, s.cache.slots, 2 ** 31 - 1):
            sl = s.slots.clone()
            sl[2] = slot
            out = call(sl=sl)
            assert gdn.device_error(ws) == 2
            assert out[2].isnan().all() and torch.equal(out[:2], ref[:2])
            sl = s.slots.clone()  # not needed where nothing waits in the tail
            sl[0] = slot
            m = n.clone()
            m[0] = 48
            call(n=m, sl=sl)
            assert gdn.device_error(ws) == 0
        out = call(t=s.table[:, :2].contiguous())  # block tables shorter than the lengths
        assert gdn.device_error(ws) == 7 and out.isnan().all()
        assert torch.equal(call(), ref) and gdn.device_error(ws) == 0


def test_workspace_serves_any_length_up_to_its_bound(attn, gdn):
    """Windows whose granules straddle their ends need a run more than their keys alone would."""
    for window, sinks, hk in ((2048, 0, 1), (2033, 17, 1), (4096, 1, 2), (640, 640, 8)):
        for L in (window + sinks + 1, window + sinks + 9, 3 * window + 5):
            check(attn, gdn, [L], 2 * hk, hk, 32, 16, 16, "int8", BF, window, sinks, max_len=L)


def test_offsets_past_32_bits(attn, gdn):
    page, d, hk, block = 256, 128, 8, 128
    pages = 2 ** 32 // (page * d * hk) + 9
    slots = 2 ** 31 // (block * d * hk) + 5
    k, v = (torch.zeros((pages, hk, page, d), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, hk, page // block), device="cuda") for _ in range(2))
    kt, vt = (torch.zeros((slots, hk, block, d), dtype=BF, device="cuda") for _ in range(2))
    c = attn.QuantCache.wrap(k, v, ks, vs, kt, vt)
    x, y, q = rows([600], hk, d, BF, 1)[0], rows([600], hk, d, BF, 2)[0], rows([1], 16, d, BF, 3)[0]
    table, slot = ints([[pages - 1, pages - 3, pages - 2]]), ints([slots - 1])
    attn.quant_append(x.cuda(), y.cuda(), c, table, ints([600]), ints([0, 600]), slots=slot)
    out = attn.quant_decode(q.cuda(), c, table, ints([600]), slots=slot)
    r = reference(q, expect(x, block, "int8", F32), expect(y, block, "int8", F32), 600, BF)
    assert A.worst(out, r["out"], r["tol"]["out"]) <= 1


def test_captured_in_a_graph(attn, gdn):
    """One graph serves growing lengths up to max_len."""
    s, ks, vs = filled(attn, gdn, [500, 400], 2, 128, 16, 16, "int8", BF)
    q = rows([2], 8, 128, BF, 7)[0].cuda()
    ws = gdn.alloc_workspace(8 << 20, "cuda")
    out, live = torch.empty_like(q), ints([500, 400])
    kw = dict(slots=s.slots, max_len=512)
    attn.quant_decode(q, s.cache, s.table, live, ws=ws, out=out, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn.quant_decode(q, s.cache, s.table, live, ws=ws, out=out, **kw)
    for lens in ([500, 400], [0, 16], [256, 128], [500, 0]):
        live.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        assert torch.equal(out, attn.quant_decode(q, s.cache, s.table, live, **kw))


@pytest.mark.parametrize("code,block", [("int8", 16), ("e4m3", 64)])
def test_a_serving_loop(attn, gdn, code, block):
    """page_map, norm and rotation, append and decode, a prompt and then tokens one by one, against plain attention over
    what the cache holds at each step."""
    hq, hk, d, page, lens, steps = 8, 2, 64, 64, [70, 1, 128], 70
    total = [n + steps for n in lens]
    g = torch.Generator().manual_seed(1)
    w = 1 + 0.1 * torch.randn(d, generator=g).cuda()
    cos, sin = attn.rope_tables(256, d)
    text = [torch.randn((n, hq + 2 * hk, d), generator=g).to(BF) for n in total]
    pages = sum(-(-n // page) for n in total)
    c = attn.QuantCache(pages, page, hk, d, 3, code=code, block=block)
    free, table = torch.arange(pages, dtype=torch.int32, device="cuda"), torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    held_k, held_v = [torch.empty(0, hk, d, dtype=BF)] * 3, [torch.empty(0, hk, d, dtype=BF)] * 3
    n, at, new = ints([0, 0, 0]), [0, 0, 0], lens
    for step in range(steps + 1):
        x = torch.cat([t[a:a + m] for t, a, m in zip(text, at, new)]).cuda()
        m = attn.page_map(n, ints(new), free, table, page, sum(new))
        assert gdn.device_error(m["ws"]) == 0
        free, n = free[int(m["pages_used"]):].clone(), m["seq_lens"]
        q, k, v = x.split([hq, hk, hk], 1)
        q, k = attn.qk_norm_rope(q, k, q_weight=w, k_weight=w, cos=cos, sin=sin, positions=m["positions"])
        attn.quant_append(k, v, c, table, n, m["cu_seqlens"])
        held_k = [torch.cat([h, y]) for h, y in zip(held_k, k.cpu().split(new))]
        held_v = [torch.cat([h, y]) for h, y in zip(held_v, v.cpu().split(new))]
        at = [a + b for a, b in zip(at, new)]
        if step:
            o = attn.quant_decode(q, c, table, n, window=90, sinks=2)
            for i in range(3):
                r = reference(q[i:i + 1].cpu(), expect(held_k[i], block, code, F32), expect(held_v[i], block, code, F32),
                              at[i], BF, 90, 2)
                assert A.worst(o[i:i + 1], r["out"], r["tol"]["out"]) <= 1, (step, i)
        new = [1, 1, 1]
