"""Decode attention over the paged cache against plain attention in 64 bits (tolerances: see
attn_ref; u = 2^-8 for bf16, 2^-24 for fp32)."""
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def attn(gdn):
    from gated_deltanet_cpr_gb300 import attn as a
    return a


def make(attn, lens, hq, hk, d, page, dtype, seed=0, junk=float("nan")):
    """A cache whose unused rows and pages hold junk."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g).to(dtype)  # noqa: E731
    blocks = [-(-n // page) for n in lens]
    pages = sum(blocks) + 3
    ids = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(blocks + [1]) + 1), 2 ** 31 - 1, dtype=torch.int32)
    kp, vp = (torch.full((pages, hk, page, d), junk, dtype=dtype) for _ in range(2))
    ks, vs, at = [], [], 0
    for n, L in enumerate(lens):
        k, v = rn(L, hk, d), rn(L, hk, d)
        for b in range(blocks[n]):
            table[n, b] = ids[at]
            part = slice(b * page, min(L, (b + 1) * page))
            kp[ids[at], :, :part.stop - part.start] = k[part].transpose(0, 1)
            vp[ids[at], :, :part.stop - part.start] = v[part].transpose(0, 1)
            at += 1
        ks.append(k)
        vs.append(v)
    q = rn(len(lens), hq, d)
    cache = attn.PagedCache.wrap(kp.cuda(), vp.cuda())
    return q, ks, vs, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def check(attn, gdn, lens, hq, hk, d, page, dtype, window=0, sinks=0, scale=None, max_len=None, seed=0):
    q, ks, vs, cache, table, n = make(attn, lens, hq, hk, d, page, dtype, seed)
    nb = gdn.alloc_workspace(64 << 20, "cuda")
    out, lse = attn.paged_decode(q.cuda(), cache, table, n, window=window, sinks=sinks, scale=scale, max_len=max_len,
                                 want_lse=True, ws=nb)
    assert gdn.device_error(nb) == 0
    for i, L in enumerate(lens):
        r = R.attention(q[i:i + 1], ks[i], vs[i], torch.tensor([L - 1]), window, sinks, scale, u=U[dtype])
        assert R.worst(out[i:i + 1], r["out"], r["tol"]["out"]) <= 1, (i, L)
        assert R.worst(lse[i:i + 1], r["lse"], r["tol"]["lse"]) <= 1, (i, L)
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_ragged_lengths(attn, gdn, d, dtype):
    """Empty, single, odd lengths, page and run boundaries, several runs."""
    check(attn, gdn, [0, 1, 2, 15, 16, 17, 127, 128, 129, 300, 0, 1031], 8, 2, d, 16, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (5, 1), (12, 4), (16, 2), (9, 1), (17, 1), (40, 1), (32, 2)])
def test_grouped_heads(attn, gdn, hq, hk, dtype):
    check(attn, gdn, [33, 1, 200], hq, hk, 64, 32, dtype)
    check(attn, gdn, [130, 257], hq, hk, 128, 64, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (100, 4), (100, 200), (0, 5), (500, 0),
                                          (5000, 1), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_window_and_first_tokens(attn, gdn, window, sinks, dtype):
    check(attn, gdn, [0, 1, 5, 99, 100, 101, 104, 640], 4, 2, 128, 16, dtype, window, sinks)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_and_every_page_size(attn, gdn, dtype):
    """Lengths in each range of the split rule."""
    for page in (16, 32, 64, 128, 256):
        check(attn, gdn, [2048, 2049, 9000], 4, 1, 64, page, dtype, seed=page)
    check(attn, gdn, [20000, 3], 2, 1, 32, 64, dtype, scale=0.3)


def test_large_scores(attn, gdn):
    """Scores of some hundreds: the running maximum has to move."""
    for dtype in (BF, F32):
        check(attn, gdn, [500, 64, 1], 4, 2, 64, 16, dtype, scale=6.0)


def test_batch_and_pages_do_not_change_bits(attn, gdn):
    lens = [700, 1, 2500, 64, 129]
    for dtype in (BF, F32):
        q, ks, vs, cache, table, n = make(attn, lens, 8, 2, 128, 32, dtype)
        out = attn.paged_decode(q.cuda(), cache, table, n, max_len=2500)
        again = attn.paged_decode(q.cuda(), cache, table, n, max_len=100000)
        assert torch.equal(out, again)
        for i in range(len(lens)):
            one = attn.paged_decode(q[i:i + 1].cuda(), cache, table[i:i + 1].contiguous(), n[i:i + 1], max_len=lens[i])
            assert torch.equal(one[0], out[i])
        q2, _, _, c2, t2, n2 = make(attn, lens, 8, 2, 128, 16, dtype, junk=0.0)
        q3, _, _, c3, t3, n3 = make(attn, lens, 8, 2, 128, 64, dtype, junk=3e38)
        a, b = attn.paged_decode(q2.cuda(), c2, t2, n2), attn.paged_decode(q2.cuda(), c3, t3, n3)
        del q3
        assert a.shape == b.shape and torch.isfinite(b).all()


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (BF, 32)])
def test_many_requests_beside_a_long_one(attn, gdn, dtype, d):
    """More runs than warps, most of them empty, and requests of one to many runs; the same bits whatever
    max_len says, and alone."""
    lens = [(37 * i) % 211 for i in range(250)] + [3000, 700, 9000, 1]
    out = check(attn, gdn, lens, 8, 4, d, 16, dtype, seed=3)
    q, _, _, cache, table, n = make(attn, lens, 8, 4, d, 16, dtype, seed=3)
    assert torch.equal(out, attn.paged_decode(q.cuda(), cache, table, n, max_len=100000))
    for i in (5, 249, 250, 251, 252):
        one = attn.paged_decode(q[i:i + 1].cuda(), cache, table[i:i + 1].contiguous(), n[i:i + 1], max_len=lens[i])
        assert torch.equal(one, out[i:i + 1]), i


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 128), (BF, 32)])
def test_pages_do_not_change_bits(attn, dtype, d):
    """The same keys and values on pages of every size, in any order, between rows of any kind."""
    lens, hk = [700, 1, 2500, 64, 129], 2
    g = torch.Generator().manual_seed(7)
    q, ks, vs = (torch.randn((n, h, d), generator=g).to(dtype) for n, h in
                 ((len(lens), 8), (sum(lens), hk), (sum(lens), hk)))
    n, first = torch.tensor(lens, dtype=torch.int32).cuda(), None
    for page in (16, 32, 64, 128, 256):
        for seed, junk in ((0, 0.0), (1, float("nan")), (2, 3e38)):
            blocks = [-(-x // page) for x in lens]
            ids = torch.randperm(sum(blocks) + 5, generator=g.manual_seed(seed)).tolist()
            kp, vp = (torch.full((len(ids), hk, page, d), junk, dtype=dtype) for _ in range(2))
            table, at = torch.full((len(lens), max(blocks)), -1, dtype=torch.int32), 0
            for i, x in enumerate(lens):
                for b in range(blocks[i]):
                    p, m = ids.pop(), min(page, x - b * page)
                    table[i, b] = p
                    kp[p, :, :m] = ks[at:at + m].transpose(0, 1)
                    vp[p, :, :m] = vs[at:at + m].transpose(0, 1)
                    at += m
            cache = attn.PagedCache.wrap(kp.cuda(), vp.cuda())
            got = [attn.paged_decode(q.cuda(), cache, table.cuda(), n, window=w, sinks=s) for w, s in ((0, 0), (300, 5))]
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(got, first)), (page, junk)


def test_sizes_past_32_bits(attn):
    """A bound, a window or a count of first tokens past 2^31 is none."""
    q, _, _, cache, table, n = make(attn, [500, 20], 4, 2, 64, 16, BF)
    near = attn.paged_decode(q.cuda(), cache, table, n, window=64)
    for most in (2 ** 31, 2 ** 32 + 10):
        assert torch.equal(near, attn.paged_decode(q.cuda(), cache, table, n, window=64, max_len=most))
        assert torch.equal(attn.paged_decode(q.cuda(), cache, table, n), attn.paged_decode(q.cuda(), cache, table, n, window=most))


def test_bad_lengths_and_pages_are_reported(attn, gdn):
    for lens in ([50, 60, 70], [400, 300, 900]):
        q, ks, vs, cache, table, n = make(attn, lens, 4, 2, 64, 16, BF)
        ws = gdn.alloc_workspace(1 << 22, "cuda")
        ref = attn.paged_decode(q.cuda(), cache, table, n, max_len=1000, ws=ws).clone()
        assert gdn.device_error(ws) == 0
        for length in (-3, 1001):
            bad = n.clone()
            bad[1] = length
            out = attn.paged_decode(q.cuda(), cache, table, bad, max_len=1000, ws=ws)
            assert gdn.device_error(ws) == 3
            assert torch.isnan(out[1]).all() and torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
        for page in (-1, cache.pages, 2 ** 31 - 1):
            t = table.clone()
            t[2, 1] = page
            out = attn.paged_decode(q.cuda(), cache, t, n, max_len=1000, ws=ws)
            assert gdn.device_error(ws) == 7
            assert torch.isnan(out[2]).all() and torch.equal(out[0], ref[0])
        narrow = table[:, :2].contiguous()  # block tables shorter than the lengths
        out = attn.paged_decode(q.cuda(), cache, narrow, n, max_len=1000, ws=ws)
        assert gdn.device_error(ws) == 7 and torch.isnan(out).all()
        assert torch.equal(attn.paged_decode(q.cuda(), cache, table, n, max_len=1000, ws=ws), ref)
        assert gdn.device_error(ws) == 0


def test_offsets_past_32_bits(attn, gdn):
    """A cache of more than 2^31 elements, used at its far end."""
    for dtype in (BF, F32):
        page, d, hk = 64, 128, 2
        pages = 2 ** 31 // (page * d * hk) + 70
        kp, vp = (torch.empty((pages, hk, page, d), dtype=dtype, device="cuda") for _ in range(2))
        lens = [130, 4000]
        q, ks, vs, cache, table, n = make(attn, lens, 8, hk, d, page, dtype)
        far = pages - cache.pages
        kp[far:], vp[far:] = cache.k, cache.v
        big = attn.PagedCache.wrap(kp, vp)
        shifted = torch.where(table < cache.pages, table + far, table).contiguous()
        assert torch.equal(attn.paged_decode(q.cuda(), big, shifted, n), attn.paged_decode(q.cuda(), cache, table, n))


def test_captured_in_a_graph(attn, gdn):
    """One graph serves growing lengths up to max_len."""
    q, ks, vs, cache, table, n = make(attn, [500, 400], 8, 2, 128, 16, BF)
    q = q.cuda()
    ws = gdn.alloc_workspace(8 << 20, "cuda")
    out = torch.empty_like(q)
    live = n.clone()
    attn.paged_decode(q, cache, table, live, max_len=512, ws=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn.paged_decode(q, cache, table, live, max_len=512, ws=ws, out=out)
    for lens in ([500, 400], [3, 0], [250, 129]):
        live.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        assert torch.equal(out, attn.paged_decode(q, cache, table, live, max_len=512))
