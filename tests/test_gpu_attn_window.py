"""Sliding-window attention over packed sequences and its gradient against plain attention in
64 bits (tolerances: see attn_ref; u = 2^-8 for bf16, 2^-24 for fp32)."""
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


def cu(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)


def make(ql, kl, hq, hk, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g).to(dtype)  # noqa: E731
    return dict(q=rn(sum(ql), hq, d), k=rn(sum(kl), hk, d), v=rn(sum(kl), hk, d), do=rn(sum(ql), hq, d), cq=cu(ql), ck=cu(kl))


def run(attn, x, **kw):
    c = {n: t.cuda() for n, t in x.items()}
    kw["cu_seqlens_k"] = c["ck"]
    out, lse = attn.window_attn(c["q"], c["k"], c["v"], c["cq"], **kw)
    g = attn.window_attn_bwd(c["q"], c["k"], c["v"], out, lse, c["do"], c["cq"], **kw)
    return dict(out=out, lse=lse, **g)


def check(attn, ql, kl=None, hq=4, hk=2, d=64, dtype=BF, window=0, sinks=0, scale=None, seed=0):
    kl = kl or ql
    x = make(ql, kl, hq, hk, d, dtype, seed)
    got = run(attn, x, window=window, sinks=sinks, scale=scale)
    ref = R.packed(x["q"], x["k"], x["v"], x["cq"].tolist(), x["ck"].tolist(), window, sinks, scale, x["do"], U[dtype])
    for n in ("out", "lse", "dq", "dk", "dv"):
        assert got[n].dtype == (F32 if n == "lse" else dtype)
        w = R.worst(got[n], ref[n], ref["tol"][n])
        assert w <= 1, (n, w)
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_ragged_lengths(attn, d, dtype):
    """Single tokens, empty sequences, lengths about the tiles' edges."""
    check(attn, [1, 63, 64, 0, 65, 127, 128, 129, 2, 300], d=d, dtype=dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (6, 2), (8, 1), (5, 1)])
def test_grouped_heads(attn, hq, hk, dtype):
    check(attn, [70, 200], hq=hq, hk=hk, d=128, dtype=dtype, window=50, sinks=2)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 32), (F32, 128), (F32, 32)])
@pytest.mark.parametrize("hq", [9, 12, 17])
def test_more_than_eight_heads_of_a_key_head(attn, dtype, d, hq):
    """In 32 bits the gradient shares them out over at most eight CTAs, some of which then have none."""
    check(attn, [90, 0, 150], hq=hq, hk=1, d=d, dtype=dtype, window=60, sinks=3)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 2), (64, 0), (100, 4), (128, 130), (129, 300), (0, 7),
                                          (300, 1), (1000, 3), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_window_and_first_tokens(attn, dtype, d, window, sinks):
    check(attn, [400, 5, 131], hq=2, hk=1, d=d, dtype=dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 32)])
def test_queries_at_the_end_of_longer_keys(attn, dtype, d):
    """Fewer queries than keys; more queries than keys, whose first rows see nothing; none of either."""
    check(attn, [1, 50, 130, 200, 40, 0, 9], [300, 333, 131, 120, 0, 77, 9], d=d, dtype=dtype)
    check(attn, [1, 50, 130, 200, 40, 0, 9], [300, 333, 131, 120, 0, 77, 9], d=d, dtype=dtype, window=33, sinks=5)
    check(attn, [300], [4], d=d, dtype=dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_window(attn, dtype):
    check(attn, [1500, 700], hq=2, hk=1, d=128, dtype=dtype, window=600, sinks=4)
    check(attn, [1100], hq=2, hk=2, d=64, dtype=dtype)


def test_large_scores(attn):
    """Scores of some hundreds: the running maximum has to move."""
    for dtype, d in ((BF, 128), (F32, 64)):
        x = make([300], [300], 2, 1, d, dtype)
        got = run(attn, x, scale=5.0, window=200, sinks=1)
        ref = R.packed(x["q"], x["k"], x["v"], [0, 300], [0, 300], 200, 1, 5.0, x["do"], U[dtype])
        for n in ("out", "lse", "dq", "dk", "dv"):
            assert R.worst(got[n], ref[n], ref["tol"][n]) <= 1, n


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
def test_other_sequences_do_not_matter(attn, dtype, d):
    """The same bits alone and packed, whatever lies in the other sequences' rows."""
    lens = [200, 77, 130]
    x = make(lens, lens, 4, 2, d, dtype)
    got = run(attn, x, window=90, sinks=3)
    a, b = 200, 277
    one = {n: x[n][a:b] for n in ("q", "k", "v", "do")} | dict(cq=cu([77]), ck=cu([77]))
    alone = run(attn, one, window=90, sinks=3)
    for n in alone:
        assert torch.equal(alone[n], got[n][a:b]), n
    for junk in (float("nan"), float("inf")):
        y = {n: t.clone() for n, t in x.items()}
        for n in ("q", "k", "v", "do"):
            y[n][:a], y[n][b:] = junk, junk
        dirty = run(attn, y, window=90, sinks=3)
        for n in alone:
            assert torch.equal(alone[n], dirty[n][a:b]), (n, junk)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("n,window,sinks,scale", [(200, 73, 0, None), (333, 90, 3, 0.5), (333, 0, 0, None), (530, 0, 0, 0.4),
                                                  (141, 0, 0, 5.0), (700, 256, 1, 5.0)])
def test_later_sequences_do_not_move_a_row_s_maximum(attn, dtype, d, n, window, sinks, scale):
    """Sequences of several key blocks that end inside a tile and inside a warp's rows: the same bits alone
    and before rows of any size, whose scores move their running maximum at every block."""
    kw = dict(window=window, sinks=sinks, scale=scale)
    x = make([n, 150], [n, 150], 4, 2, d, dtype, seed=n)
    one = {m: x[m][:n] for m in ("q", "k", "v", "do")} | dict(cq=cu([n]), ck=cu([n]))
    alone = run(attn, one, **kw)
    for size in (1.0, 1e3, -1e3, float("nan"), float("inf")):
        y = {m: t.clone() for m, t in x.items()}
        for m in ("q", "k", "v", "do"):
            y[m][n:] *= size
        got = run(attn, y, **kw)
        for m in alone:
            assert torch.equal(alone[m], got[m][:n]), (m, size)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 128), (F32, 32)])
def test_batch_size_does_not_change_bits(attn, dtype, d):
    """A sequence alone and among many (which may choose other tiles and schedules)."""
    lens = [150] * 20 + [333] * 40
    x = make(lens, lens, 4, 2, d, dtype)
    got = run(attn, x, window=90, sinks=3)
    for s, (a, b) in {3: (450, 600), 30: (3000 + 10 * 333, 3000 + 11 * 333)}.items():
        one = {n: x[n][a:b] for n in ("q", "k", "v", "do")} | dict(cq=cu([b - a]), ck=cu([b - a]))
        alone = run(attn, one, window=90, sinks=3)
        for n in alone:
            assert torch.equal(alone[n], got[n][a:b]), (n, s)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_repeatable_and_on_another_stream(attn, dtype, d):
    x = make([500, 260], [500, 260], 6, 2, d, dtype)
    a = run(attn, x, window=100, sinks=2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = run(attn, x, window=100, sinks=2)
    st.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_gradient_against_differences(attn):
    """<dx, e> against central differences of <dout, out> along unit vectors e, fp32: steps of 0.05
    leave a third-order remainder and 2^-24 |loss| / step, below 1e-2 of the gradient's size."""
    x = make([90, 20], [90, 35], 4, 2, 64, F32)
    kw = dict(window=30, sinks=2)
    g = run(attn, x, **kw)
    c = {n: t.cuda() for n, t in x.items()}
    gen = torch.Generator().manual_seed(1)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        e = torch.randn(x[name].shape, generator=gen)
        e = (e / e.norm()).cuda()
        h, f = 5e-2, []
        for s in (1, -1):
            y = dict(c)
            y[name] = c[name] + s * h * e
            o, _ = attn.window_attn(y["q"], y["k"], y["v"], y["cq"], cu_seqlens_k=y["ck"], **kw)
            f.append(float((o.double() * c["do"]).sum()))
        assert abs((f[0] - f[1]) / (2 * h) - float((g[grad].double() * e).sum())) <= 1e-2 * float(g[grad].norm())


def test_bad_tables_are_reported(attn, gdn):
    for dtype, d in ((BF, 128), (F32, 64)):
        x = make([100, 30], [100, 30], 2, 1, d, dtype)
        c = {n: t.cuda() for n, t in x.items()}
        ws = gdn.alloc_workspace(1 << 20, "cuda")
        for bad in ([0, 140, 130], [0, -5, 130], [1, 100, 130], [0, 100, 129], [0, 2 ** 30, 130]):
            t = torch.tensor(bad, dtype=torch.int32, device="cuda")
            out, lse = attn.window_attn(c["q"], c["k"], c["v"], t, ws=ws)
            assert gdn.device_error(ws) == 1
            attn.window_attn_bwd(c["q"], c["k"], c["v"], out, lse, c["do"], t, ws=ws)
            assert gdn.device_error(ws) == 1
        attn.window_attn(c["q"], c["k"], c["v"], c["cq"], ws=ws)
        assert gdn.device_error(ws) == 0


def test_nothing_to_do(attn, gdn):
    for dtype, d in ((BF, 128), (F32, 32)):
        got = run(attn, make([0, 0], [0, 0], 2, 1, d, dtype))
        assert got["out"].numel() == 0 and got["dk"].numel() == 0
        got = run(attn, make([0, 0], [10, 0], 2, 1, d, dtype))
        assert (got["dk"] == 0).all() and (got["dv"] == 0).all()
        got = run(attn, make([5, 0], [0, 0], 2, 1, d, dtype))
        assert (got["out"] == 0).all() and (got["dq"] == 0).all() and (got["lse"] == -float("inf")).all()


def test_empty_calls_set_the_error_word(attn, gdn):
    """A workspace that held an error, or anything at all, says after a call of no sequences that nothing was wrong."""
    for dtype, d in ((BF, 128), (BF, 32), (F32, 64)):
        x = {n: t.cuda() for n, t in make([100, 30], [100, 30], 2, 1, d, dtype).items()}
        e = {n: t.cuda() for n, t in make([], [], 2, 1, d, dtype).items()}
        q1 = torch.zeros((1, 2, d), dtype=dtype, device="cuda")
        cache = attn.PagedCache(2, 16, 1, d, dtype)
        table, none = torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
        bad = torch.tensor([0, 140, 130], dtype=torch.int32, device="cuda")
        ws = gdn.alloc_workspace(1 << 20, "cuda")
        empty = (lambda: attn.window_attn(e["q"], e["k"], e["v"], e["cq"], ws=ws),
                 lambda: attn.window_attn_bwd(e["q"], e["k"], e["v"], e["q"], e["q"][..., 0].float(), e["q"], e["cq"], ws=ws),
                 lambda: attn.paged_decode(q1[:0], cache, table[:0], none, ws=ws))
        for call in empty:
            attn.window_attn(x["q"], x["k"], x["v"], bad, ws=ws)
            assert gdn.device_error(ws) == 1
            call()
            assert gdn.device_error(ws) == 0
            ws.fill_(0x55)
            call()
            assert gdn.device_error(ws) == 0
    # and inside a graph
    ws.fill_(0x55)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in empty:
            call()
    for _ in range(2):
        ws.fill_(0x55)
        g.replay()
        assert gdn.device_error(ws) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out_is_reported(attn, gdn, d):
    """The test hook makes the kernels start a copy, wait for a phase that nothing completes, and give up: their
    memory is given back, the error word says so, and the next calls run as usual."""
    x = make([500, 260], [500, 260], 4, 2, d, BF)
    ref = run(attn, x, window=100, sinks=2)
    c = {n: t.cuda() for n, t in x.items()}
    ws = gdn.alloc_workspace(1 << 20, "cuda")
    kw = dict(cu_seqlens_k=c["ck"], window=100, sinks=2, ws=ws)
    calls = (lambda: attn.window_attn(c["q"], c["k"], c["v"], c["cq"], **kw),
             lambda: attn.window_attn_bwd(c["q"], c["k"], c["v"], ref["out"], ref["lse"], c["do"], c["cq"], **kw))
    for call in calls:
        gdn.test_wait_timeout(1)
        try:
            call()
            assert gdn.device_error(ws) == 4  # GDN_DEVERR_TIMEOUT
        finally:
            gdn.test_wait_timeout(0)
        call()
        assert gdn.device_error(ws) == 0
    got = run(attn, x, window=100, sinks=2)
    assert all(torch.equal(got[n], ref[n]) for n in ref)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens,window,sinks", [([2, 1, 7, 16, 3, 12, 17, 40], 0, 0), ([300, 1, 2], 2, 0), ([150, 65], 3, 2),
                                               ([90, 0, 33], 12, 4), ([140], 1, 1), ([200, 31], 9, 8), ([50], 1, 0)])
def test_gradients_of_rows_that_see_few_keys(attn, d, lens, window, sinks):
    """With few visible keys dP - delta cancels, so delta may not carry the rounding of the output to bf16.
    Bounds for rows of at most 16 keys: the score gradients' own rounding to bf16 (u of ds) and c roundings to 32
    bits of everything else, c as in attn_ref; nothing of the size of the output's rounding."""
    hq, hk, u = 4, 2, U[BF]
    x = make(lens, lens, hq, hk, d, BF, seed=d)
    got = run(attn, x, window=window, sinks=sinks)
    at = 0
    for n in lens:
        q, k, v, do = (x[m][at:at + n].double().transpose(0, 1) for m in ("q", "k", "v", "do"))
        k, v = k.repeat_interleave(hq // hk, 0), v.repeat_interleave(hq // hk, 0)
        see = R.visible(torch.arange(n), torch.arange(n), window, sinks)
        few = see.sum(1) <= 16
        sc = d ** -0.5
        size = torch.where(see, (q.abs() @ k.abs().transpose(1, 2)) * sc, 0.0)
        p = torch.softmax(torch.where(see, (q @ k.transpose(1, 2)) * sc, -float("inf")), -1) if n else size
        o, dp = p @ v, do @ v.transpose(1, 2)
        ds = p * (dp - (do * o).sum(-1, keepdim=True)) * sc
        dq = ds @ k
        c = 16 + d ** 0.5 + 2 * (float(size.max()) if n else 0.0)
        mag = do.abs() @ v.abs().transpose(1, 2) + (do.abs() * (p @ v.abs())).sum(-1, keepdim=True)
        e_ds = (u + 2 * c * R.EPS) * ds.abs() + c * R.EPS * sc * p * mag
        tol = u * dq.abs() + e_ds @ k.abs() + 1e-30
        err = (got["dq"][at:at + n].cpu().double().transpose(0, 1) - dq).abs()
        assert n == 0 or not bool(few.any()) or float((err / tol)[:, few].max()) <= 1, n
        if n and bool(few.all()):
            group = lambda t: t.view(hk, hq // hk, n, d).sum(1)  # noqa: E731
            dk, tk = group(ds.transpose(1, 2) @ q), group(e_ds.transpose(1, 2) @ q.abs())
            tk = tk + u * dk.abs() + 8 * c * R.EPS * group(ds.abs().transpose(1, 2) @ q.abs()) + 1e-30
            err = (got["dk"][at:at + n].cpu().double().transpose(0, 1) - dk).abs()
            assert float((err / tk).max()) <= 1, n
        at += n
