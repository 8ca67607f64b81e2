"""Norms of queries and keys with the rotation in the same pass, its gradient, and the page
tables, against plain forms in 64 bits.

Tolerances: one rounding of the output (u = 2^-8 for bf16, 2^-24 for fp32, of the value), and 2^-18
of the absolute sum of the terms for the fp32 arithmetic (64 roundings: a sum of up to 128
squares in a tree, its root and reciprocal, and a handful of products).  The weights' gradients
sum thousands of terms, in runs of at most a few hundred and then trees: 2^-16 of the absolute sum."""
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


def inputs(T, hq, hk, d, rot, dtype, seed, weights):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = dict(q=rn(T, hq, d).to(dtype), k=rn(T, hk, d).to(dtype), v=rn(T, hk, d).to(dtype),
             wq=1 + 0.2 * rn(d) if weights else None, wk=1 + 0.2 * rn(d) if weights else None, cos=None, sin=None, pos=None)
    if rot:
        ang = 3 * rn(50, rot // 2).double()
        x.update(cos=ang.cos().float(), sin=ang.sin().float(),
                 pos=torch.randint(50, (T,), generator=g, dtype=torch.int32))
    return x, rn


def kw(x, norm, layout, eps=1e-6):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    return dict(norm=norm, layout=layout, eps=eps, q_weight=c(x["wq"]), k_weight=c(x["wk"]), cos=c(x["cos"]),
                sin=c(x["sin"]), positions=c(x["pos"]))


def close(got, ref, mag, u, f=2.0 ** -18):
    got = got.cpu().double()
    return float(((got - ref).abs() / (u * ref.abs() + f * mag + 1e-30)).max()) if got.numel() else 0.0


@pytest.mark.parametrize("T,hq,hk,d,rot,norm,layout,weights,dtype,out,grad", [
    (1, 4, 1, 128, 128, "rms", "half", True, BF, BF, BF),
    (5, 3, 2, 64, 16, "rms", "interleaved", True, BF, BF, BF),
    (33, 5, 5, 32, 8, "l2", "half", False, F32, F32, F32),
    (129, 16, 2, 128, 64, "rms", "half", False, BF, F32, F32),
    (70, 2, 1, 64, 64, "none", "half", True, F32, BF, BF),
    (257, 16, 16, 128, 0, "l2", "half", False, BF, BF, F32),
    (1000, 9, 3, 32, 32, "rms", "interleaved", True, F32, F32, F32),
    (40, 8, 0, 64, 24, "rms", "half", True, BF, BF, BF),
    (3000, 7, 1, 128, 40, "rms", "interleaved", True, BF, BF, F32),
])
def test_norm_rope_and_gradient(attn, T, hq, hk, d, rot, norm, layout, weights, dtype, out, grad):
    x, rn = inputs(T, hq, hk, d, rot, dtype, T + d, weights)
    dy = {"q": rn(T, hq, d).to(grad), "k": rn(T, hk, d).to(grad)}
    args = kw(x, norm, layout)
    yq, yk = attn.qk_norm_rope(x["q"].cuda(), x["k"].cuda(), out_dtype=out, **args)
    gr = attn.qk_norm_rope_bwd(x["q"].cuda(), x["k"].cuda(), dy["q"].cuda(), dy["k"].cuda(), **args)
    assert yq.dtype == out and gr["dq"].dtype == dtype
    for n, y in (("q", yq), ("k", yk)):
        r = R.norm_rope(x[n], x["w" + n], norm, 1e-6, x["cos"], x["sin"], x["pos"], layout, dy[n])
        assert close(y, r["y"], r["y_abs"], U[out]) <= 1
        assert close(gr["d" + n], r["dx"], r["dx_abs"], U[dtype]) <= 1
        if weights:
            assert close(gr[f"d{n}_weight"], r["dw"], r["dw_abs"] + 1e-20, 2.0 ** -24, 2.0 ** -16) <= 1


def test_strided_projection_and_other_stream(attn):
    """q, k and v as parts of one projection's rows, on a stream of the caller's."""
    T, hq, hk, d = 77, 6, 2, 64
    qkv = torch.randn(T, (hq + 2 * hk) * d, device="cuda").to(BF)
    q, k, v = (t.view(T, -1, d) for t in qkv.split([hq * d, hk * d, hk * d], 1))
    ref, refk = attn.qk_norm_rope(q.contiguous(), k.contiguous(), norm="l2")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y, yk = attn.qk_norm_rope(q, k, norm="l2")
        g = attn.qk_norm_rope_bwd(q, k, y, yk, norm="l2")
    st.synchronize()
    assert torch.equal(y, ref) and torch.equal(yk, refk)
    g2 = attn.qk_norm_rope_bwd(q.contiguous(), k.contiguous(), ref, refk, norm="l2")
    assert torch.equal(g["dq"], g2["dq"]) and torch.equal(g["dk"], g2["dk"])
    # k as every other pair of heads: a token's heads are not contiguous
    with pytest.raises(ValueError):
        attn.qk_norm_rope(q[:, ::2], k, norm="l2")


def test_one_head_of_any_stride(attn):
    """The stride of an axis of one head says nothing: a tensor that is dense all the same is taken."""
    k = torch.randn(1, 9, 64, device="cuda").to(BF).transpose(0, 1)
    q = torch.randn(9, 2, 64, device="cuda").to(BF)
    assert k.is_contiguous() and k.stride(1) != 64
    got, ref = attn.qk_norm_rope(q, k, norm="l2"), attn.qk_norm_rope(q, k.clone(memory_format=torch.contiguous_format).view(9, 1, 64), norm="l2")
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_cache_write_and_skipped_slots(attn):
    T, hq, hk, d, page = 37, 4, 2, 128, 16
    x, _ = inputs(T, hq, hk, d, 32, BF, 3, True)
    cache = attn.PagedCache(5, page, hk, d)
    cache.k.fill_(7)
    cache.v.fill_(7)
    slots = torch.randperm(5 * page)[:T].int()
    slots[3], slots[9], slots[20] = -1, 5 * page, -(2 ** 31)  # not kept
    q, k = attn.qk_norm_rope(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), cache=cache, slot_map=slots.cuda(),
                             **kw(x, "rms", "half"))
    want_k, want_v = torch.full_like(cache.k, 7), torch.full_like(cache.v, 7)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < 5 * page:
            want_k[s // page, :, s % page], want_v[s // page, :, s % page] = k[t], x["v"][t].cuda()
    assert torch.equal(cache.k, want_k) and torch.equal(cache.v, want_v)
    # only the cache wanted: the same pages
    c2 = attn.PagedCache.wrap(torch.full_like(cache.k, 7), torch.full_like(cache.v, 7))
    q2, none = attn.qk_norm_rope(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), cache=c2, slot_map=slots.cuda(),
                                 want_k=False, **kw(x, "rms", "half"))
    assert none is None and torch.equal(q2, q) and torch.equal(c2.k, cache.k)


def test_positions_outside_the_tables_and_special_values(attn):
    x, _ = inputs(6, 2, 2, 64, 64, F32, 5, True)
    x["pos"][1], x["pos"][4] = -1, 50
    x["q"][2] = 0  # a row of zeros stays one
    x["q"][3, 0, 5] = float("inf")
    y, yk = attn.qk_norm_rope(x["q"].cuda(), x["k"].cuda(), **kw(x, "rms", "half"))
    g = attn.qk_norm_rope_bwd(x["q"].cuda(), x["k"].cuda(), torch.ones_like(y), torch.ones_like(yk),
                              **kw(x, "rms", "half"))
    bad = torch.tensor([False, True, False, False, True, False])
    assert torch.isnan(yk.cpu()).all((1, 2)).tolist() == bad.tolist()
    assert torch.isnan(g["dk"].cpu()).all((1, 2)).tolist() == bad.tolist()
    assert (y[2] == 0).all() and torch.isfinite(y[3, 1]).all()
    assert torch.isfinite(g["dk_weight"]).all()


def test_norm_gradient_against_differences(attn):
    """<dx, e> against central differences of <dy, y> along e, fp32: 4e-2 steps of unit vectors leave
    a third-order remainder and 2^-24 |loss| / step, both below 2e-3 of the gradient's size."""
    x, rn = inputs(9, 3, 2, 64, 32, F32, 8, True)
    args = kw(x, "rms", "interleaved")
    dq, dk = rn(9, 3, 64).cuda(), rn(9, 2, 64).cuda()
    g = attn.qk_norm_rope_bwd(x["q"].cuda(), x["k"].cuda(), dq, dk, **args)
    for _ in range(4):
        e = rn(9, 3, 64)
        e = (e / e.norm()).cuda()
        h = 4e-2
        f = [float((attn.qk_norm_rope((x["q"].cuda() + s * h * e), x["k"].cuda(), **args)[0].double() * dq).sum())
             for s in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * h) - float((g["dq"] * e).sum())) <= 2e-3 * float(g["dq"].norm())


def test_weight_gradients_repeat(attn):
    x, rn = inputs(5000, 8, 2, 128, 0, BF, 9, True)
    dq, dk = rn(5000, 8, 128).cuda(), rn(5000, 2, 128).cuda()
    a, b = (attn.qk_norm_rope_bwd(x["q"].cuda(), x["k"].cuda(), dq, dk, **kw(x, "rms", "half")) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


# ------------------------------------------------------------------------- page tables ----
def plain_map(old, new, free, table, page):
    table = [list(r) for r in table]
    used, pos, slots, cu = 0, [], [], [0]
    for n, (l, m) in enumerate(zip(old, new)):
        for b in range(-(-l // page), -(-(l + m) // page)):
            table[n][b] = free[used]
            used += 1
        for p in range(l, l + m):
            pos.append(p)
            slots.append(table[n][p // page] * page + p % page)
        cu.append(cu[-1] + m)
    return dict(table=table, seq_lens=[a + b for a, b in zip(old, new)], cu_seqlens=cu, positions=pos, slot_map=slots,
                pages_used=[used])


def make_map(N, old_hi, new_hi, page, seed, slack=2):
    g = torch.Generator().manual_seed(seed)
    old = torch.randint(old_hi + 1, (N,), generator=g).tolist()
    new = torch.randint(new_hi + 1, (N,), generator=g).tolist()
    have = [-(-o // page) for o in old]
    width = max(-(-(a + b) // page) for a, b in zip(old, new)) + slack
    need = sum(-(-(a + b) // page) - c for a, b, c in zip(old, new, have))
    ids = torch.randperm(sum(have) + need + 3, generator=g).tolist()
    table, at = [], 0
    for h in have:
        table.append(ids[at:at + h] + [-9] * (width - h))
        at += h
    return old, new, ids[at:], table


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("N,old_hi,new_hi,page", [(1, 0, 1, 16), (3, 40, 1, 16), (5, 0, 0, 32), (17, 500, 90, 64),
                                                  (64, 0, 3000, 16), (1100, 300, 7, 128), (8192, 20, 2, 256)])
def test_page_map(attn, gdn, N, old_hi, new_hi, page):
    old, new, free, table = make_map(N, old_hi, new_hi, page, N)
    want = plain_map(old, new, free, table, page)
    t = i32(table)
    for _ in range(2):  # nothing is taken off the list: a call may be repeated
        m = attn.page_map(i32(old), i32(new), i32(free), t, page, sum(new))
        assert gdn.device_error(m["ws"]) == 0
        assert t.tolist() == want["table"]
        for n in ("seq_lens", "cu_seqlens", "positions", "slot_map", "pages_used"):
            assert m[n].tolist() == want[n], n


def test_page_map_refuses_without_touching_the_table(attn, gdn):
    old, new, free, table = make_map(6, 50, 40, 16, 2)
    t = i32(table)

    def code(old=old, new=new, free=free, total=None, tab=None):
        tt = t if tab is None else tab
        before = tt.clone()
        m = attn.page_map(i32(old), i32(new), i32(free), tt, 16, sum(new) if total is None else total)
        c = gdn.device_error(m["ws"])
        if c in (1, 3) or (c == 7 and m["slot_map"].numel() and bool((m["positions"] == -1).all())):
            assert torch.equal(tt, before) and m["pages_used"].item() == 0
        return c, m

    used = plain_map(old, new, free, table, 16)["pages_used"][0]
    assert code(total=sum(new) + 1)[0] == 1
    assert code(old=[-1] + old[1:])[0] == 3
    assert code(new=[2 ** 31 - 1] + new[1:], total=10)[0] == 3
    assert code(free=free[:used - 1])[0] == 7
    assert code(tab=t[:, :2].contiguous())[0] == 7
    bad = list(free)
    bad[0] = -4
    c, m = code(free=bad, tab=t.clone())
    assert c == 7 and (m["slot_map"] == -1).any() and (m["slot_map"] >= 0).any()
    assert code()[0] == 0
