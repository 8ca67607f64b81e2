"""The attention-layer operators without a GPU: refusals of the C ABI before anything is queued,
and the plain forms that the GPU tests compare with, checked by differences."""
import ctypes

import pytest
import torch

import attn_ref as R
from gated_deltanet_cpr_gb300 import api, attn, build

FAKE = 1 << 20  # aligned and never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


def norm_struct(**kw):
    base = dict(tokens=4, h_q=2, h_k=1, d=64, rot=16, table_rows=8, norm=1, layout=0, eps=1e-6, in_dtype=1, out_dtype=1,
                grad_dtype=0, q_stride=128, k_stride=64, v_stride=64)
    base.update(kw)
    return attn.NormRopeStruct(*base.values())


def test_norm_rope_refusals(lib):
    def fwd(pages=False, page=16, **kw):
        names = ("q", "k", "v", "wq", "wk", "cos", "sin", "pos", "qo", "ko")
        p = {n: kw.pop(n, FAKE) for n in names}
        slots, vp = kw.pop("slots", FAKE), kw.pop("vp", FAKE)
        st = norm_struct(**kw)
        return lib.gdn_cpr_qk_norm_rope(ctypes.byref(st), *p.values(), FAKE if pages else None, vp if pages else None, 4,
                                        page, slots if pages else None, None)

    for kw, code in [(dict(d=96), 2), (dict(rot=12), 2), (dict(rot=72), 2), (dict(norm=7), 2), (dict(layout=2), 2),
                     (dict(in_dtype=3), 2), (dict(tokens=-1), 1), (dict(h_q=0, h_k=0), 1), (dict(eps=-1.0), 1),
                     (dict(eps=float("nan")), 1), (dict(q_stride=120), 1), (dict(q_stride=129), 1), (dict(q=None), 1),
                     (dict(k=FAKE + 2), 1), (dict(cos=None), 1), (dict(pos=None), 1), (dict(wq=FAKE + 4), 1),
                     (dict(qo=FAKE + 8), 1), (dict(pages=True, page=24), 2), (dict(pages=True, page=8), 2),
                     (dict(pages=True, page=0), 1), (dict(pages=True, slots=None), 1), (dict(pages=True, v=None), 1),
                     (dict(pages=True, vp=None), 1), (dict(pages=True, v_stride=8), 1), (dict(tokens=0, q=None, k=None), 0)]:
        assert fwd(**kw) == code, kw

    def bwd(ws=FAKE, n=1 << 30, dwq=FAKE, dwk=FAKE, **kw):
        st = norm_struct(**kw)
        return lib.gdn_cpr_qk_norm_rope_bwd(ctypes.byref(st), *[FAKE] * 11, dwq, dwk, ws, n, None)

    assert bwd(n=10) == 4 and bwd(ws=None) == 4 and bwd(ws=FAKE + 16) == 4
    assert bwd(dwk=None) == 1 and bwd(rot=12) == 2 and bwd(k_stride=32) == 1


def test_norm_rope_refuses_empty_tables(lib):
    """Tokens outside the tables read their first row, so there has to be one."""
    for rows, tokens, rot, code in [(0, 4, 16, 1), (0, 0, 16, 0), (-1, 4, 16, 1)]:
        st = norm_struct(table_rows=rows, tokens=tokens, rot=rot)
        assert lib.gdn_cpr_qk_norm_rope(ctypes.byref(st), *[FAKE] * 10, None, None, 0, 16, None, None) == code
    st = norm_struct(table_rows=0)
    assert lib.gdn_cpr_qk_norm_rope_bwd(ctypes.byref(st), *[FAKE] * 13, FAKE, 1 << 30, None) == 1


def test_page_map_refusals(lib):
    def call(N=2, T=4, page=16, blocks=4, free=3, ws=FAKE, n=256, **kw):
        p = {m: kw.pop(m, FAKE) for m in ("lens", "new", "fp", "table", "seq", "cu", "pos", "slots", "used")}
        return lib.gdn_cpr_page_map(N, T, page, blocks, free, *p.values(), ws, n, None)

    for kw, code in [(dict(N=-1), 1), (dict(T=-1), 1), (dict(page=0), 1), (dict(page=20), 2), (dict(page=512), 2),
                     (dict(N=8193), 2), (dict(lens=None), 1), (dict(cu=None), 1), (dict(pos=FAKE + 4), 1),
                     (dict(fp=None), 1), (dict(table=None), 1), (dict(n=255), 4), (dict(ws=None), 4)]:
        assert call(**kw) == code, kw


def attn_struct(**kw):
    base = dict(h_q=4, h_kv=2, d=64, window=0, sinks=0, scale=0.0, dtype=1)
    base.update(kw)
    return attn.AttnStruct(*base.values())


BAD_ATTN = [(dict(d=80), 2), (dict(h_kv=3), 2), (dict(dtype=4), 2), (dict(h_q=0), 1), (dict(window=-1), 1),
            (dict(sinks=-2), 1), (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1)]


def test_paged_decode_refusals(lib):
    def call(N=2, max_len=300, pages=4, page=16, blocks=20, ws=FAKE, n=1 << 30, q=FAKE, kp=FAKE, table=FAKE, lens=FAKE,
             out=FAKE, **kw):
        st = attn_struct(**kw)
        return lib.gdn_cpr_paged_decode(ctypes.byref(st), N, max_len, q, kp, FAKE, pages, page, table, blocks, lens, out,
                                        None, ws, n, None)

    for kw, code in BAD_ATTN + [(dict(N=-1), 1), (dict(N=65536), 2), (dict(max_len=-1), 1), (dict(page=17), 2),
                                (dict(q=None), 1), (dict(kp=FAKE + 8), 1), (dict(table=None), 1), (dict(lens=None), 1),
                                (dict(out=None), 1), (dict(n=256), 4), (dict(ws=FAKE + 128), 4), (dict(N=0), 0)]:
        assert call(**kw) == code, kw


def test_decode_workspace_grows_with_the_splits(lib):
    def size(max_len, **kw):
        n, st = ctypes.c_size_t(0), attn_struct(**kw)
        assert lib.gdn_cpr_paged_decode_workspace_size(ctypes.byref(st), 3, max_len, ctypes.byref(n)) == 0
        return n.value

    assert size(0) == size(1) == 256
    sizes = [size(m) for m in list(range(0, 9000, 37)) + [20000, 131072]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))  # a longer bound never needs less
    assert size(10 ** 6, window=100, sinks=4) == size(104)


def split_runs(n, hkv):
    """Runs of a request that sees n keys, by the rule of csrc/attn.h in unbounded integers."""
    x = n * hkv
    shift = 6 if x < 128 * 32 else 7 if x < 256 * 32 else 8 if x < 512 * 32 else 9
    r = max(1, (n + (1 << shift >> 1)) >> shift)
    keys = (-(-n // r) + 31) // 32 * 32
    return -(-n // keys) if n else 0


@pytest.mark.parametrize("hkv", [1, 2, 3, 8, 40])
def test_decode_workspace_holds_every_run(lib, hkv):
    """Up to the largest length that 32 bits hold; the join reads a record for each run."""
    d, N = 64, 2
    top = 2 ** 31 - 1
    lengths = sorted({*range(1, 700), *range(700, 40000, 97), *(32 * x // hkv + e for x in (128, 256, 512) for e in (-2, -1, 0, 1, 2)),
                      10 ** 6, 10 ** 8, *(top - e for e in (300, 257, 256, 255, 254, 129, 128, 64, 32, 31, 1, 0))})
    before = 0
    for m in lengths:
        n, st = ctypes.c_size_t(0), attn_struct(h_q=hkv, h_kv=hkv, d=d)
        assert lib.gdn_cpr_paged_decode_workspace_size(ctypes.byref(st), N, m, ctypes.byref(n)) == 0
        runs = split_runs(m, hkv)
        assert runs <= 1 or n.value >= 256 + N * hkv * runs * (d + 2) * 4, m
        assert n.value >= before, m
        before = n.value


def test_window_attn_refusals(lib):
    def fwd(N=2, Tq=10, Tk=10, ws=FAKE, n=1 << 30, cq=FAKE, q=FAKE, k=FAKE, out=FAKE, lse=FAKE, **kw):
        st = attn_struct(**kw)
        return lib.gdn_cpr_window_attn(ctypes.byref(st), N, Tq, Tk, cq, FAKE, q, k, FAKE, out, lse, ws, n, None)

    def bwd(ws=FAKE, n=1 << 30, dout=FAKE, dk=FAKE, **kw):
        st = attn_struct(**kw)
        return lib.gdn_cpr_window_attn_bwd(ctypes.byref(st), 2, 10, 10, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, dout,
                                           FAKE, dk, FAKE, ws, n, None)

    for kw, code in BAD_ATTN + [(dict(N=-1), 1), (dict(N=0), 1), (dict(Tq=-1), 1), (dict(Tk=2 ** 30 + 1), 2),
                                (dict(cq=None), 1), (dict(q=None), 1), (dict(k=FAKE + 2), 1), (dict(out=None), 1),
                                (dict(lse=None), 1), (dict(n=255), 4), (dict(ws=None), 4), (dict(N=0, Tq=0, Tk=0), 0)]:
        assert fwd(**kw) == code, kw
    for kw, code in BAD_ATTN + [(dict(dout=None), 1), (dict(dk=FAKE + 4), 1), (dict(n=256), 4)]:
        assert bwd(**kw) == code, kw


def test_binding_refuses_tensors_that_do_not_fit():
    q, k = torch.zeros(4, 2, 64), torch.zeros(4, 1, 64)
    for call in (lambda: attn.qk_norm_rope(q, k),  # not on the GPU
                 lambda: attn.qk_norm_rope(q, k[:3]),
                 lambda: attn.qk_norm_rope(q, k.double()),
                 lambda: attn.window_attn(q, k, k, torch.zeros(2, dtype=torch.int32)),
                 lambda: attn.PagedCache.wrap(k, k),
                 lambda: attn.page_map(torch.zeros(2), torch.zeros(2), torch.zeros(2), torch.zeros(3, 2), 16, 4)):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_binding_keeps_sizes_past_32_bits():
    """They used to wrap: a window of 2^32 + 5 became one of 5."""
    top = 2 ** 31 - 1
    for given, meant in [(0, 0), (5, 5), (top, top), (top + 1, top), (2 ** 32, top), (2 ** 32 + 5, top), (-1, -1),
                         (-2 ** 31 - 3, -1)]:
        st = attn._attn_struct(4, 2, 64, given, given, None, torch.bfloat16)
        assert st.window == st.sinks == meant
    z = torch.zeros(2, dtype=torch.int32)
    for total in (2 ** 31, 2 ** 32 + 4, -1):
        with pytest.raises(ValueError, match="total_tokens"):
            attn.page_map(z, z, z, z[:, None], 16, total)


def test_rope_tables():
    c, s = attn.rope_tables(10, 8, base=100.0, scale=2.0, device="cpu")
    ang = 7 / 2.0 * 100.0 ** (-torch.arange(0, 8, 2).double() / 8)
    assert c.shape == (10, 4) and torch.equal(c[7], ang.cos().float()) and torch.equal(s[7], ang.sin().float())


# ------------------------------------------------------------- the plain forms themselves ----
def diff(f, x, e, h=1e-6):
    return float(f(x + h * e) - f(x - h * e)) / (2 * h)


def test_attention_gradient_by_differences():
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=g).double()  # noqa: E731
    for Lq, Lk, window, sinks in [(9, 9, 0, 0), (7, 12, 4, 2), (9, 5, 3, 1), (6, 6, 1, 0)]:
        x = dict(q=rn(Lq, 4, 8), k=rn(Lk, 2, 8), v=rn(Lk, 2, 8))
        do, pos = rn(Lq, 4, 8), torch.arange(Lq) + Lk - Lq
        r = R.attention(**x, pos=pos, window=window, sinks=sinks, dout=do)
        for n in x:
            e = rn(*x[n].shape)
            f = lambda t: (R.attention(**{**x, n: t}, pos=pos, window=window, sinks=sinks)["out"] * do).sum()  # noqa: E731
            assert abs(diff(f, x[n], e) - float((r["d" + n] * e).sum())) <= 1e-6 * (1 + float(r["d" + n].norm() * e.norm()))


def test_attention_masks_by_hand():
    """Equal scores: a row's output is the mean of the values that it sees."""
    v = torch.arange(6.0).view(6, 1, 1)
    z = torch.zeros(6, 1, 1)
    out = R.attention(z, z, v, torch.arange(6), window=2, sinks=1)["out"].flatten()
    assert torch.allclose(out, torch.tensor([0, 0.5, 1, 5 / 3, 7 / 3, 3]).double())  # {0} {0,1} {0,1,2} {0,2,3} ...
    out = R.attention(torch.zeros(3, 1, 1), z[:2], v[:2], torch.arange(3) - 1)
    assert torch.equal(out["out"].flatten(), torch.tensor([0, 0, 0.5]).double()) and out["lse"][0, 0] == -float("inf")


def test_norm_rope_gradient_by_differences():
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=g).double()  # noqa: E731
    x, w, dy = rn(5, 2, 16), rn(16), rn(5, 2, 16)
    ang, pos = rn(9, 4), torch.tensor([0, 8, 3, 3, 5])
    for norm in ("none", "rms", "l2"):
        for layout in ("half", "interleaved"):
            kw = dict(norm=norm, eps=1e-3, cos=ang.cos(), sin=ang.sin(), pos=pos, layout=layout)
            r = R.norm_rope(x, w, dy=dy, **kw)
            ex, ew = rn(5, 2, 16), rn(16)
            fx = lambda t: (R.norm_rope(t, w, **kw)["y"] * dy).sum()  # noqa: E731
            fw = lambda t: (R.norm_rope(x, t, **kw)["y"] * dy).sum()  # noqa: E731
            assert abs(diff(fx, x, ex) - float((r["dx"] * ex).sum())) < 1e-6
            assert abs(diff(fw, w, ew) - float((r["dw"] * ew).sum())) < 1e-6
