"""The 8-bit cache without a GPU: refusals of the C ABI before anything is queued, and the plain form that the GPU
tests compare with."""
import ctypes

import pytest
import torch

import quant_ref as R
from gated_deltanet_cpr_gb300 import api, attn, build

FAKE = 1 << 20  # aligned and never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


def cache(**kw):
    base = dict(num_pages=8, page_size=64, block=16, slots=4, h_kv=2, d=64, code=0, dtype=1, k_pages=FAKE, v_pages=FAKE,
                k_scale=FAKE, v_scale=FAKE, k_tail=FAKE, v_tail=FAKE)
    base.update(kw)
    return attn.QuantCacheStruct(*base.values())


BAD_CACHE = [(dict(num_pages=-1), 1), (dict(page_size=0), 1), (dict(page_size=24), 2), (dict(page_size=512), 2), (dict(block=0), 1),
             (dict(block=-16), 1), (dict(block=8), 2), (dict(block=24), 2), (dict(block=256, page_size=256), 2), (dict(block=128), 2),
             (dict(slots=-1), 1), (dict(h_kv=0), 1), (dict(h_kv=65536), 2), (dict(d=96), 2), (dict(code=2), 2), (dict(dtype=2), 2),
             (dict(num_pages=1 << 26), 2), (dict(slots=1 << 27), 2), (dict(k_pages=None), 1), (dict(v_pages=FAKE + 8), 1),
             (dict(k_scale=FAKE + 2), 1), (dict(v_scale=None), 1), (dict(k_tail=None), 1), (dict(v_tail=FAKE + 4), 1)]
BAD_ROWS = [(dict(N=-1), 1), (dict(T=-1), 1), (dict(blocks=-1), 1), (dict(N=0), 1), (dict(N=65536), 2), (dict(cu=None), 1),
            (dict(lens=None), 1), (dict(table=None), 1), (dict(slot=FAKE + 1), 1), (dict(k=None), 1), (dict(v=FAKE + 8), 1),
            (dict(ws=FAKE + 64), 4), (dict(n=255), 4), (dict(h_kv=65535, T=1 << 30), 2),
            (dict(N=0, T=0, cu=None, lens=None, k_pages=None, k_tail=None), 0), (dict(N=0, T=0, ws=None, n=0), 0)]


def split(kw):
    names = ("N", "T", "blocks", "cu", "lens", "table", "slot", "k", "v", "ws", "n", "ks", "vs", "out")
    return {n: kw[n] for n in kw if n in names}, cache(**{n: kw[n] for n in kw if n not in names})


def test_append_refusals(lib):
    def call(**kw):
        p, c = split(kw)
        g = lambda n, x=FAKE: p.get(n, x)  # noqa: E731
        row = c.h_kv * c.d if c.d > 0 else 64
        return lib.gdn_cpr_quant_append(ctypes.byref(c), g("N", 2), g("T", 10), g("k"), g("v"), g("ks", row), g("vs", row), g("cu"),
                                        g("lens"), g("table"), g("blocks", 4), g("slot"), g("ws"), g("n", 256), None)

    for kw, code in BAD_CACHE + BAD_ROWS + [(dict(ks=120), 1), (dict(vs=132), 1), (dict(dtype=0, ks=130), 1), (dict(vs=-128), 1)]:
        assert call(**kw) == code, kw
    assert lib.gdn_cpr_quant_append(None, 2, 10, FAKE, FAKE, 128, 128, FAKE, FAKE, FAKE, 4, None, FAKE, 256, None) == 1


def test_read_refusals(lib):
    def call(**kw):
        p, c = split(kw)
        g = lambda n, x=FAKE: p.get(n, x)  # noqa: E731
        return lib.gdn_cpr_quant_read(ctypes.byref(c), g("N", 2), g("T", 10), g("cu"), g("lens"), g("table"), g("blocks", 4),
                                      g("slot"), g("out", 1), g("k"), g("v"), g("ws"), g("n", 256), None)

    for kw, code in BAD_CACHE + BAD_ROWS + [(dict(out=2), 2), (dict(out=-1), 2)]:
        assert call(**kw) == code, kw


def test_binding_refuses_tensors_that_do_not_fit():
    k, t = torch.zeros((4, 2, 32, 64), dtype=torch.int8), torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    s = torch.zeros((4, 2, 2))
    for call in (lambda: attn.QuantCache.wrap(k, k, s, s, t, t),  # not on the GPU
                 lambda: attn.QuantCache.wrap(k.float(), k, s, s, t, t),
                 lambda: attn.QuantCache.wrap(k[0], k[0], s, s, t, t),
                 lambda: attn.QuantCache.wrap(k, k, s, s, t.double(), t),
                 lambda: attn.QuantCache.wrap(k[:, :, :24], k[:, :, :24], s, s, t, t),
                 lambda: attn.QuantCache(4, 32, 2, 64, 3, block=24, device="cpu"),
                 lambda: attn.QuantCache(4, 32, 2, 64, 3, code="int4", device="cpu")):
        with pytest.raises((ValueError, TypeError, KeyError)):
            call()


def test_plain_rounding_by_hand():
    # 127 x / m of a block with m = 254: halves go to the even whole number
    x = torch.zeros(1, 16, 32)
    x[0, 0, :6] = torch.tensor([254.0, 1.0, 3.0, -1.0, -3.0, 5.0])
    c, s = R.quantise(x, "int8")
    assert c[0, 0, :6].tolist() == [127, 0, 2, 0, -2, 2] and s.tolist() == [2.0]
    # the format's values: 448 at the top, ties between 16 and 18, and below the least one
    x[0, 0, :6] = torch.tensor([448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10])
    c, s = R.quantise(x, "e4m3")
    assert c[0, 0, :6].tolist() == [448, 16, 20, -16, 0, 2.0 ** -8] and s.tolist() == [1.0]
    x[0, 0, 0] = 449.0
    assert R.quantise(x, "e4m3")[1].tolist() == [2.0]
    x[0, 0, 0] = 447.0
    assert R.quantise(x, "e4m3")[1].tolist() == [1.0]
    g = torch.Generator().manual_seed(0)
    for dtype in (torch.bfloat16, torch.float32):
        x = (torch.randn((50, 16, 64), generator=g) * torch.exp(3 * torch.randn((50, 1, 1), generator=g))).to(dtype)
        for code, most in (("int8", 0.5 / 127), ("e4m3", 2.0 ** -4)):
            c, s = R.quantise(x, code)
            err = (c * s.double()[:, None, None] - x.double()).abs()
            m = x.double().abs().amax((1, 2), keepdim=True)
            # half a step of the largest (int8), or of the value, with its least step (e4m3); s has 24 bits
            bound = most * m if code == "int8" else torch.maximum(most * x.double().abs(), 2.0 ** -10 * s.double()[:, None, None])
            assert bool((err <= bound * (1 + 2.0 ** -15)).all())
    for v, want in [(float("nan"), float("nan")), (float("inf"), float("nan")), (2.0 ** -101, 0.0)]:
        x = torch.zeros(1, 16, 32)
        x[0, 2, 3] = v
        c, s = R.quantise(x, "int8")
        assert c.eq(0).all() and (s.isnan().all() if want != want else s.eq(0).all())


BAD_ATTN = [(dict(h_q=3), 2), (dict(h_q=0), 1), (dict(window=-1), 1), (dict(sinks=-2), 1), (dict(scale=-1.0), 1),
            (dict(scale=float("inf")), 1), (dict(a_h_kv=4), 1), (dict(a_d=128), 1), (dict(a_dtype=0), 1), (dict(a_d=80), 2)]


def test_decode_refusals(lib):
    def call(**kw):
        at = {n: kw.pop(n) for n in ("h_q", "window", "sinks", "scale", "a_h_kv", "a_d", "a_dtype", "max_len", "q") if n in kw}
        p, c = split(kw)
        g = lambda n, x=FAKE: p.get(n, x)  # noqa: E731
        st = attn.AttnStruct(at.get("h_q", 4), at.get("a_h_kv", 2), at.get("a_d", 64), at.get("window", 0), at.get("sinks", 0),
                             at.get("scale", 0.0), at.get("a_dtype", 1))
        return lib.gdn_cpr_quant_decode(ctypes.byref(st), ctypes.byref(c), g("N", 2), at.get("max_len", 300), at.get("q", FAKE),
                                        g("table"), g("blocks", 4), g("lens"), g("slot"), g("out"), None, g("ws"), g("n", 1 << 30), None)

    # a head count or size that is refused by itself is refused before it is compared with attn's
    for kw, code in BAD_CACHE + BAD_ATTN + [
            (dict(N=-1), 1), (dict(N=65536), 2), (dict(max_len=-1), 1), (dict(blocks=-1), 1), (dict(q=None), 1), (dict(out=FAKE + 8), 1),
            (dict(lens=None), 1), (dict(table=None), 1), (dict(slot=FAKE + 2), 1), (dict(n=256), 4), (dict(ws=FAKE + 128), 4),
            (dict(N=0, q=None, k_pages=None), 0)]:
        assert call(**kw) == code, kw


def split_runs(n, hkv):
    """Runs of a request of n granules, by the rule of csrc/attn_quant.h in unbounded integers."""
    s = 2
    while s < 5 and n * hkv >= 32 << (s + 1):
        s += 1
    keys = -(-n // max(1, (n + (1 << s >> 1)) >> s))
    return -(-n // keys) if n else 0


def granules(L, window, sinks):
    """Granules of 16 keys that hold visible ones."""
    if not window or L <= window:
        return -(-L // 16)
    first = (L - window) // 16
    return min(-(-min(sinks, L) // 16), first) + (L - 1) // 16 - first + 1


@pytest.mark.parametrize("hkv", [1, 3, 8, 40])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4), (2033, 17), (1, 0), (5000, 3000)])
def test_decode_workspace_holds_every_run(lib, hkv, window, sinks):
    """Of every length up to its bound, the join reads a record for each run."""
    d, N, top = 64, 2, 2 ** 31 - 1

    def size(m):
        n, st = ctypes.c_size_t(0), attn.AttnStruct(hkv, hkv, d, window, sinks, 0.0, 1)
        assert lib.gdn_cpr_quant_decode_workspace_size(ctypes.byref(st), N, m, ctypes.byref(n)) == 0
        return n.value

    most, before = 0, 0
    for L in sorted({*range(0, 6000), *range(6000, 40000, 97), 10 ** 6, 10 ** 8, top - 300, top - 16, top - 1, top}):
        most = max(most, split_runs(granules(L, window, sinks), hkv))
        n = size(L)
        assert most <= 1 or n >= 256 + N * hkv * most * (d + 2) * 4, L
        assert n >= before
        before = n
