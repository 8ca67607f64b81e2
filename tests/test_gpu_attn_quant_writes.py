"""What an append to the 8-bit cache writes, bit for bit: of both keys and values everything that it should and nothing else, also
where the call's descriptions are wrong, with an error word and without."""
import pytest
import torch

import quant_ref as R
from test_gpu_attn_quant_rows import BF, F32, Store, attn, ints, offsets, rows  # noqa: F401

pytestmark = pytest.mark.gpu
NAMES = ("k pages", "v pages", "k scale", "v scale", "k tail", "v tail")


def assert_state(got, want, what):
    for name, a, b in zip(NAMES, got, want):
        assert torch.equal(a, b), (what, name, (a != b).nonzero()[:4].tolist())


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page,block", [(32, 16, 16), (64, 32, 16), (128, 64, 64), (64, 128, 128)])
def test_all_of_the_cache_after_an_append(attn, gdn, d, page, block, dtype, code):
    """Pages, scales and tails of every request and of nobody."""
    lens, hk = [0, 1, 15, 16, 17, 0, 127, 128, 129, 300], 3
    s = Store(attn, gdn, lens, hk, d, page, block, code, dtype)
    want = [t.clone().cpu() for t in s.state()]
    xs = rows(lens, hk, d, dtype, 1), rows(lens, hk, d, dtype, 2)
    s.append(*xs, lens)
    table = s.table.cpu()
    for side in (0, 1):
        for n, x in enumerate(xs[side]):
            w = len(x) // block
            c, sc = R.quantise(x[:w * block].view(w, block, hk, d).transpose(1, 2), code)
            codes = c.to(torch.int8).view(torch.uint8) if code == "int8" else c.float().to(torch.float8_e4m3fn).view(torch.uint8)
            for b in range(w):
                p, j = int(table[n, b * block // page]), b % (page // block)
                want[side][p, :, j * block:(j + 1) * block] = codes[b]
                want[2 + side][p, :, j] = sc[b].view(torch.int32)
            r, slot = len(x) - w * block, int(s.slots[n])
            tail = want[4 + side][slot].view(dtype)
            tail[:, :r] = x[w * block:].transpose(0, 1)
    got = [t.cpu() for t in s.state()]
    if code == "e4m3":  # a code of 0 has two signs
        for g, w in zip(got[:2], want[:2]):
            g[g == 0x80], w[w == 0x80] = 0, 0
    assert_state(got, want, "append")


OLD, NEW, LENS = [5, 20, 0], [35, 30, 70], [40, 50, 70]


class Faulty:
    """Requests of OLD tokens to which NEW ones are appended, and what the cache holds before (`old`) and after that (`good`)."""

    def __init__(self, attn, gdn, page, block, dtype=BF):
        self.attn, self.gdn, self.hk = attn, gdn, 2
        self.s = Store(attn, gdn, LENS, self.hk, 64, page, block, "int8", dtype)
        xs = [rows(LENS, self.hk, 64, dtype, seed) for seed in (1, 2)]
        self.s.append(*([x[:m] for x, m in zip(y, OLD)] for y in xs), OLD)
        self.old = self.s.state()
        self.k, self.v = (torch.cat([x[m:] for x, m in zip(y, OLD)]).cuda() for y in xs)
        assert self.call() == 0
        self.good = self.s.state()

    def call(self, table=None, lens=LENS, cu=None, slots=None, ws=True, rows=None):
        """The append over what `old` holds; its error, if asked for."""
        s, c = self.s, self.s.cache
        for t, x in zip((c.k, c.v, c.k_scale, c.v_scale, c.k_tail, c.v_tail), self.old):
            t.view(x.dtype).copy_(x)
        T = len(self.k) if rows is None else rows
        s.ws.fill_(0x7f)
        self.attn.quant_append(self.k[:T], self.v[:T], c, s.table if table is None else table, ints(lens),
                               offsets(NEW) if cu is None else ints(cu), slots=s.slots if slots is None else slots,
                               ws=s.ws if ws else None)
        return self.gdn.device_error(s.ws) if ws else None

    def without(self, pages=(), slots=()):
        """`good` with these pages and tails as in `old`."""
        want = [t.clone() for t in self.good]
        for i in range(4):
            for p in pages:
                want[i][p] = self.old[i][p]
        for i in (4, 5):
            for x in slots:
                want[i][x] = self.old[i][x]
        return want

    def pages(self, n):
        return [int(p) for p in self.s.table[n] if p < self.s.cache.pages]


@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (64, 32)])
@pytest.mark.parametrize("ws", [True, False])
def test_what_a_wrong_description_leaves(attn, gdn, page, block, ws):
    f = Faulty(attn, gdn, page, block)
    s = f.s
    for bad in (-1, s.cache.pages, 10 ** 6, 2 ** 31 - 1):  # a page
        for n, j in ((1, 0), (2, 1), (0, 40 // page)):
            if j * page >= LENS[n] // block * block:
                continue  # it holds no whole block
            t = s.table.clone()
            t[n, j] = bad
            completes = (j + 1) * page > OLD[n] // block * block  # if not, the call has no block there, and does not look
            assert f.call(table=t, ws=ws) == ((7 if completes else 0) if ws else None)
            assert_state(s.state(), f.without(pages=[int(s.table[n, j])]), ("page", bad, n, j))
    for bad in (-1, s.cache.slots, 2 ** 31 - 1, -2 ** 31):  # a slot
        for n in range(3):
            sl = s.slots.clone()
            sl[n] = bad
            assert f.call(slots=sl, ws=ws) == (2 if ws else None)
            assert_state(s.state(), f.without(pages=f.pages(n), slots=[int(s.slots[n])]), ("slot", bad, n))
    for n in range(3):  # a length
        for bad in (NEW[n] - 1, 0, -1, -2 ** 31):
            lens = list(LENS)
            lens[n] = bad
            assert f.call(lens=lens, ws=ws) == (3 if ws else None)
            assert_state(s.state(), f.without(pages=f.pages(n), slots=[int(s.slots[n])]), ("length", bad, n))
    short = 32 // page  # a block table that ends before the requests do
    gone = [int(s.table[n, b]) for n in range(3) for b in range(short, len(f.pages(n)))]
    assert f.call(table=s.table[:, :short].contiguous(), ws=ws) == (7 if ws else None)
    assert_state(s.state(), f.without(pages=gone), "short table")
    assert f.call(ws=ws) == (0 if ws else None)
    assert_state(s.state(), f.good, "nothing wrong")


@pytest.mark.parametrize("ws", [True, False])
def test_wrong_offsets_write_nothing_of_others(attn, gdn, ws):
    """Pages and tails that belong to nobody stay as they were, and so does a request whose own offsets do not fit."""
    f = Faulty(attn, gdn, 16, 16)
    s, T = f.s, len(f.k)
    nobody = [p for p in range(s.cache.pages) if all(p not in f.pages(n) for n in range(3))]
    idle = [x for x in range(s.cache.slots) if x not in s.slots.tolist()]
    for cu in ([0, 35, 65, T - 10], [1, 35, 65, T], [0, 70, 65, T], [0, -5, 65, T], [0, 35, 65, 2 ** 31 - 1], [0, 0, 0, 0],
               [0, 35, 65, -2 ** 31], [T, 35, 65, 0]):
        assert f.call(cu=cu, ws=ws) == (1 if ws else None), cu
        got = s.state()
        for i in range(4):
            assert torch.equal(got[i][nobody], f.old[i][nobody]), cu
        for i in (4, 5):
            assert torch.equal(got[i][idle], f.old[i][idle]), cu
        for n in range(3):
            a, b = cu[n], cu[n + 1]
            if not 0 <= a <= b <= T:
                for i in range(4):
                    assert torch.equal(got[i][f.pages(n)], f.old[i][f.pages(n)]), (cu, n)
                for i in (4, 5):
                    assert torch.equal(got[i][int(s.slots[n])], f.old[i][int(s.slots[n])]), (cu, n)


@pytest.mark.parametrize("ws", [True, False])
def test_a_request_that_appends_nothing_is_left_alone(attn, gdn, ws):
    """Whatever its length, its slot and its pages say; the one that appends is written."""
    f = Faulty(attn, gdn, 16, 16)
    s = f.s
    t, sl = s.table.clone(), s.slots.clone()
    t[1:] = 2 ** 31 - 1
    sl[1], sl[2] = -9, 2 ** 31 - 1
    for lens in ([40, -1, 2 ** 31 - 1], [40, 20, 0]):
        assert f.call(table=t, lens=lens, cu=[0, 35, 35, 35], slots=sl, ws=ws, rows=35) == (0 if ws else None)
        assert_state(s.state(), f.without(pages=f.pages(1) + f.pages(2), slots=[int(s.slots[1]), int(s.slots[2])]), lens)
