"""The 8-bit cache's rows: appended and read back.  Codes, scales and tails are whole numbers, one fp32 division or
copies, so they are compared bit for bit; a row read back is code times scale rounded to fp32 and then to the
output's type."""
import pytest
import torch

import attn_ref as A
import quant_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def attn(gdn):
    from gated_deltanet_cpr_gb300 import attn as a
    return a


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lens):
    return ints([0] + torch.tensor(lens).cumsum(0).tolist())


class Store:
    """An 8-bit cache for requests of at most `most` tokens, with pages and slots in random order."""

    def __init__(self, attn, gdn, most, hk, d, page, block, code, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.attn, self.gdn, self.code, self.block, self.page = attn, gdn, code, block, page
        blocks = [-(-n // page) for n in most]
        pages = sum(blocks) + 3
        self.cache = attn.QuantCache(pages, page, hk, d, len(most) + 2, code=code, block=block, dtype=dtype)
        for t in (self.cache.k, self.cache.v):
            t.view(torch.uint8).fill_(0x55)
        for t in (self.cache.k_scale, self.cache.v_scale, self.cache.k_tail, self.cache.v_tail):
            t.fill_(float("nan"))
        ids = torch.randperm(pages, generator=g).tolist()
        table = torch.full((len(most), max(blocks + [1]) + 1), 2 ** 31 - 1, dtype=torch.int32)
        at = 0
        for n, b in enumerate(blocks):
            table[n, :b] = torch.tensor(ids[at:at + b], dtype=torch.int32)
            at += b
        self.free = ids[at:]
        self.table = table.cuda()
        self.slots = torch.randperm(len(most) + 2, generator=g)[:len(most)].int().cuda()
        self.ws = gdn.alloc_workspace(256, "cuda")

    def append(self, ks, vs, lens, **kw):
        """ks, vs: new rows of every request; lens: lengths after."""
        new = [len(k) for k in ks]
        self.attn.quant_append(torch.cat(ks).cuda(), torch.cat(vs).cuda(), self.cache, self.table, ints(lens), offsets(new),
                               slots=self.slots, ws=self.ws, **kw)
        assert self.gdn.device_error(self.ws) == 0

    def read(self, lens, last=None, **kw):
        last = lens if last is None else last
        k, v = self.attn.quant_read(self.cache, self.table, ints(lens), offsets(last), sum(last), slots=self.slots,
                                    ws=self.ws, **kw)
        assert self.gdn.device_error(self.ws) == 0
        return k.cpu().split(list(last)), v.cpu().split(list(last))

    def state(self):
        c = self.cache
        return [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale.view(torch.int32),
                                    c.v_scale.view(torch.int32), c.k_tail.view(torch.uint8), c.v_tail.view(torch.uint8))]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def rows(lens, hk, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn((hk, d), generator=g))
    return [(torch.randn((n, hk, d), generator=g) * size).to(dtype) for n in lens]


def expect(x, block, code, dtype):
    """What reading x back gives."""
    y, _ = R.held(x, block, code)
    return y.float().to(dtype)


def check(attn, gdn, lens, hk, d, page, block, code, dtype, seed=0):
    s = Store(attn, gdn, lens, hk, d, page, block, code, dtype, seed)
    ks, vs = rows(lens, hk, d, dtype, seed), rows(lens, hk, d, dtype, seed + 1)
    before = s.state()
    s.append(ks, vs, lens)
    for out in (dtype, F32):
        k, v = s.read(lens, out_dtype=out)
        for n in range(len(lens)):
            assert torch.equal(k[n], expect(ks[n], block, code, out)), (n, lens[n])
            assert torch.equal(v[n], expect(vs[n], block, code, out)), (n, lens[n])
    # the pages' scales, and everything that no whole block covers as it was
    touched = torch.zeros(s.cache.k_scale.shape, dtype=torch.bool)
    scales = s.cache.k_scale.cpu()
    table = s.table.cpu()
    for n, x in enumerate(ks):
        _, sc = R.held(x, block, code)
        for b in range(len(x) // block):
            p, j = int(table[n, b * block // page]), b % (page // block)
            assert torch.equal(scales[p, :, j], sc[b])
            touched[p, :, j] = True
    keep = ~touched.cuda()
    after = s.state()
    for i in (0, 1):
        assert torch.equal(after[i].view(*keep.shape, block, d)[keep], before[i].view(*keep.shape, block, d)[keep])
        assert torch.equal(after[2 + i][keep], before[2 + i][keep])
    # the tails: rows of the unfinished blocks, and nothing else
    tail = s.cache.k_tail.cpu()
    for n, x in enumerate(ks):
        t = tail[int(s.slots[n])]
        r = len(x) % block
        assert torch.equal(t[:, :r].transpose(0, 1), x[len(x) - r:]) and t[:, r:].isnan().all()
    return s


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page,block", [(32, 16, 16), (64, 32, 16), (128, 64, 32), (64, 256, 128), (128, 64, 64), (32, 128, 128),
                                          (128, 16, 16)])
def test_append_and_read(attn, gdn, d, page, block, dtype, code):
    """Empty requests, one token, lengths beside a block's and a page's end."""
    check(attn, gdn, [0, 1, 15, 16, 17, 0, 127, 128, 129, 300], 3, d, page, block, code, dtype)


def ties(dtype, code, d):
    """Blocks [., 16, 1, d] whose quotients lie on and beside the middle between two codes."""
    out = []
    for scale in (1.0, 2.0 ** -96, 2.0 ** 119, 0.75, 1.9375):
        for m in (127.0, 126.5, 101.0, 64.0, 254.0):
            m = torch.tensor(m * scale, dtype=dtype)
            k = torch.arange(16 * d) % 255 - 127.5
            x = (k.to(R.D) * m.to(R.D) / 127).to(dtype)  # the middles, and what lies next to them in the type
            bits = torch.int16 if dtype == BF else torch.int32
            n = torch.arange(16 * d) // 255 % 3 - 1
            x = (x.view(bits) + n.to(bits)).view(dtype)
            x = torch.where(x.abs() > m.abs(), m, x)
            x[0] = m
            out.append(x.view(16, 1, d))
    if code == "e4m3":
        for e in (0, 1, -30):
            k = torch.arange(16 * d)
            x = ((8 + k % 8).to(R.D) + 0.5) * 2.0 ** (k // 8 % 17 - 12 + e)  # middles of every binade
            x[0] = 448 * 2.0 ** e
            out.append(x.to(dtype).view(16, 1, d))
    return torch.cat(out)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_ties_go_to_even(attn, gdn, dtype, code):
    for d in (32, 128):
        x = ties(dtype, code, d)
        s = Store(attn, gdn, [len(x)], 1, d, 64, 16, code, dtype)
        s.append([x], [-x], [len(x)])
        k, v = s.read([len(x)], out_dtype=F32)
        ref = expect(x, 16, code, F32)
        assert torch.equal(k[0], ref) and torch.equal(v[0], -ref)


def test_every_bf16_value_under_every_largest(attn, gdn):
    """Quotients depend on the two significands and the gap of the exponents: 128 largest values, 128 values and 10 gaps, after
    which all of them round to 0; the codes themselves are compared."""
    sig = torch.arange(128, 256, dtype=R.D)
    x = torch.zeros((128, 16, 128), dtype=R.D)
    for i, m in enumerate(sig):
        v = torch.cat([sig * 2.0 ** -gap for gap in range(10)])
        v = v[v <= m]
        x[i].view(-1)[:len(v)] = v
        x[i].view(-1)[-1] = m
    x = x.view(-1, 1, 128)
    assert torch.equal(x.to(BF).to(R.D), x)
    for scale in (1.0, 2.0 ** -100, 2.0 ** 119):
        b = (x * scale).to(BF)
        s = Store(attn, gdn, [len(b)], 1, 128, 64, 16, "int8", BF)
        s.append([b], [-b], [len(b)])
        pages = s.table[0, :len(b) // 64].long()
        c, _ = R.quantise(b.view(128, 1, 16, 128), "int8")
        assert torch.equal(s.cache.k[pages].cpu().view(-1).to(R.D), c.view(-1))
        assert torch.equal(s.cache.v[pages].cpu().view(-1).to(R.D), -c.view(-1))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_extreme_blocks(attn, gdn, dtype, code):
    """Zeros, values below 2^-100, next to it, subnormal beside ordinary, the type's largest, infinities and NaN."""
    big, inf, nan = torch.finfo(dtype).max, float("inf"), float("nan")
    for block in (16, 64):
        tops = [0.0, 2.0 ** -140, 2.0 ** -100 * 0.99, 2.0 ** -100, 1e-20, 1.0, 1e30, big, inf, -inf, nan, 3.0]
        x = torch.randn((len(tops), block, 2, 64), generator=torch.Generator().manual_seed(1)).clamp(-1, 1) * 0.9
        for i, t in enumerate(tops):
            x[i, :, 0] *= abs(t) if t == t and abs(t) < inf else 1.0
            x[i, 3, 0, 5] = t
            x[i, 4, 0, 7] = 1e-39
        x = x.view(-1, 2, 64).to(dtype)
        s = Store(attn, gdn, [len(x)], 2, 64, 64, block, code, dtype)
        s.append([x], [x], [len(x)])
        k, _ = s.read([len(x)], out_dtype=F32)
        ref = expect(x, block, code, F32)
        assert torch.equal(k[0].isnan(), ref.isnan()) and torch.equal(k[0].nan_to_num(7.0), ref.nan_to_num(7.0))
        assert ref.view(len(tops), block, 2, 64)[8:11, :, 0].isnan().all() and ref.view(len(tops), block, 2, 64)[:, :, 1].isfinite().all()


@pytest.mark.parametrize("code,dtype,d,page,block", [("int8", BF, 128, 64, 16), ("e4m3", BF, 64, 32, 32), ("int8", F32, 32, 128, 128),
                                                     ("e4m3", F32, 128, 64, 64)])
def test_how_tokens_are_split_over_calls_does_not_matter(attn, gdn, code, dtype, d, page, block):
    """Chunks that end inside a block, complete one and begin another, and single tokens leave the same bits."""
    lens = [3 * block + 5, 1, 2 * block, 7 * block + block // 2, 0]
    ks, vs = rows(lens, 2, d, dtype, 5), rows(lens, 2, d, dtype, 6)
    whole = Store(attn, gdn, lens, 2, d, page, block, code, dtype, 3)
    whole.append(ks, vs, lens)
    g = torch.Generator().manual_seed(9)
    for most in (1, 7, block - 1, block + 1, 3 * block):
        s = Store(attn, gdn, lens, 2, d, page, block, code, dtype, 3)
        at = [0] * len(lens)
        while at != lens:
            step = [min(L - a, int(torch.randint(0, most + 1, (1,), generator=g))) for a, L in zip(at, lens)]
            to = [a + b for a, b in zip(at, step)]
            s.append([k[a:b] for k, a, b in zip(ks, at, to)], [v[a:b] for v, a, b in zip(vs, at, to)], to)
            at = to
        a, b = s.state(), whole.state()
        assert same(a[:4], b[:4])
        for n, L in enumerate(lens):  # rows past a tail's end may hold what was there
            r, slot = L % block, int(s.slots[n])
            assert torch.equal(s.cache.k_tail[slot, :, :r], whole.cache.k_tail[slot, :, :r])
            assert torch.equal(s.cache.v_tail[slot, :, :r], whole.cache.v_tail[slot, :, :r])


def test_strided_tokens(attn, gdn):
    """k and v as parts of one projection's rows."""
    for dtype in (BF, F32):
        x = rows([200], 6, 64, dtype, 2)[0]
        q, k, v = x.cuda().split([2, 2, 2], 1)
        s = Store(attn, gdn, [200], 2, 64, 32, 16, "int8", dtype)
        attn.quant_append(k, v, s.cache, s.table, ints([200]), ints([0, 200]), slots=s.slots, ws=s.ws)
        kr, vr = s.read([200])
        assert torch.equal(kr[0], expect(x[:, 2:4].contiguous(), 16, "int8", dtype))
        assert torch.equal(vr[0], expect(x[:, 4:].contiguous(), 16, "int8", dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_the_last_rows(attn, gdn, dtype):
    lens = [0, 5, 33, 200, 131, 64, 16]
    s = check(attn, gdn, lens, 2, 64, 32, 32, "int8", dtype)
    k, v = s.read(lens)
    for last in ([0] * 7, [0, 1, 1, 1, 1, 1, 1], [0, 5, 2, 17, 4, 33, 0], [0, 0, 33, 199, 131, 0, 15]):
        ka, va = s.read(lens, last)
        for n in range(7):
            assert torch.equal(ka[n], k[n][lens[n] - last[n]:]) and torch.equal(va[n], v[n][lens[n] - last[n]:])
    a, b = torch.empty((33, 2, 64), device="cuda"), torch.empty((33, 2, 64), device="cuda")
    only = attn.quant_read(s.cache, s.table, ints(lens), offsets([0, 0, 33, 0, 0, 0, 0]), 33, slots=s.slots, k_out=a, v_out=b)
    assert only[0] is a and torch.equal(a.cpu().to(dtype), k[2]) and torch.equal(b.cpu().to(dtype), v[2])


def test_many_requests(attn, gdn):
    """More requests than one round of the search tells apart, most with one token or none."""
    lens = [(n * 37) % 41 for n in range(1500)]
    check(attn, gdn, lens, 1, 32, 16, 16, "int8", BF)
    new = [int(n % 3 > 0 and L > 0) for n, L in enumerate(lens)]
    s = Store(attn, gdn, lens, 1, 32, 16, 16, "int8", BF, 1)
    ks, vs = rows(lens, 1, 32, BF, 1), rows(lens, 1, 32, BF, 2)
    s.append([k[:L - m] for k, L, m in zip(ks, lens, new)], [v[:L - m] for v, L, m in zip(vs, lens, new)],
             [L - m for L, m in zip(lens, new)])
    s.append([k[L - m:] for k, L, m in zip(ks, lens, new)], [v[L - m:] for v, L, m in zip(vs, lens, new)], lens)
    k, v = s.read(lens)
    assert all(torch.equal(k[n], expect(ks[n], 16, "int8", BF)) and torch.equal(v[n], expect(vs[n], 16, "int8", BF))
               for n in range(len(lens)))


def test_bad_descriptions_are_reported(attn, gdn):
    """The others' rows are written, and nothing outside them."""
    lens = [40, 50, 70]
    ks, vs = rows(lens, 2, 64, BF, 1), rows(lens, 2, 64, BF, 2)
    k, v = torch.cat(ks).cuda(), torch.cat(vs).cuda()

    def call(table=None, seq=None, cu=None, slots=None):
        s = Store(attn, gdn, lens, 2, 64, 16, 16, "int8", BF)
        empty = s.state()
        s.append(ks, vs, lens)
        good = s.state()
        c = s.cache
        for t, x in zip((c.k, c.v, c.k_scale, c.v_scale, c.k_tail, c.v_tail), empty):
            t.view(x.dtype).copy_(x)
        t = s.table.clone()
        if table:
            t[table[0], table[1]] = table[2]
        seq_t, cu_t = ints(seq or lens), ints(cu or [0, 40, 90, 160])
        sl = s.slots.clone()
        if slots:
            sl[slots[0]] = slots[1]
        attn.quant_append(k, v, c, t, seq_t, cu_t, slots=sl, ws=s.ws)
        err = gdn.device_error(s.ws)
        for dst, x in zip((c.k, c.v, c.k_scale, c.v_scale, c.k_tail, c.v_tail), good):
            dst.view(x.dtype).copy_(x)  # read from what is there
        kr, vr = attn.quant_read(c, t, seq_t, cu_t, 160, slots=sl, ws=s.ws)
        return err, gdn.device_error(s.ws), kr.cpu()

    ref = torch.cat([expect(x, 16, "int8", BF) for x in ks])
    for page in (-1, 10 ** 6, 2 ** 31 - 1):
        e, e2, kr = call(table=(1, 2, page))
        assert e == e2 == 7
        assert kr[40 + 32:40 + 48].isnan().all() and torch.equal(kr[:72], ref[:72]) and torch.equal(kr[88:], ref[88:])
    for slot in (-1, 5, 2 ** 31 - 1):
        e, e2, kr = call(slots=(2, slot))
        assert e == e2 == 2
        assert torch.equal(kr[:90 + 64], ref[:90 + 64]) and kr[154:].isnan().all()
    for L in (49, 0, -7):
        e, e2, kr = call(seq=[40, L, 70])
        assert e == e2 == 3
        assert torch.equal(kr[:40], ref[:40]) and kr[40:90].isnan().all() and torch.equal(kr[90:], ref[90:])
    for cu in ([0, 40, 90, 150], [1, 40, 90, 160], [0, 95, 90, 160], [0, -5, 90, 160], [0, 40, 90, 2 ** 31 - 1], [0, 0, 0, 0]):
        assert call(cu=cu)[:2] == (1, 1), cu
    # block tables shorter than the lengths
    s = Store(attn, gdn, lens, 2, 64, 16, 16, "int8", BF)
    short = s.table[:, :2].contiguous()
    attn.quant_append(k, v, s.cache, short, ints(lens), ints([0, 40, 90, 160]), slots=s.slots, ws=s.ws)
    assert gdn.device_error(s.ws) == 7
    # a request that appends nothing is left alone, whatever its entries
    s = Store(attn, gdn, lens, 2, 64, 16, 16, "int8", BF)
    sl = s.slots.clone()
    sl[1] = -9
    attn.quant_append(k[:40], v[:40], s.cache, s.table, ints([40, -1, 70]), ints([0, 40, 40, 40]), slots=sl, ws=s.ws)
    assert gdn.device_error(s.ws) == 0


def test_empty_calls(attn, gdn):
    s = Store(attn, gdn, [20], 1, 32, 16, 16, "int8", BF)
    z = torch.zeros((0, 1, 32), dtype=BF, device="cuda")
    s.ws.fill_(0x7f)
    attn.quant_append(z, z, s.cache, s.table[:0], ints([]), ints([0]), ws=s.ws)
    assert gdn.device_error(s.ws) == 0
    s.ws.fill_(0x7f)
    attn.quant_append(z, z, s.cache, s.table, ints([20]), ints([0, 0]), slots=s.slots, ws=s.ws)
    assert gdn.device_error(s.ws) == 0
    s.ws.fill_(0x7f)
    k, v = attn.quant_read(s.cache, s.table, ints([20]), ints([0, 0]), 0, slots=s.slots, ws=s.ws)
    assert gdn.device_error(s.ws) == 0 and k.shape == v.shape == (0, 1, 32)


def test_offsets_past_32_bits(attn, gdn):
    """Pages past 2^32 bytes, and tails past 2^31 elements."""
    page, d, hk, block = 256, 128, 8, 128
    pages = 2 ** 32 // (page * d * hk) + 9
    slots = 2 ** 31 // (block * d * hk) + 5
    k, v = (torch.zeros((pages, hk, page, d), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, hk, page // block), device="cuda") for _ in range(2))
    kt, vt = (torch.zeros((slots, hk, block, d), dtype=BF, device="cuda") for _ in range(2))
    c = attn.QuantCache.wrap(k, v, ks, vs, kt, vt)
    x, y = rows([600], hk, d, BF, 1)[0], rows([600], hk, d, BF, 2)[0]
    table, slot = ints([[pages - 1, pages - 3, pages - 2]]), ints([slots - 1])
    attn.quant_append(x.cuda(), y.cuda(), c, table, ints([600]), ints([0, 600]), slots=slot)
    kr, vr = attn.quant_read(c, table, ints([600]), ints([0, 600]), 600, slots=slot)
    assert torch.equal(kr.cpu(), expect(x, block, "int8", BF)) and torch.equal(vr.cpu(), expect(y, block, "int8", BF))


def test_captured_and_on_another_stream(attn, gdn):
    """A graph that appends a token per replay, from lengths that the caller moves on."""
    lens = [13, 31, 64]
    most = [60, 60, 100]
    s = Store(attn, gdn, most, 2, 128, 32, 16, "e4m3", BF)
    ks, vs = rows(most, 2, 128, BF, 1), rows(most, 2, 128, BF, 2)
    s.append([k[:n] for k, n in zip(ks, lens)], [v[:n] for v, n in zip(vs, lens)], lens)
    k, v = (torch.empty((3, 2, 128), dtype=BF, device="cuda") for _ in range(2))
    n, cu = ints(lens), ints([0, 1, 2, 3])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            n += 1
            attn.quant_append(k, v, s.cache, s.table, n, cu, slots=s.slots, ws=s.ws)
        for step in range(25):
            at = [a + step for a in lens]
            k.copy_(torch.stack([x[a] for x, a in zip(ks, at)]))
            v.copy_(torch.stack([x[a] for x, a in zip(vs, at)]))
            g.replay()
    torch.cuda.synchronize()
    now = [a + 25 for a in lens]
    kr, vr = s.read(now)
    for i, m in enumerate(now):
        assert torch.equal(kr[i], expect(ks[i][:m], 16, "e4m3", BF)) and torch.equal(vr[i], expect(vs[i][:m], 16, "e4m3", BF))


def test_continued_prefill(attn, gdn):
    """page_map, append and read together, and window_attn over what was read: prompts in chunks, each against plain
    attention over what the cache holds then (tolerances: see attn_ref)."""
    hk, hq, d, page, block = 2, 4, 64, 16, 16
    lens, chunks = [90, 37, 128], [[48, 0, 64], [13, 37, 0], [29, 0, 64]]
    qs = rows(lens, hq, d, BF, 4)
    ks, vs = rows(lens, hk, d, BF, 5), rows(lens, hk, d, BF, 6)
    pages = sum(-(-n // page) for n in lens)
    c = attn.QuantCache(pages, page, hk, d, 3, block=block)
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int().cuda()
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    n, at = ints([0, 0, 0]), [0, 0, 0]
    for new in chunks:
        q, k, v = (torch.cat([x[a:a + m] for x, a, m in zip(xs, at, new)]).cuda() for xs in (qs, ks, vs))
        m = attn.page_map(n, ints(new), free, table, page, sum(new))
        assert gdn.device_error(m["ws"]) == 0
        free, n = free[int(m["pages_used"]):].clone(), m["seq_lens"]
        at = [a + b for a, b in zip(at, new)]
        attn.quant_append(k, v, c, table, n, m["cu_seqlens"])
        cu_k = offsets(at)
        k, v = attn.quant_read(c, table, n, cu_k, sum(at))
        o, _ = attn.window_attn(q, k, v, m["cu_seqlens"], cu_seqlens_k=cu_k)
        for i, x in enumerate(o.split(new)):
            L, b = at[i], new[i]
            r = A.attention(qs[i][L - b:L], expect(ks[i][:L], block, "int8", BF), expect(vs[i][:L], block, "int8", BF),
                            torch.arange(L - b, L), u=2.0 ** -8)
            assert not b or A.worst(x, r["out"], r["tol"]["out"]) <= 1, (new, i)
