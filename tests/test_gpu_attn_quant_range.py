"""Decode attention over the 8-bit cache at the ends of its range, against plain attention in 64 bits over what the cache
holds: scores that leave no fraction in fp32, values up to the type's largest, keys far from 1 in an unfinished
block."""
import pytest
import torch

import attn_ref as A
from test_gpu_attn_quant_decode import reference
from test_gpu_attn_quant_rows import BF, F32, Store, attn, expect, ints, rows  # noqa: F401

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950408889634


def decode(attn, gdn, q, ks, vs, block, code, dtype, page=32, **kw):
    """(store, out, lse) of a cache that holds the rows ks and vs, error word checked."""
    lens = [len(k) for k in ks]
    s = Store(attn, gdn, lens, ks[0].shape[1], ks[0].shape[2], max(page, block), block, code, dtype)
    s.append(ks, vs, lens)
    ws = gdn.alloc_workspace(64 << 20, "cuda")
    out, lse = attn.quant_decode(q.to(dtype).cuda(), s.cache, s.table, ints(lens), slots=s.slots, want_lse=True, ws=ws, **kw)
    assert gdn.device_error(ws) == 0
    return s, out, lse


def along(signs, c, dtype):
    """Keys c[j] times a row of signs: their products with a multiple of it are whole numbers, exact in any order."""
    return (c[:, None, None] * signs).to(dtype)


def tolerance(r, v, dtype):
    """One key has all of the weight, or several share it equally, so that sums of p and p v are exact but for the product
    with a scale, a tail's two f16 parts (2^-22 of a value, 2^-36 of the largest beside it), the division and the output's
    rounding.  A score is off by the roundings of four factors, its log-sum-exp by three more: 2^-20 of it."""
    u = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    return (u + 2.0 ** -20) * r["out"].abs() + 2.0 ** -36 * float(v.abs().max()), 2.0 ** -20 * r["lse"].abs() + 1e-30


@pytest.mark.parametrize("power", [24, 25, 26, 27, 29])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_scores_of_any_size(attn, gdn, dtype, d, code, sign, power):
    """Largest scores (times log2 e) of 2^power to 1.75 2^power of either sign: the largest wins outright, and equal ones
    share.  One key or many, in pages, in a tail or both, in one run or several."""
    g = torch.Generator().manual_seed(power)
    hk, group, lens = 2, 4, [1, 16, 17, 40, 300, 1031]
    signs = torch.randint(0, 2, (hk, d), generator=g) * 2.0 - 1
    top, low, high = (127, 1, 97) if sign > 0 else (20, 40, 128)
    ks, vs = [], rows(lens, hk, d, dtype, power)
    for n, L in enumerate(lens):
        c = torch.randint(low, high, (L,), generator=g).double()
        c[(7 * n) % L] = top
        if sign > 0 and L >= 300:  # the same key in another block, where its scale is the same
            c[L // 32 * 16 + 3] = top
        ks.append(along(signs, c, dtype))
        vs[n][:, :, ::3] = 0  # codes of 0, and
        vs[n][:, 0, 1] *= 300  # many small ones
    scale = 2.0 ** power / (LOG2E * d * top)
    q = sign * signs.repeat_interleave(group, 0) * torch.tensor([1.0, 1.25, 1.5, 1.75]).repeat(hk)[:, None]
    q = q.expand(len(lens), -1, -1)
    for window in (0, 1):
        _, out, lse = decode(attn, gdn, q, ks, vs, 16, code, dtype, scale=scale, window=window)
        for i, L in enumerate(lens):
            k, v = expect(ks[i], 16, code, F32), expect(vs[i], 16, code, F32)
            r = A.attention(q[i:i + 1], k, v, torch.tensor([L - 1]), window, 0, scale)
            to, tl = tolerance(r, v, dtype)
            assert A.worst(out[i:i + 1], r["out"], to) <= 1, (i, L, window)
            assert A.worst(lse[i:i + 1], r["lse"], tl) <= 1, (i, L, window)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_log_sum_of_one_key_is_its_score(attn, gdn, dtype, code):
    """Near 0 as well, where nothing of another size may be added to it and taken off again; in a page and in a tail."""
    d, hk, group = 64, 1, 16
    g = torch.Generator().manual_seed(3)
    signs = torch.randint(0, 2, (hk, d), generator=g) * 2.0 - 1
    lens = [1] * 16 + [16] * 16
    ks = [along(signs, torch.tensor([1.0 + n % 16] * L), dtype) for n, L in enumerate(lens)]
    vs = rows(lens, hk, d, dtype, 4)
    q = signs.expand(group, d) * ((torch.arange(group) % 8 + 1) / 8 * (1 - 2.0 * (torch.arange(group) // 8)))[:, None]
    q = q.expand(len(lens), -1, -1)
    for top in (0.01, 0.1, 1.0):
        scale = top / (16 * d)
        _, out, lse = decode(attn, gdn, q, ks, vs, 16, code, dtype, scale=scale, window=1)
        for i, L in enumerate(lens):
            k, v = expect(ks[i], 16, code, F32), expect(vs[i], 16, code, F32)
            r = A.attention(q[i:i + 1], k, v, torch.tensor([L - 1]), 1, 0, scale)
            to, tl = tolerance(r, v, dtype)
            assert A.worst(out[i:i + 1], r["out"], to) <= 1 and A.worst(lse[i:i + 1], r["lse"], tl) <= 1, (i, top)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [16, 128])
def test_values_up_to_the_largest(attn, gdn, block, dtype, code):
    """Sums over keys of equal weights pass the type's largest value, the outputs do not.  (In fp32 2^-10 is left for roundings;
    e4m3 holds 240 2^120 exactly, and the type's largest as 2^128.)"""
    top = 240 * 2.0 ** 120 if code == "e4m3" else torch.finfo(dtype).max * (1 if dtype == BF else 1 - 2.0 ** -10)
    hk, hq, d, lens = 2, 6, 64, [1, 16, 17, 100, 128, 130, 1031, 20000]
    g = torch.Generator().manual_seed(5)
    ks = rows(lens, hk, d, dtype, 6)
    for kind in range(3):
        q = rows([len(lens)], hq, d, dtype, 7)[0].float() * (0.0 if kind < 2 else 0.3)
        vs = []
        for L in lens:
            v = torch.full((L, hk, d), top, dtype=torch.float64)
            if kind:
                v *= 1 - torch.rand((L, hk, d), generator=g, dtype=torch.float64) / 2
            v[:, 1] *= -1
            if kind == 2:
                v[::2] *= -1
            vs.append(v.to(dtype))
        _, out, lse = decode(attn, gdn, q, ks, vs, block, code, dtype)
        for i, L in enumerate(lens):
            k, v = expect(ks[i], block, code, F32), expect(vs[i], block, code, F32)
            assert v.isfinite().all()
            r = reference(q[i:i + 1].to(dtype), k, v, L, dtype)
            assert A.worst(out[i:i + 1], r["out"], r["tol"]["out"]) <= 1, (kind, i, L)
            assert A.worst(lse[i:i + 1], r["lse"], r["tol"]["lse"]) <= 1, (kind, i, L)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_small_values_keep_their_bits(attn, gdn, dtype, code):
    """Down to what the cache holds as more than zeros, 2^-100, over many keys."""
    hk, hq, d, lens = 1, 3, 64, [1, 16, 100, 3000, 20000]
    ks, q = rows(lens, hk, d, dtype, 6), rows([len(lens)], hq, d, dtype, 7)[0]
    for size in (2.0 ** -100, 2.0 ** -96, 2.0 ** -80):
        vs = [(size * (1 + x.float().abs())).to(dtype) for x in rows(lens, hk, d, dtype, 8)]
        _, out, _ = decode(attn, gdn, q, ks, vs, 16, code, dtype)
        for i, L in enumerate(lens):
            k, v = (expect(x[i], 16, code, F32) for x in (ks, vs))
            # in units of 2^-60, beside which what is added to a bound for sums of 0 is nothing
            r = reference(q[i:i + 1], k, v.double() * 2.0 ** 60, L, dtype)
            assert A.worst(out[i:i + 1].double() * 2.0 ** 60, r["out"], r["tol"]["out"]) <= 1, (size, i, L)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [16, 128])
def test_keys_of_any_size(attn, gdn, block, dtype):
    """Keys far from 1 with queries that make up for it, in an unfinished block and, a token later, in a whole one."""
    hk, hq, d = 2, 6, 64
    lens = [1, 7, 15, 16, 100, 127, 128, 300]
    for fq, fk in ((1e-36, 1e36), (1e-33, 3e33), (1e34, 1e-34), (1e-35, 3e35)):
        q = (rows([len(lens)], hq, d, dtype, 9)[0].float() * fq).to(dtype)
        ks = [(x.float() * fk).to(dtype) for x in rows(lens, hk, d, dtype, 1)]
        vs = rows(lens, hk, d, dtype, 2)
        assert all(k.isfinite().all() for k in ks)
        for code in ("int8", "e4m3"):
            s, out, lse = decode(attn, gdn, q, ks, vs, block, code, dtype, page=64)
            for i, L in enumerate(lens):
                r = reference(q[i:i + 1], expect(ks[i], block, code, F32), expect(vs[i], block, code, F32), L, dtype)
                assert A.worst(out[i:i + 1], r["out"], r["tol"]["out"]) <= 1, (fq, code, i, L)
                assert A.worst(lse[i:i + 1], r["lse"], r["tol"]["lse"]) <= 1, (fq, code, i, L)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_key_that_is_not_finite_gives_nan_in_a_tail(attn, gdn, dtype):
    """Of either sign and whatever its weight would be: its request's rows, and none of the others'."""
    lens, hk, hq, d = [9, 40, 23], 2, 6, 64
    ks, vs, q = rows(lens, hk, d, dtype, 1), rows(lens, hk, d, dtype, 2), rows([3], hq, d, dtype, 3)[0]
    _, ref, _ = decode(attn, gdn, q, ks, vs, 16, "int8", dtype)
    for bad in (float("inf"), -float("inf"), float("nan")):
        for at in ([8], [2, 5]):
            bent = [k.clone() for k in ks]
            for j in at:
                bent[0][j, 1, 11] = bad
            _, out, _ = decode(attn, gdn, q, bent, vs, 16, "int8", dtype)
            assert out[0, 3:].isnan().all() and torch.equal(out[0, :3], ref[0, :3]) and torch.equal(out[1:], ref[1:])


def test_small_entries_beside_large_ones_in_an_fp32_tail(attn, gdn):
    """Columns of a value from 1e-9 to 1e9: one key's output is the value, off by the two f16 parts' 2^-22 and three roundings.  A key
    of 1e9 that has no weight: what the others give is off by their own sizes alone."""
    hk, hq, d, lens = 2, 6, 128, [1, 4, 15, 16 + 9]
    size = 10.0 ** (torch.arange(d) % 19 - 9)
    ks, vs = rows(lens, hk, d, F32, 1), [x * size for x in rows(lens, hk, d, F32, 2)]
    q = rows([len(lens)], hq, d, F32, 3)[0]
    _, out, _ = decode(attn, gdn, q, ks, vs, 16, "int8", F32, window=1)
    for i, x in enumerate(vs):
        want = x[-1].double().repeat_interleave(hq // hk, 0)
        assert A.worst(out[i], want, 2.0 ** -21 * want.abs()) <= 1, i
    q[:, :, 0] = 1.0  # the only column where the last key is not 0, and the others are
    for far in (0.0, 1e9):
        for k in ks:
            k[:, :, 0], k[-1] = 0, 0
            k[-1, :, 0] = -far
        _, out, lse = decode(attn, gdn, q, ks, vs, 16, "int8", F32)
        for i, L in enumerate(lens):
            if far and L == 1:
                continue
            keep = L - 1 if far else L
            k, v = (expect(x[i], 16, "int8", F32)[:keep] for x in (ks, vs))
            r = reference(q[i:i + 1], k, v, keep, F32)
            assert A.worst(out[i:i + 1], r["out"], r["tol"]["out"]) <= 1, (far, i)
            assert A.worst(lse[i:i + 1], r["lse"], r["tol"]["lse"]) <= 1, (far, i)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_cache_without_tails_serves_whole_blocks(attn, gdn, dtype):
    """Requests of whole blocks, with no slot; one with an unfinished block gives NaN, and its append and its rows are reported."""
    lens, hk, hq, d = [32, 48, 64], 2, 6, 64
    ks, vs, q = rows(lens, hk, d, dtype, 1), rows(lens, hk, d, dtype, 2), rows([3], hq, d, dtype, 3)[0].cuda()
    s, ref, _ = decode(attn, gdn, q.cpu(), ks, vs, 16, "int8", dtype)
    c = attn.QuantCache.wrap(s.cache.k, s.cache.v, s.cache.k_scale, s.cache.v_scale, s.cache.k_tail[:0], s.cache.v_tail[:0])
    ws = gdn.alloc_workspace(1 << 20, "cuda")
    none = ints([0, 0, 0])
    assert torch.equal(attn.quant_decode(q, c, s.table, ints(lens), slots=none, ws=ws), ref) and gdn.device_error(ws) == 0
    out = attn.quant_decode(q, c, s.table, ints([32, 47, 64]), slots=none, ws=ws)
    assert gdn.device_error(ws) == 2 and out[1].isnan().all() and torch.equal(out[::2], ref[::2])
    k, _ = attn.quant_read(c, s.table, ints([32, 47, 64]), ints([0, 32, 79, 143]), 143, slots=none, ws=ws)
    assert gdn.device_error(ws) == 2 and k[32:64].isfinite().all() and k[64:79].isnan().all() and k[79:].isfinite().all()
    before = s.state()
    new = torch.zeros((3, hk, d), dtype=dtype, device="cuda")
    attn.quant_append(new, new, c, s.table, ints([33, 49, 65]), ints([0, 1, 2, 3]), slots=none, ws=ws)
    assert gdn.device_error(ws) == 2 and all(torch.equal(a, b) for a, b in zip(before, s.state()))
