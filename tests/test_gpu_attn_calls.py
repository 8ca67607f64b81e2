"""How the attention-layer operators take what is not a tensor's memory: numbers given as tensors."""
import pytest
import torch

from test_gpu_attn_quant_rows import BF, Store, attn, ints, offsets, rows  # noqa: F401

pytestmark = pytest.mark.gpu


def test_numbers_given_as_tensors_count_as_they_are_now(attn, gdn):
    """A scale, a window or a bound in a tensor that changes between two calls."""
    lens, hq, hk, d = [70, 33], 4, 2, 64
    ks, vs, q = rows(lens, hk, d, BF, 1), rows(lens, hk, d, BF, 2), rows([2], hq, d, BF, 3)[0].cuda()
    s = Store(attn, gdn, lens, hk, d, 32, 16, "int8", BF)
    s.append(ks, vs, lens)
    p = attn.PagedCache(s.cache.pages, 32, hk, d)
    p.k.normal_(), p.v.normal_()
    x = [rows(lens, h, d, BF, 4 + h) for h in (hq, hk, hk)]
    packed = [torch.cat(y).cuda() for y in x]
    cu = offsets(lens)
    table = s.table[:, :3].contiguous()

    def calls(**kw):
        bound = {"max_len": kw.pop("max_len")}
        out, lse = attn.window_attn(*packed, cu, **kw)
        g = attn.window_attn_bwd(*packed, out, lse, torch.ones_like(out), cu, **kw)
        norm = attn.qk_norm_rope(q, q, eps=kw["scale"])[0]
        return [attn.quant_decode(q, s.cache, table, ints(lens), slots=s.slots, **kw, **bound),
                attn.paged_decode(q, p, table, ints(lens), **kw, **bound), out, lse, g["dq"], g["dk"], g["dv"], norm]

    at = dict(scale=torch.tensor(0.1), window=torch.tensor(20), sinks=torch.tensor(2), max_len=torch.tensor(96))
    for scale, window, sinks, bound in ((0.125, 20, 2, 96), (0.5, 7, 0, 80), (0.25, 0, 5, 70)):
        for name, x in zip(at, (scale, window, sinks, bound)):
            at[name].fill_(x)
        for a, b in zip(calls(**at), calls(scale=scale, window=window, sinks=sinks, max_len=bound)):
            assert torch.equal(a, b)


def test_workspaces_that_the_kernels_could_not_write_are_refused(attn, gdn):
    """On the host, or one byte repeated: refused before anything is queued, by every call that takes one."""
    lens, hq, hk, d = [20, 33], 4, 2, 64
    q, k, v = (torch.cat(rows(lens, h, d, BF, h)).cuda() for h in (hq, hk, hk))
    s = Store(attn, gdn, lens, hk, d, 32, 16, "int8", BF)
    p = attn.PagedCache(s.cache.pages, 32, hk, d)
    cu, n, w = offsets(lens), ints(lens), torch.ones(d, device="cuda")
    out, lse = attn.window_attn(q, k, v, cu)
    calls = [lambda ws: attn.quant_append(k, v, s.cache, s.table, n, cu, slots=s.slots, ws=ws),
             lambda ws: attn.quant_read(s.cache, s.table, n, cu, sum(lens), slots=s.slots, ws=ws),
             lambda ws: attn.quant_decode(q[:2], s.cache, s.table, n, slots=s.slots, ws=ws),
             lambda ws: attn.paged_decode(q[:2], p, s.table, n, ws=ws),
             lambda ws: attn.window_attn(q, k, v, cu, ws=ws),
             lambda ws: attn.window_attn_bwd(q, k, v, out, lse, out, cu, ws=ws),
             lambda ws: attn.qk_norm_rope_bwd(q, k, q, k, q_weight=w, k_weight=w, ws=ws)]
    before = s.state()
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20)):
        for i, call in enumerate(calls):
            with pytest.raises(ValueError, match="ws is on"):
                call(ws)
    assert all(torch.equal(a, b) for a, b in zip(before, s.state()))
