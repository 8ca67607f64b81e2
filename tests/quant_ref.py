"""Plain form of the 8-bit cache for the tests, in 64 bits on the CPU, from the formulas: a request is the list of
its rows; its whole blocks are held as codes and a scale, the rest as it came."""
import torch

D = torch.float64
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def e4m3_values():
    """Every finite value of the format with its code, ascending."""
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(D)
    keep = v.isfinite()
    codes = torch.arange(256)[keep]
    v = v[keep]
    order = torch.argsort(v, stable=True)
    return v[order], codes[order]


def nearest_e4m3(y):
    """Nearest value of the format, by comparison with its neighbours; a tie goes to the even code."""
    v, codes = e4m3_values()
    keep = torch.ones(len(v), dtype=torch.bool)
    keep[1:] = v[1:] != v[:-1]  # one zero
    v, codes = v[keep], codes[keep]
    hi = torch.searchsorted(v, y.contiguous()).clamp(1, len(v) - 1)
    lo = hi - 1
    a, b = y - v[lo], v[hi] - y
    up = (b < a) | ((a == b) & (codes[hi] % 2 == 0))
    return torch.where(up, v[hi], v[lo])


def quantise(x, code):
    """Blocks x [..., block, d] -> (codes as 64-bit values, scales fp32)."""
    m = x.to(D).abs().flatten(-2).amax(-1)
    finite = m.isfinite()
    some = finite & (m >= 2.0 ** -100)
    one = torch.where(some, m, 1.0)
    if code == "int8":
        # the products and the quotients below are exact or far from a tie: 127 x has at most 31 bits
        c = torch.round(127 * x.to(D) / one[..., None, None])
        s = (one.float() / 127)
    else:
        e = torch.floor(torch.log2(one)) - 9
        while bool((one > 448 * 2.0 ** e).any()):
            e = torch.where(one > 448 * 2.0 ** e, e + 1, e)
        s = (2.0 ** e).float()
        c = nearest_e4m3(torch.where(some[..., None, None], x.to(D) / s.to(D)[..., None, None], 0.0))
    c = torch.where(some[..., None, None], c, 0.0)
    s = torch.where(some, s, torch.where(finite, 0.0, float("nan")))
    return c, s


def held(rows, block, code):
    """What a request's rows [L, H, d] are held as, 64 bits, and the scales [blocks, H] of its whole blocks."""
    L, H, d = rows.shape
    w = L // block * block
    c, s = quantise(rows[:w].view(-1, block, H, d).transpose(1, 2), code)
    y = c * s.to(D)[..., None, None]
    return torch.cat([y.transpose(1, 2).reshape(w, H, d), rows[w:].to(D)]), s
