"""A two-layer hybrid model's attention part, end to end on the library's operators: a Gated
DeltaNet layer and a sliding-window attention layer with first tokens that stay visible, in
prefill, decode and training.

    python examples/hybrid_layer.py

Serving: page_map hands out cache pages; prefill runs both layers over the packed prompts and
fills the recurrent and the paged cache; decode steps continue every request and are checked
against one prefill of the whole text.  Training: forward and backward through both layers'
operators.  Weights and inputs are random.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_deltanet_cpr_gb300 import api, attn  # noqa: E402

HQ, HKV, D, CHUNK = 8, 2, 128, 64  # attention heads and their size; the recurrence uses HQ / 2 and HQ heads
WIDTH, WINDOW, SINKS, PAGE = 512, 96, 4, 16
BF = torch.bfloat16


class Hybrid:
    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def w(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[0] ** -0.5).to(BF)

        self.gdn_in = w(WIDTH, (HQ // 2 * 2 + HQ) * D)
        self.gdn_gate = w(WIDTH, 2 * HQ)
        self.gdn_out = w(HQ * D, WIDTH)
        self.qkv = w(WIDTH, (HQ + 2 * HKV) * D)
        self.out = w(HQ * D, WIDTH)
        self.q_weight = 1 + 0.1 * torch.randn(D, generator=g, device=device)
        self.k_weight = 1 + 0.1 * torch.randn(D, generator=g, device=device)
        self.cos, self.sin = attn.rope_tables(4096, D // 2)

    def gdn_inputs(self, x):
        """q, k (L2-normalised per head), v, log decay and beta of the recurrence."""
        T = x.shape[0]
        q, k, v = (x @ self.gdn_in).view(T, -1, D).split([HQ // 2, HQ // 2, HQ], 1)
        qn, kn = attn.qk_norm_rope(q, k, norm="l2")
        gate, beta = (x @ self.gdn_gate).float().split(HQ, 1)
        return q, k, qn, kn, v.contiguous(), (-0.1 * torch.sigmoid(gate)).contiguous(), torch.sigmoid(beta).contiguous()

    def qkv_of(self, x):
        return (x @ self.qkv).view(x.shape[0], -1, D).split([HQ, HKV, HKV], 1)

    def norm(self):
        return dict(norm="rms", q_weight=self.q_weight, k_weight=self.k_weight, cos=self.cos, sin=self.sin)

    # ------------------------------------------------------------------ serving ----
    def prefill(self, x, lens, rec, slots, cache, table, free):
        """Packed prompts through both layers; fills the caches.  Returns (outputs, lengths, pages taken)."""
        m = attn.page_map(torch.zeros_like(lens), lens, free, table, PAGE, x.shape[0])
        if api.device_error(m["ws"]):
            raise RuntimeError(api.DEVERR[api.device_error(m["ws"])])
        cu = m["cu_seqlens"]
        _, _, q, k, v, g, beta = self.gdn_inputs(x)
        o, _ = api.prefill(q, k, v, g, beta, cu, chunk=CHUNK, cache=rec, slot_of_seq=slots)
        x = x + o.view(x.shape[0], -1) @ self.gdn_out
        q, k, v = self.qkv_of(x)
        q, k = attn.qk_norm_rope(q, k, v, positions=m["positions"], cache=cache, slot_map=m["slot_map"], **self.norm())
        o, _ = attn.window_attn(q, k, v.contiguous(), cu, window=WINDOW, sinks=SINKS)
        return x + o.view(x.shape[0], -1) @ self.out, m["seq_lens"], m["pages_used"]

    def decode(self, x, lens, rec, slots, cache, table, free):
        """One token per request."""
        m = attn.page_map(lens, torch.ones_like(lens), free, table, PAGE, x.shape[0])
        _, _, q, k, v, g, beta = self.gdn_inputs(x)
        o = api.decode_step(q, k, v, g, beta, slots, rec)
        x = x + o.view(x.shape[0], -1) @ self.gdn_out
        q, k, v = self.qkv_of(x)
        q, _ = attn.qk_norm_rope(q, k, v, positions=m["positions"], cache=cache, slot_map=m["slot_map"], want_k=False,
                                 **self.norm())
        o = attn.paged_decode(q, cache, table, m["seq_lens"], window=WINDOW, sinks=SINKS)
        return x + o.view(x.shape[0], -1) @ self.out, m["seq_lens"], m["pages_used"]

    # ----------------------------------------------------------------- training ----
    def train(self, x, cu, positions, dout):
        """Forward, and the gradient of <dout, output> with respect to x and the norm weights."""
        T = x.shape[0]
        gq, gk, qn, kn, v, g, beta = self.gdn_inputs(x)
        o1, _, saved = api.fwd(qn, kn, v, g, beta, cu, chunk=CHUNK)
        x1 = x + o1.view(T, -1) @ self.gdn_out
        q, k, va = self.qkv_of(x1)
        qr, kr = attn.qk_norm_rope(q, k, positions=positions, **self.norm())
        va = va.contiguous()
        o2, lse = attn.window_attn(qr, kr, va, cu, window=WINDOW, sinks=SINKS)
        y = x1 + o2.view(T, -1) @ self.out

        do2 = (dout @ self.out.T).view_as(o2)
        a = attn.window_attn_bwd(qr, kr, va, o2, lse, do2, cu, window=WINDOW, sinks=SINKS)
        n = attn.qk_norm_rope_bwd(q, k, a["dq"], a["dk"], positions=positions, **self.norm())
        dx1 = dout + torch.cat([n["dq"], n["dk"], a["dv"]], 1).view(T, -1) @ self.qkv.T
        r = api.bwd(qn, kn, v, g, beta, cu, saved, (dx1 @ self.gdn_out.T).view_as(o1), chunk=CHUNK)
        n1 = attn.qk_norm_rope_bwd(gq, gk, r["dq"], r["dk"], norm="l2")
        gate = torch.cat([r["dg"] * g * (1 + 10 * g), r["dbeta"] * beta * (1 - beta)], 1).to(BF)  # g = -0.1 sigmoid
        dx = dx1 + torch.cat([n1["dq"], n1["dk"], r["dv"].to(BF)], 1).view(T, -1) @ self.gdn_in.T + gate @ self.gdn_gate.T
        return y, dx, n["dq_weight"], n["dk_weight"]


def serve_check(model, lens=(150, 37, 1, 210), steps=24):
    """The largest difference between decoded outputs and one prefill of the whole text, over its size."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(1)
    total = [n + steps for n in lens]
    text = [torch.randn((n, WIDTH), generator=g, device=dev).to(BF) for n in total]
    slots = torch.arange(len(lens), dtype=torch.int32, device=dev)

    def caches():
        pages = sum(-(-n // PAGE) for n in total) + 4
        rec = api.Cache(len(lens), HQ // 2, HQ, D, CHUNK)
        free = torch.randperm(pages, generator=g, device=dev).int()
        return rec, attn.PagedCache(pages, PAGE, HKV, D), torch.full((len(lens), 32), -1, dtype=torch.int32, device=dev), free

    rec, cache, table, free = caches()
    whole, _, _ = model.prefill(torch.cat(text), torch.tensor(total, dtype=torch.int32, device=dev), rec, slots, cache, table, free)
    whole = whole.split(total)
    rec, cache, table, free = caches()
    y, cur, used = model.prefill(torch.cat([t[:n] for t, n in zip(text, lens)]),
                                 torch.tensor(lens, dtype=torch.int32, device=dev), rec, slots, cache, table, free)
    free = free[int(used):]
    worst = 0.0
    for s in range(steps):
        x = torch.stack([t[n + s] for t, n in zip(text, lens)])
        y, cur, used = model.decode(x, cur, rec, slots, cache, table, free)
        free = free[int(used):]
        ref = torch.stack([w[n + s] for w, n in zip(whole, lens)])
        worst = max(worst, float((y.float() - ref.float()).abs().max() / ref.float().abs().max()))
    return worst


def train_check(model, lens=(130, 64, 200)):
    """Gradient along a direction against the difference of two forward passes: (gradient, difference)."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(2)
    T = sum(lens)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=dev)
    pos = torch.cat([torch.arange(n) for n in lens]).int().to(dev)
    x = torch.randn((T, WIDTH), generator=g, device=dev).to(BF)
    dout = torch.randn((T, WIDTH), generator=g, device=dev).to(BF)
    _, dx, _, _ = model.train(x, cu, pos, dout)
    e = dx.float() / dx.float().norm()  # along the gradient itself, where the difference is largest
    h = 0.02 * float(x.float().norm())
    f = [float((model.train((x.float() + s * h * e).to(BF), cu, pos, dout)[0].double() * dout).sum()) for s in (1, -1)]
    return float((dx.float() * e).sum()), (f[0] - f[1]) / (2 * h)


if __name__ == "__main__":
    m = Hybrid()
    print(f"decode against prefill: {serve_check(m):.2e} of the largest output")
    a, b = train_check(m)
    print(f"gradient {a:.4e}, difference {b:.4e}")
