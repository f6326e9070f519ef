"""Shared by the tests of the 4-bit cache: a plain implementation in 64 bits,
written from the formulas, and device state whose unused slots hold NaN scales,
so that a stray read shows.

Codes are compared for equality: the writes round the exact value, and the
64-bit one here is off by under 2^-44 (the fp32 epsilon), so that the two differ only where a
value lies that near to a border, which no test's does."""

from __future__ import annotations

import torch

from paged_kv_gqa_16_gb300 import pkv

import q8_cases
from q8_cases import DEV

GROUP = 32
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantise(x):
    """x [..., D] in 64 bits: (codes [..., D], scale bytes [..., D / 32])."""
    x = x.double().unflatten(-1, (-1, GROUP))
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(amax) | torch.isnan(x).any(-1)
    e = torch.where((amax > 0) & ~bad, torch.ceil(torch.log2(amax / 6)), torch.full_like(amax, -40.0))
    e = e.clamp(-40, 40)
    size = torch.where(bad[..., None], 0.0, x.abs()) * torch.exp2(-e)[..., None]
    # the distance to every value; of two as near, the even code
    off = (size.clamp(max=6.0)[..., None] - GRID).abs()
    best = off.amin(-1, keepdim=True)
    near = off == best
    even = near & (torch.arange(8) % 2 == 0)
    code = torch.where(even.any(-1), even.int().argmax(-1), near.int().argmax(-1))
    code = torch.where(bad[..., None], 0, code + 8 * torch.signbit(x).int())
    return code.flatten(-2).to(torch.uint8), torch.where(bad, 255.0, e + 127).to(torch.uint8)


def values(codes, scale):
    """Codes [..., D] and scale bytes [..., D / 32] as what they stand for, in 64 bits."""
    x = torch.where(codes >= 8, -1.0, 1.0) * GRID[(codes & 7).long()]
    s = torch.exp2(scale.double() - 127)
    s = torch.where(scale == 255, float("nan"), s)
    return (x.double().unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def unpacked(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def packed(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def bf16_of(x):
    """64-bit values rounded once to bf16 (the codes' values fit it)."""
    return x.to(torch.float32).to(torch.bfloat16)


class Cache(q8_cases.Cache):
    """Rows of a 4-bit cache over scattered pages, beside the bf16 pools; every
    slot starts with NaN scales."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        heads = (self.n_pool, self.ps, self.Hkv)
        self.kc, self.vc = (torch.full((*heads, self.D // 2), 0x77, dtype=torch.uint8, device=DEV) for _ in range(2))
        self.ks, self.vs = (torch.full((*heads, self.D // GROUP), 255, dtype=torch.uint8, device=DEV)
                            for _ in range(2))

    @property
    def q4(self):
        return self.kc, self.vc, self.ks, self.vs

    def fill(self, k_gain=(-3, 1), v_gain=(-3, 1)):
        """Random codes and scales for every row's tokens (gains: the range of the
        scales' exponents)."""
        for c, s, (lo, hi) in ((self.kc, self.ks, k_gain), (self.vc, self.vs, v_gain)):
            codes, scale = c.cpu(), s.cpu()
            for b, L in enumerate(self.lens):
                if L:
                    at = self.places(b, 0, L)
                    codes[at] = torch.randint(0, 256, (L, self.Hkv, self.D // 2), generator=self.g).to(torch.uint8)
                    scale[at] = torch.randint(lo + 127, hi + 128, (L, self.Hkv, self.D // GROUP),
                                              generator=self.g).to(torch.uint8)
            c.copy_(codes)
            s.copy_(scale)
        return self

    def stored(self, b, first, last):
        """Codes and scale bytes of row b's tokens, K then V, on the CPU."""
        at = self.places(b, first, last)
        kc, vc, ks, vs = (x.cpu()[at] for x in self.q4)
        return unpacked(kc), ks, unpacked(vc), vs

    def held(self, b, L=None):
        kc, ks, vc, vs = self.stored(b, 0, self.lens[b] if L is None else L)
        return values(kc, ks), values(vc, vs)


# --------------------------------------------------------------- the attention
def seen(L, window=0, sinks=0):
    """Positions that a row's last token sees."""
    t = torch.arange(L)
    return t if window == 0 else t[(t >= L - window) | (t < sinks)]


def attention(q, k, v, scale, weight_eps, v_top=None):
    """q [Hq, D], k and v [n, Hkv, D] (what is seen): the output [Hq, D] in 64 bits
    and its bound: the output's rounding (2^-8), the weights' (weight_eps of each,
    in the sum too) against sum_t w_t |v_t|, and the scores' error (128 products and
    sums of 2^-23 each at most, so under 2^-16 of sum |q k|, twice in the weights
    and their sum).  v_top [n, Hkv] (4 bits): the largest scale of each token's
    values.  A weight times its values' scale goes to f16 with the row's largest such
    product W at 2^7 or more; f16 ends in steps of 2^-24, so one is off by up to
    2^-25, 2^-32 W, where that is more than 2^-11 of it: times codes of up to 6."""
    Hq, D = q.shape
    Hkv = k.shape[1]
    q = q.double().view(Hkv, Hq // Hkv, D)
    x = torch.einsum("grd,lgd->grl", q, k) * scale
    w = torch.softmax(x, -1)
    out = torch.einsum("grl,lgd->grd", w, v)
    size = torch.einsum("grl,lgd->grd", w, v.abs())
    far = torch.einsum("grd,lgd->grl", q.abs(), k.abs()).amax(-1, keepdim=True) * scale * 2.0 ** -16
    bound = out.abs() * 2.0 ** -8 + size * (2 * weight_eps + 2 * far) + 1e-30
    if v_top is not None:
        top = (w * v_top.T[:, None]).amax(-1, keepdim=True)
        bound = bound + 2.0 ** -32 * top * 6 * len(k)
    return out.reshape(Hq, D), bound.reshape(Hq, D)


F16_EPS, BF16_EPS = 2.0 ** -11, 2.0 ** -8


def unread(c, window, sinks):
    """c's table with ids outside the pool at every page without a seen token."""
    table = c.table.clone()
    for b, L in enumerate(c.lens):
        pages = set((seen(L, window, sinks) // c.ps).tolist())
        for i in range(-(-L // c.ps)):
            if i not in pages:
                table[c.starts[b] + i] = (-7, c.n_pool, 1 << 30)[i % 3]
    return table.to(DEV)


def decode(c, q, bits=4, window=0, sinks=0, splits=None, rows=None, d=None, ws=None, out=None):
    """(out, status word) of the 4-bit or the bf16 pools' call."""
    d = d or c.d
    S = splits or pkv.plan(d)[0]
    ws = pkv.alloc_workspace(d, S, DEV) if ws is None else ws
    if out is None:
        out = torch.full((d.B, c.Hq, c.D), float("nan"), dtype=torch.bfloat16, device=DEV)
    rows = rows or c.rows
    if bits == 4:
        pkv.paged_decode_attn_q4(d, q, *c.q4, *rows, S, ws, out, window=window, sinks=sinks)
    else:
        pkv.paged_decode_attn_window(d, q, c.k16, c.v16, *rows, window, sinks, S, ws, out)
    return out, pkv.status_word(ws)


def v_tops(c, b):
    """The largest scale of each of row b's values, [L, Hkv]."""
    return torch.exp2(c.stored(b, 0, c.lens[b])[3].double().amax(-1) - 127)


def check(c, q, out, bits=4, window=0, sinks=0):
    q, out = q.cpu(), out.cpu().double()
    for b, L in enumerate(c.lens):
        if L == 0:
            assert torch.equal(out[b], torch.zeros_like(out[b])), b
            continue
        at = seen(L, window, sinks)
        if bits == 4:
            k, v = (x[at] for x in c.held(b))
        else:
            k, v = (x.cpu()[c.places(b, 0, L)][at].double() for x in (c.k16, c.v16))
        want, bound = attention(q[b], k, v, c.scale, F16_EPS if bits == 4 else BF16_EPS,
                                v_tops(c, b)[at] if bits == 4 else None)
        off = (out[b] - want).abs()
        assert bool((off <= bound).all()), (b, L, float((off / bound).max()))


def fill16(c, gain=1.0):
    """bf16 values for every row's tokens (the pools' other slots stay NaN)."""
    for x in (c.k16, c.v16):
        h = x.cpu()
        for b, L in enumerate(c.lens):
            if L:
                h[c.places(b, 0, L)] = (c.randn(L, c.Hkv, c.D) * gain).to(torch.bfloat16)
        x.copy_(h)
    return c
