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
