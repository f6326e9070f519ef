"""Shared by the tests of the normalising cache writes and the 8-bit cache: a
plain implementation in 64 bits, written from the formulas, and device state
whose unused slots hold NaN, so that a stray read shows.

Bounds.  A value rounded to bf16 is off by at most 2^-8 of itself, an e4m3
code by 2^-4 of itself or 2^-10 of its scale (its steps under 2^-6 are 2^-9).
FP32 is 2^-24 an operation: the norm's sum of at most 128 squares and its root
are off by under 2^-18, the rotation by 2 more roundings of products as large
as its pair."""

from __future__ import annotations

import math

import numpy as np
import torch

from paged_kv_gqa_16_gb300 import pkv

EPS = 1e-6
NAN_CODE = 0x7F
DEV = "cuda"


# ------------------------------------------------------------- 64-bit reference
def norm_rotate(x, weight, cos_sin):
    """x [T, H, D]: the norm (weight [D] or None) and the rotation (cos_sin
    [T, D/2, 2] or None), and how far 32-bit arithmetic may be off."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.double()
    pair = x.reshape(*x.shape[:-1], -1, 2)
    size = pair.abs().sum(-1, keepdim=True).expand_as(pair).reshape(x.shape)
    if cos_sin is not None:
        z = torch.view_as_complex(pair.contiguous()) * torch.view_as_complex(
            cos_sin.double().contiguous())[:, None]
        x = torch.view_as_real(z).reshape(x.shape)
    return x, size * 2.0 ** -17


def exponents(amax):
    """clamp(ceil(log2(amax / 448)), -40, 40), the lowest for zero."""
    e = torch.full_like(amax, -40.0)
    some = amax > 0
    e[some] = torch.ceil(torch.log2(amax[some] / 448.0)).clamp(-40, 40)
    return e


def decode_values(codes, scale):
    """Codes [..., D] (uint8) and scale bytes [...] as the values they stand for."""
    return codes.view(torch.float8_e4m3fn).double() * torch.exp2(scale.double() - 127)[..., None]


def attention(q, k, v, scale):
    """q [Hq, D], k and v [L, Hkv, D]: the output [Hq, D] and its bound: the
    output's rounding (2^-8), the weights' rounding to 11 bits (2^-11 of each) and
    the scores' error (128 products of 2^-23 each at most, so under 2^-16 of
    sum |q k|, twice in the weights and their sum) against sum_t w_t |v_t|."""
    Hq, D = q.shape
    L, Hkv, _ = k.shape
    q = q.double().view(Hkv, Hq // Hkv, D)
    x = torch.einsum("grd,lgd->grl", q, k) * scale
    w = torch.softmax(x, -1)
    out = torch.einsum("grl,lgd->grd", w, v)
    size = torch.einsum("grl,lgd->grd", w, v.abs())
    far = torch.einsum("grd,lgd->grl", q.abs(), k.abs()).amax(-1, keepdim=True) * scale * 2.0 ** -16
    bound = out.abs() * 2.0 ** -8 + size * (2.0 ** -10 + 2 * far) + 1e-30
    return out.reshape(Hq, D), bound.reshape(Hq, D)


# ---------------------------------------------------------------- device state
class Cache:
    """Rows of an 8-bit or bf16 cache: a table over scattered pages, pools
    filled with NaN, lengths on both sides."""

    def __init__(self, lens, Hq, Hkv, D, ps, seed=0, room=0, max_seq_len=None, spare=3):
        self.g = torch.Generator().manual_seed(seed)
        self.lens, self.Hq, self.Hkv, self.D, self.ps = list(lens), Hq, Hkv, D, ps
        B = len(self.lens)
        pages = [-(-(L + room) // ps) for L in self.lens]
        self.starts = [0] + list(np.cumsum(pages))
        self.n_ref = int(self.starts[-1])
        self.n_pool = self.n_ref + spare
        self.table = torch.randperm(self.n_pool, generator=self.g)[:self.n_ref].to(torch.int32)
        self.kv_indices = self.table.to(DEV)
        self.kv_indptr = torch.tensor(self.starts, dtype=torch.int32, device=DEV)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.scale = 1.0 / math.sqrt(D)
        self.d = pkv.dims(B, Hq, Hkv, D, ps, self.n_pool, self.n_ref,
                          max_seq_len or max(self.lens + [0]) + room + 1)
        pool = (self.n_pool, ps, Hkv, D)
        self.k16, self.v16 = (torch.full(pool, float("nan"), dtype=torch.bfloat16, device=DEV)
                              for _ in range(2))
        self.kc, self.vc = (torch.full(pool, NAN_CODE, dtype=torch.uint8, device=DEV)
                            for _ in range(2))
        self.ks, self.vs = (torch.full(pool[:3], 255, dtype=torch.uint8, device=DEV)
                            for _ in range(2))
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    @property
    def q8(self):
        return self.kc, self.vc, self.ks, self.vs

    @property
    def rows(self):
        return self.kv_indices, self.kv_indptr, self.seq_lens

    def places(self, b, first, last):
        """(page, slot) of tokens first .. last - 1 of row b, on the CPU."""
        t = torch.arange(first, last)
        return self.table.long()[self.starts[b] + t // self.ps], t % self.ps

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g)

    def fill(self, k_gain=None, v_gain=None):
        """Random codes and scales for every row's tokens (gains: the range of
        the scales' exponents)."""
        for c, s, (lo, hi) in ((self.kc, self.ks, k_gain or (-9, -5)),
                               (self.vc, self.vs, v_gain or (-9, -5))):
            codes, scale = c.cpu(), s.cpu()
            for b, L in enumerate(self.lens):
                if L:
                    at = self.places(b, 0, L)
                    x = self.randn(L, self.Hkv, self.D) * 100
                    codes[at] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    scale[at] = torch.randint(lo + 127, hi + 128, (L, self.Hkv), generator=self.g).to(torch.uint8)
            c.copy_(codes)
            s.copy_(scale)
        return self

    def held(self, b, L=None):
        """Row b's K and V as values [L, Hkv, D] in 64 bits."""
        at = self.places(b, 0, self.lens[b] if L is None else L)
        kc, vc, ks, vs = (x.cpu()[at] for x in self.q8)
        return decode_values(kc, ks), decode_values(vc, vs)

    def decode(self, q, splits=None, out=None, d=None):
        d = d or self.d
        S = splits or pkv.plan(d)[0]
        ws = pkv.alloc_workspace(d, S, DEV)
        out = torch.full((d.B, self.Hq, self.D), float("nan"), dtype=torch.bfloat16,
                         device=DEV) if out is None else out
        pkv.paged_decode_attn_q8(d, q, *self.q8, *self.rows, S, ws, out)
        return out, pkv.status_word(ws)

    def check_decode(self, q, out):
        q, out = q.cpu(), out.cpu().double()
        for b, L in enumerate(self.lens):
            if L == 0:
                assert torch.equal(out[b], torch.zeros_like(out[b])), b
                continue
            want, bound = attention(q[b], *self.held(b), self.scale)
            off = (out[b] - want).abs()
            assert bool((off <= bound).all()), (b, L, float((off / bound).max()))


def rope_table(n, D):
    t = torch.empty(n, D // 2, 2, dtype=torch.float32, device=DEV)
    pkv.rope_table(t, n, D, 10000.0)
    return t


def check_stored(cache, kind, x, off, b, first, last):
    """Row b's stored tokens against x [n, H, D] in 64 bits; `off`: how far the
    32-bit values may be from x."""
    at = cache.places(b, first, last)
    codes, scale = (t.cpu()[at] for t in ((cache.kc, cache.ks) if kind == "k" else (cache.vc, cache.vs)))
    e = scale.double() - 127
    amax = x.abs().amax(-1)
    slack = off.amax(-1)
    # the scale is the exact one wherever amax is not within its error of a border
    assert bool(((e >= exponents((amax - slack).clamp(min=0))) & (e <= exponents(amax + slack))).all())
    y = decode_values(codes, scale)
    step = torch.exp2(e)[..., None]
    bound = torch.maximum(x.abs() * 2.0 ** -4, step * 2.0 ** -10) + off * 1.1
    sat = x.abs() > 448 * step                      # over the format's range: the largest value
    want = torch.where(sat, torch.sign(x) * 448 * step, x)
    assert bool(((y - want).abs() <= bound).all()), float(((y - want).abs() / bound).max())
