"""How much paged_decode_attn_q8 keeps of weights and values that lie far below
the largest of their row, against the definition in 64 bits.

Bounds.  A token's weight is rounded to 11 significant bits, or to 2^-32 of the
row's largest weight times value scale, whichever is more; the weights' sum is
kept in 32 bits.  The output is rounded to 2^-8 of itself, the scores are off by
under 2^-16 of the largest sum of |q k| (128 products, each within 2^-23)."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import pkv
from q8_cases import DEV, Cache

pytestmark = pytest.mark.gpu


def _reference(c, b, q):
    """Output [Hq, D] of row b and its bound, from the format's definition."""
    k, v = c.held(b)
    at = c.places(b, 0, c.lens[b])
    step = torch.exp2(c.vs.cpu()[at].double() - 127)                  # [L, Hkv]
    Hkv = c.Hkv
    x = torch.einsum("grd,lgd->grl", q.double().view(Hkv, -1, c.D), k) * c.scale
    w = torch.softmax(x, -1)
    out = torch.einsum("grl,lgd->grd", w, v)
    size = torch.einsum("grl,lgd->grd", w, v.abs())
    far = torch.einsum("grd,lgd->grl", q.double().abs().view(Hkv, -1, c.D), k.abs()).amax(-1, keepdim=True)
    top = (w * step.T[:, None]).amax(-1, keepdim=True)                 # the largest weight times scale
    codes = (v / step[..., None]).abs().sum(0)[:, None]                # [Hkv, 1, D]
    bound = out.abs() * 2.0 ** -8 + size * (2.0 ** -10 + far * c.scale * 2.0 ** -15)
    return out.reshape(c.Hq, c.D), (bound + top * codes * 2.0 ** -32).reshape(c.Hq, c.D)


def _check(c, q, splits=None):
    out, status = c.decode(q, splits)
    assert status == 0
    for b in range(len(c.lens)):
        want, bound = _reference(c, b, q[b].cpu())
        off = (out[b].cpu().double() - want).abs()
        assert bool((off <= bound).all()), (b, float((off / bound.clamp(min=1e-300)).max()))


def _set(c, which, b, t, codes, exponent):
    """Tokens t (a slice) of row b: the same codes [D] (as values) and scale."""
    t = range(c.lens[b])[t]
    at = c.places(b, t[0], t[-1] + 1)
    pool, scale = (c.kc, c.ks) if which == "k" else (c.vc, c.vs)
    pool[at[0], at[1]] = codes.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    scale[at[0], at[1]] = exponent + 127


# a kv head has 8, 4, 2 and 1 warps of a block; 9 to 16 query heads are two product columns
HEADS = [(1, 1, 64), (4, 1, 128), (8, 2, 64), (12, 1, 128), (16, 4, 128), (16, 8, 64)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("below", [15.5, 20.0, 25.5])
def test_long_flat_tail_under_a_heavy_token(Hq, Hkv, D, below):
    """One token takes nearly all of the weight and has zero values; 30,000 others,
    2^-below of it each, are all that the output is made of."""
    L = 30_000
    c = Cache([L], Hq, Hkv, D, 16, seed=1)
    ones = torch.ones(D)
    _set(c, "k", 0, slice(None), torch.zeros(D), 0)
    _set(c, "k", 0, slice(0, 1), ones, 0)                              # the heavy token
    _set(c, "v", 0, slice(None), ones * 3.5, -7)
    _set(c, "v", 0, slice(0, 1), ones * 0, -7)
    # scores: q.1 * scale = below ln 2 for the heavy token, 0 for the others
    q = torch.zeros(1, Hq, D)
    q[:] = below * 0.6931471805599453 / (D * c.scale)
    _check(c, q.to(torch.bfloat16).to(DEV), 1)
    _check(c, q.to(torch.bfloat16).to(DEV))


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("loud", [8, 14, 18])
def test_loud_tokens_with_zeros_beside_quiet_ones(Hq, Hkv, D, loud):
    """Values 2^loud larger in half of the channels, zero in the others, which then
    hold what the quiet tokens say."""
    c = Cache([513, 40, 3000], Hq, Hkv, D, 16, seed=2).fill(k_gain=(-9, -8), v_gain=(-8, -8))
    half = torch.zeros(D)
    half[::2] = 448
    for b, L in enumerate(c.lens):
        for t in range(1, L, 7):
            _set(c, "v", b, slice(t, t + 1), half, -8 + loud)
    q = (c.randn(3, Hq, D) * 0.5).to(torch.bfloat16).to(DEV)
    _check(c, q, 1)
    _check(c, q)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("loud", [10, 18, 22, 31])
def test_one_large_query_element_over_zero_keys(Hq, Hkv, D, loud):
    """A query element 2^loud times the others meets zero codes: the scores are what
    the others make of them, exactly (an element keeps its bits down to 2^-32 of its
    head's largest)."""
    c = Cache([300, 17, 2000], Hq, Hkv, D, 16, seed=3).fill()
    c.kc[..., 5] = 0
    q = c.randn(3, Hq, D) * 2
    q[..., 5] = 3.0 * 2.0 ** loud
    q = q.to(torch.bfloat16)
    # an element nearer zero than 2^-32 of the largest is off by 2^-40 of it at most: none here
    q[q.abs() < 3.0 * 2.0 ** (loud - 32)] = 0
    _check(c, q.to(DEV), 1)
    _check(c, q.to(DEV))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [-133, -126, -112, -111, -110, 14, 15, 16, 126, 127])
def test_queries_at_both_ends_of_the_type(D, power):
    """Heads whose largest element is the type's smallest or lies near its largest,
    over keys that are zero or as small as keys get."""
    c = Cache([77, 5], 8, 2, D, 16, seed=4).fill()
    if power > 15:
        c.kc[c.kc != 0x7F] = 0
    q = torch.randint(-1, 2, (2, 8, D), generator=c.g).double() * 2.0 ** power
    _check(c, q.to(torch.bfloat16).to(DEV))
