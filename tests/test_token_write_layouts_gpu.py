"""The normalising writes on layouts at the edge of what they take: queries in
place over ragged chunks, row strides whose offsets pass 31 and 32 bits."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import pkv
from q8_cases import DEV, Cache, rope_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(32, 8, 128, 16), (80, 5, 64, 7), (7, 7, 64, 1), (4, 2, 128, 24)])
@pytest.mark.parametrize("chunks", [[3, 1, 0, 2], [131, 0, 40, 257], [1500, 1100]], ids=["few", "some", "many"])
def test_extend_in_place(q8, Hq, Hkv, D, ps, chunks):
    """Several lane groups a token, one, and a block of several tokens: the same bits
    as into an output of its own."""
    T = sum(chunks)
    c = Cache([n + 9 for n in chunks], Hq, Hkv, D, ps, seed=T)
    table = rope_table(max(chunks) + 9, D)
    new = lambda H: c.randn(T, H, D).to(torch.bfloat16).to(DEV)  # noqa: E731
    q, k, v = new(Hq), new(Hkv), new(Hkv)
    w = (1 + 0.3 * c.randn(D)).to(torch.bfloat16).to(DEV)
    qo = torch.tensor([0] + chunks, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)
    how = dict(q_norm=w, k_norm=w, rope_cos_sin=table, rope_max_pos=table.shape[0])
    cache = c.q8 if q8 else (c.k16, c.v16)
    write = pkv.paged_kv_extend_q8 if q8 else pkv.paged_kv_extend_norm
    q_out = torch.full_like(q, float("nan"))
    write(c.d, pkv.tokens(q, k, v, q_out, **how), qo, *cache, *c.rows, status=c.status)
    kept = [x.clone() for x in cache]
    for out in (None, q):                          # both name q itself
        again = q.clone()
        write(c.d, pkv.tokens(again, k, v, out if out is None else again, **how), qo, *cache, *c.rows,
              status=c.status)
        assert torch.equal(again.view(torch.int16), q_out.view(torch.int16))
    assert int(c.status.item()) == 0
    for a, b in zip(kept, cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("extend", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_row_strides_past_31_bits(extend, q8):
    """Three rows 2^30 + 8 elements apart: the third starts past 2^31 elements and
    2^32 bytes."""
    step, Hq, Hkv, D = (1 << 30) + 8, 4, 2, 64
    wide = torch.empty(2 * step + 512, dtype=torch.bfloat16, device=DEV)
    rows = wide.as_strided((3, 512), (step, 1))
    c = Cache([5, 9, 33], Hq, Hkv, D, 8, seed=8)
    rows.copy_(c.randn(3, 512).to(torch.bfloat16))
    q, k, v = (rows[:, a:b].unflatten(1, (-1, D)) for a, b in ((0, 256), (256, 384), (384, 512)))
    assert q.stride(0) == step and k.stride(0) == step
    table = rope_table(64, D)
    w = (1 + 0.3 * c.randn(D)).to(torch.bfloat16).to(DEV)
    how = dict(q_norm=w, k_norm=w, rope_cos_sin=table, rope_max_pos=64)
    cache = c.q8 if q8 else (c.k16, c.v16)
    name = "paged_kv_%s_%s" % ("extend" if extend else "append", "q8" if q8 else "norm")
    first = (torch.arange(4, dtype=torch.int32, device=DEV),) if extend else ()
    got = []
    for a in ((q, k, v), (q.contiguous(), k.contiguous(), v.contiguous())):
        q_out = torch.full((3, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        getattr(pkv, name)(c.d, pkv.tokens(*a, q_out, **how), *first, *cache, *c.rows, status=c.status)
        got.append([q_out] + [x.clone() for x in cache])
    assert int(c.status.item()) == 0 and bool(torch.isfinite(got[0][0].float()).all())
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("D", [64, 128])
def test_models_that_rotate_the_halves_of_a_head(D):
    """With the heads' elements and the norm weights in the order x[0], x[D/2], x[1], ...
    the write gives what norm and rotation of (x[i], x[i + D/2]) give, in that order."""
    c = Cache([40, 7], 4, 2, D, 16, seed=3)
    order = torch.arange(D).view(2, D // 2).T.reshape(-1)
    q, k, v = (c.randn(2, H, D).to(torch.bfloat16) for H in (4, 2, 2))
    w = (1 + 0.3 * c.randn(D)).to(torch.bfloat16)
    table = rope_table(64, D)
    q_out = torch.empty(2, 4, D, dtype=torch.bfloat16, device=DEV)
    pkv.paged_kv_append_norm(
        c.d, pkv.tokens(q[..., order].contiguous().to(DEV), k[..., order].contiguous().to(DEV), v.to(DEV), q_out,
                        w[order].to(DEV), w[order].to(DEV), rope_cos_sin=table, rope_max_pos=64),
        c.k16, c.v16, *c.rows)

    def want(x, pos):
        x = x.double()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
        cos, sin = table[pos].cpu().double().unbind(-1)
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)[..., order]

    for b, L in enumerate(c.lens):
        page, slot = c.places(b, L - 1, L)
        for got, x in ((q_out[b], q[b]), (c.k16[page[0], slot[0]], k[b])):
            # one rounding to bf16, and fp32's of a norm and a rotation of values up to 8
            assert bool(((got.cpu().double() - want(x, L - 1)).abs() <=
                         want(x, L - 1).abs() * 2.0 ** -8 + 2.0 ** -13).all())
