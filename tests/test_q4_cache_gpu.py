"""GPU tests of the 4-bit cache's writes and read-back against 64 bits."""

import pytest
import torch

import q4_cases
from paged_kv_gqa_16_gb300 import pkv
from q4_cases import bf16_of, quantise, values
from q8_cases import DEV, EPS, norm_rotate, rope_table

pytestmark = pytest.mark.gpu


def _new(c, T, seed, packed=False, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, c.Hq + 2 * c.Hkv, c.D, generator=g) * gain).to(torch.bfloat16).to(DEV)
    q, k, v = x.split([c.Hq, c.Hkv, c.Hkv], 1)
    return (q, k, v) if packed else (q.contiguous(), k.contiguous(), v.contiguous())


def _check(c, b, first, last, k, v, k_norm, rope):
    """Row b's tokens first .. last - 1 hold k and v [n, Hkv, D]."""
    pos = torch.arange(first, last)
    want, _ = norm_rotate(k.cpu(), None if k_norm is None else k_norm.cpu(), None if rope is None else rope.cpu()[pos])
    kc, ks, vc, vs = c.stored(b, first, last)
    for got_c, got_s, x in ((kc, ks, want), (vc, vs, v.cpu().double())):
        code, scale = quantise(x)
        assert torch.equal(got_s, scale), (b, got_s[got_s != scale], scale[got_s != scale])
        assert torch.equal(got_c & 7, code & 7), b
        assert torch.equal(values(got_c, got_s), values(code, scale)), b


SHAPES = [  # Hq, Hkv, D, page size, lengths
    (32, 8, 128, 16, [1, 17, 300, 0, 64]),
    (8, 1, 64, 1, [5, 1, 33]),
    (10, 5, 64, 17, [40, 0, 18, 17]),
    (16, 16, 128, 24, [25, 24, 1]),
    (4, 2, 128, 128, [129, 500]),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("norm,rope,packed", [(False, False, False), (True, True, True), (False, True, False),
                                              (True, False, True)])
def test_append(shape, norm, rope, packed):
    Hq, Hkv, D, ps, lens = shape
    c = q4_cases.Cache(lens, Hq, Hkv, D, ps, seed=1)
    before = [x.clone() for x in c.q4]
    q, k, v = _new(c, len(lens), 2, packed)
    w = (1 + 0.2 * c.randn(D)).to(torch.bfloat16).to(DEV) if norm else None
    table = rope_table(600, D) if rope else None
    q_out = torch.full((len(lens), Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    t = pkv.tokens(q, k, v, q_out, q_norm=w, k_norm=w, norm_eps=EPS, rope_cos_sin=table,
                   rope_max_pos=600 if rope else 0)
    pkv.paged_kv_append_q4(c.d, t, *c.q4, *c.rows, status=c.status)
    assert int(c.status) == 0
    touched = [x.cpu() for x in before]
    for b, L in enumerate(lens):
        if L == 0:
            assert bool(torch.isnan(q_out[b]).all())
            continue
        _check(c, b, L - 1, L, k[b:b + 1], v[b:b + 1], w, table)
        want, off = norm_rotate(q[b:b + 1].cpu(), None if w is None else w.cpu(),
                                None if table is None else table.cpu()[L - 1:L])
        assert bool(((q_out[b].cpu().double() - want[0]).abs() <= want[0].abs() * 2.0 ** -8 + off[0]).all())
        at = c.places(b, L - 1, L)
        for x, y in zip(touched, c.q4):
            x[at] = y.cpu()[at]
    # nothing but the new tokens' slots was written
    assert all(torch.equal(x, y.cpu()) for x, y in zip(touched, c.q4))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("norm,rope", [(True, True), (False, True), (False, False)])
def test_extend_and_read(shape, norm, rope):
    Hq, Hkv, D, ps, lens = shape
    c = q4_cases.Cache(lens, Hq, Hkv, D, ps, seed=3).fill()
    chunks = [min(L, n) for L, n in zip(lens, [1, 9, 250, 4, 64])]
    ends = torch.tensor([0] + chunks).cumsum(0)
    T = int(ends[-1])
    _, k, v = _new(c, T, 4, gain=3.0)
    w = (1 + 0.2 * c.randn(D)).to(torch.bfloat16).to(DEV) if norm else None
    table = rope_table(600, D) if rope else None
    t = pkv.tokens(None, k, v, k_norm=w, norm_eps=EPS, rope_cos_sin=table, rope_max_pos=600 if rope else 0)
    old = [c.held(b, L - n) for b, (L, n) in enumerate(zip(lens, chunks))]
    pkv.paged_kv_extend_q4(c.d, t, ends.to(torch.int32).to(DEV), *c.q4, *c.rows, status=c.status)
    out = [torch.full((c.n_ref, ps, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pkv.paged_kv_read_q4(c.d, *c.q4, *c.rows, *out, status=c.status)
    assert int(c.status) == 0
    for b, (L, n) in enumerate(zip(lens, chunks)):
        a, e = int(ends[b]), int(ends[b + 1])
        if n:
            _check(c, b, L - n, L, k[a:e], v[a:e], w, table)
        for was, now, got in zip(old[b], c.held(b), out):
            assert torch.equal(now[:L - n], was)                   # the cached tokens before the chunk
            flat = got.cpu().flatten(0, 1)[c.starts[b] * ps:c.starts[b + 1] * ps]
            assert torch.equal(flat[:L], bf16_of(now)) and bool((flat[L:] == 7).all())


@pytest.mark.parametrize("D", [64, 128])
def test_borders_of_codes_and_scales(D):
    """V is stored from its bf16 value: every border and tie between codes, the
    groups' largest at the borders of a scale, zeros, the range's ends, and values
    that are infinite or NaN in one group."""
    H, T = 4, 24
    c = q4_cases.Cache([T], H, H, D, 16, seed=5)
    v = torch.zeros(T, H, D)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    near = torch.cat([ties, ties * (1 + 2 ** -7), ties * (1 - 2 ** -8), -ties])     # 32 values of bf16
    for t in range(T):
        # 6 as the group's largest keeps the scale at one; powers of two move it
        x = near * 2.0 ** ((t % 12) * 8 - 44)
        v[t] = x.clamp(-6.0 * 2.0 ** 45, 6.0 * 2.0 ** 45).repeat(H, D // 32)
    v[3, 1, 5], v[4, 2, D - 1], v[5, 0, 0] = float("inf"), float("nan"), -float("inf")
    v[6] = 0
    v[7, :, 32:] = 0
    v[8] = 2.0 ** 60
    v[9] = -1e-30
    v = v.to(torch.bfloat16)
    zero = torch.zeros(T, H, D, dtype=torch.bfloat16)
    t = pkv.tokens(None, zero.to(DEV), v.to(DEV))
    pkv.paged_kv_extend_q4(c.d, t, torch.tensor([0, T], dtype=torch.int32, device=DEV), *c.q4, *c.rows,
                           status=c.status)
    assert int(c.status) == 0
    kc, ks, vc, vs = c.stored(0, 0, T)
    code, scale = quantise(v.double())
    assert torch.equal(vs, scale) and torch.equal(vc, code)
    assert int(vs[3, 1, 0]) == 255 and int((vs[3] == 255).sum()) == 1
    assert bool((kc & 7 == 0).all()) and bool((ks == 87).all())
    out = [torch.zeros(c.n_ref, 16, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pkv.paged_kv_read_q4(c.d, *c.q4, *c.rows, *out, status=c.status)
    got = out[1].cpu().flatten(0, 1)[:T]
    assert torch.equal(got.isnan(), values(code, scale).isnan())
    assert torch.equal(got[~got.isnan()], bf16_of(values(code, scale))[~got.isnan()])


@pytest.mark.parametrize("norm,rope", [(True, True), (False, True), (True, False)])
def test_keys_next_to_borders_are_rounded_as_exact_values(norm, rope):
    """Half a million keys, some thousand of which lie within 32-bit error of a
    border: every code is the exact value's."""
    H, D, T = 8, 128, 512
    c = q4_cases.Cache([T], H, H, D, 16, seed=6)
    k = c.randn(T, H, D).to(torch.bfloat16)
    # rotations that keep the value, so that bf16 keys on a border stay there but for the table's rounding
    k[::3] = (k[::3] * 4).round() / 4
    w = torch.full((D,), 1.5).to(torch.bfloat16)
    table = rope_table(T, D)
    v = c.randn(T, H, D).to(torch.bfloat16)
    t = pkv.tokens(None, k.to(DEV), v.to(DEV), k_norm=w.to(DEV) if norm else None, norm_eps=0.0 if norm else EPS,
                   rope_cos_sin=table if rope else None, rope_max_pos=T if rope else 0)
    pkv.paged_kv_extend_q4(c.d, t, torch.tensor([0, T], dtype=torch.int32, device=DEV), *c.q4, *c.rows,
                           status=c.status)
    x = k.double()
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True)) * w.double()
    want, _ = norm_rotate(x, None, table.cpu() if rope else None)
    code, scale = quantise(want)
    kc, ks, _, _ = c.stored(0, 0, T)
    assert torch.equal(ks, scale)
    assert torch.equal(kc & 7, code & 7)


def test_bad_rows_write_nothing():
    """Refused rows (length, page, position) leave the cache and their queries."""
    lens = [20, 5, 33, 8]
    c = q4_cases.Cache(lens, 8, 2, 64, 16, seed=7)
    before = [x.clone() for x in c.q4]
    q, k, v = _new(c, 4, 8)
    table = rope_table(16, 64)
    q_out = torch.full((4, 8, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    rows = [c.kv_indices.clone(), c.kv_indptr, c.seq_lens.clone()]
    rows[0][c.starts[1]] = c.n_pool           # row 1: a page outside the pool; rows 0 and 2: past the table
    rows[2][3] = c.d.max_seq_len + 1
    t = pkv.tokens(q, k, v, q_out, rope_cos_sin=table, rope_max_pos=16)
    pkv.paged_kv_append_q4(c.d, t, *c.q4, *rows, status=c.status)
    assert int(c.status) == pkv.FLAG_BAD_PAGE | pkv.FLAG_BAD_LEN | pkv.FLAG_BAD_POS
    assert all(torch.equal(a, b) for a, b in zip(before, c.q4))
    assert bool((q_out == 3).all())
    out = [torch.full((c.n_ref, 16, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    c.status.zero_()
    pkv.paged_kv_read_q4(c.d, *c.q4, *rows, *out, status=c.status)
    assert int(c.status) == pkv.FLAG_BAD_PAGE | pkv.FLAG_BAD_LEN
    read = out[0].cpu().flatten(0, 1)
    assert bool((read[c.starts[1] * 16:c.starts[1] * 16 + 5] == 7).all())
    assert bool(read[c.starts[0] * 16:c.starts[0] * 16 + 20].isnan().all())
