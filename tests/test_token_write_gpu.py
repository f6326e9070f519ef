"""paged_kv_append_norm / _extend_norm and their 8-bit forms against the
formulas in 64 bits: layouts, odd sizes, strided inputs, refusals by flag."""

import math

import pytest
import torch

from paged_kv_gqa_16_gb300 import pkv
from q8_cases import DEV, Cache, check_stored, norm_rotate, rope_table

pytestmark = pytest.mark.gpu


def _inputs(c, T, packed, norm, gain=1.0):
    heads = c.Hq + 2 * c.Hkv
    both = (c.randn(T, heads, c.D) * gain).to(torch.bfloat16).to(DEV)
    q, k, v = both[:, :c.Hq], both[:, c.Hq:c.Hq + c.Hkv], both[:, c.Hq + c.Hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw, kw = ((1 + 0.3 * c.randn(c.D)).to(torch.bfloat16).to(DEV) if n else None for n in norm)
    return q, k, v, qw, kw


def _check(c, q8, q, k, v, qw, kw, rope, q_out, b, t0, first, last):
    """Tokens first .. last - 1 of row b are input rows t0 ..."""
    n = last - first
    cs = None if rope is None else rope[first:last].cpu()
    cpu = lambda x: None if x is None else x.cpu()  # noqa: E731
    want, off = norm_rotate(q[t0:t0 + n].cpu(), cpu(qw), cs)
    got = q_out[t0:t0 + n].cpu().double()
    assert bool(((got - want).abs() <= want.abs() * 2.0 ** -8 + off * 1.01).all())
    want, off = norm_rotate(k[t0:t0 + n].cpu(), cpu(kw), cs)
    at = c.places(b, first, last)
    if q8:
        check_stored(c, "k", want, off, b, first, last)
        check_stored(c, "v", v[t0:t0 + n].cpu().double(), torch.zeros(n, c.Hkv, c.D).double(), b,
                     first, last)
    else:
        got = c.k16.cpu()[at].double()
        assert bool(((got - want).abs() <= want.abs() * 2.0 ** -8 + off * 1.01).all())
        assert torch.equal(c.v16.cpu()[at], v[t0:t0 + n].cpu())


def _untouched(c, written):
    """Every slot that is not in `written` [(b, first, last)] still holds NaN."""
    left = torch.ones(c.n_pool, c.ps, dtype=torch.bool)
    for b, first, last in written:
        left[c.places(b, first, last)] = False
    assert bool(torch.isnan(c.k16.cpu()[left]).all()) and bool(torch.isnan(c.v16.cpu()[left]).all())
    for t, v in ((c.kc, 0x7F), (c.vc, 0x7F), (c.ks, 255), (c.vs, 255)):
        assert bool((t.cpu()[left] == v).all())


HEADS = [(4, 2), (32, 8), (7, 7), (16, 1), (5, 1), (24, 3), (80, 5)]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("norm,rope,packed,ps", [((True, True), True, False, 16),
                                                 ((False, True), True, True, 1),
                                                 ((True, False), False, True, 24),
                                                 ((False, False), True, False, 5)])
def test_append(q8, D, Hq, Hkv, norm, rope, packed, ps):
    c = Cache([1, 17, 0, 100, 16, 33], Hq, Hkv, D, ps, seed=Hq * D + ps)
    q, k, v, qw, kw = _inputs(c, 6, packed, norm)
    table = rope_table(101, D) if rope else None
    q_out = torch.full((6, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    t = pkv.tokens(q, k, v, q_out, qw, kw, rope_cos_sin=table, rope_max_pos=101 if rope else 0)
    if q8:
        pkv.paged_kv_append_q8(c.d, t, *c.q8, *c.rows, status=c.status)
    else:
        pkv.paged_kv_append_norm(c.d, t, c.k16, c.v16, *c.rows, status=c.status)
    assert int(c.status.item()) == 0
    for b, L in enumerate(c.lens):
        if L:
            _check(c, q8, q, k, v, qw, kw, table, q_out, b, b, L - 1, L)
    assert bool(torch.isnan(q_out[2].float()).all())          # the idle row's queries
    _untouched(c, [(b, L - 1, L) for b, L in enumerate(c.lens) if L])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,ps,packed", [(32, 8, 128, 16, True), (32, 8, 64, 24, False),
                                                (6, 3, 64, 1, True), (16, 1, 128, 7, False),
                                                (4, 4, 128, 128, True)])
def test_extend(q8, Hq, Hkv, D, ps, packed):
    lens, chunks = [1, 40, 0, 77, 257, 30, 19], [1, 40, 0, 5, 131, 0, 18]
    c = Cache(lens, Hq, Hkv, D, ps, seed=D + ps)
    ends = torch.tensor([0] + chunks).cumsum(0)
    T = int(ends[-1])
    q, k, v, qw, kw = _inputs(c, T, packed, (True, True))
    table = rope_table(300, D)
    q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    qo = ends.to(torch.int32).to(DEV)
    t = pkv.tokens(q, k, v, q_out, qw, kw, rope_cos_sin=table, rope_max_pos=300)
    if q8:
        pkv.paged_kv_extend_q8(c.d, t, qo, *c.q8, *c.rows, status=c.status)
    else:
        pkv.paged_kv_extend_norm(c.d, t, qo, c.k16, c.v16, *c.rows, status=c.status)
    assert int(c.status.item()) == 0
    for b, (L, n) in enumerate(zip(lens, chunks)):
        if n:
            _check(c, q8, q, k, v, qw, kw, table, q_out, b, int(ends[b]), L - n, L)
    _untouched(c, [(b, L - n, L) for b, (L, n) in enumerate(zip(lens, chunks)) if n])


def _sparse(B, every, n=1):
    return [n if b % every == every - 1 else 0 for b in range(B)]


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (2, 1)])
@pytest.mark.parametrize("chunks", [[1] * 40, [2, 1] * 33, _sparse(1500, 50), _sparse(1100, 1099, 5),
                                    [0] * 33 + [3] + [0] * 31 + [1], [1] + [0] * 70 + [1] + [0] * 900 + [2],
                                    [3] + [0] * 1024, _sparse(64, 33, 2)],
                         ids=["ones", "pairs", "sparse", "far", "late", "gaps", "first", "two"])
def test_extend_finds_rows_between_empty_ones(chunks, Hq, Hkv):
    """One-token chunks, and rows without new tokens before, between and behind the
    others: a warp's tokens belong to rows that lie far apart."""
    lens = [n + (3 * b) % 7 if n else b % 3 for b, n in enumerate(chunks)]
    c = Cache(lens, Hq, Hkv, 64, 4, seed=len(chunks))
    ends = torch.tensor([0] + list(chunks)).cumsum(0)
    T = int(ends[-1])
    q, k, v, qw, kw = _inputs(c, T, False, (True, True))
    table = rope_table(32, 64)
    q_out = torch.full((T, Hq, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    qo = ends.to(torch.int32).to(DEV)
    t = pkv.tokens(q, k, v, q_out, qw, kw, rope_cos_sin=table, rope_max_pos=32)
    pkv.paged_kv_extend_q8(c.d, t, qo, *c.q8, *c.rows, status=c.status)
    assert int(c.status.item()) == 0
    live = [(b, L - n, L) for b, (L, n) in enumerate(zip(lens, chunks)) if n]
    for b, first, last in live:
        _check(c, True, q, k, v, qw, kw, table, q_out, b, int(ends[b]), first, last)
    _untouched(c, live)
    # with two tokens more than the rows take: those are refused and write nothing
    more = [torch.cat([x, x[:1], x[:1]]) for x in (q, k, v)]
    out2 = torch.full((T + 2, Hq, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    pkv.paged_kv_extend_q8(c.d, pkv.tokens(*more, out2, qw, kw, rope_cos_sin=table, rope_max_pos=32), qo,
                           *c.q8, *c.rows, status=c.status)
    assert int(c.status.item()) == pkv.FLAG_BAD_LEN
    assert torch.equal(out2[:T], q_out) and bool(torch.isnan(out2[T:].float()).all())


def test_plain_matches_append_bit_for_bit():
    """Without norms the bf16 write is paged_kv_append's, bit for bit."""
    c = Cache([9, 100, 1], 8, 2, 128, 16, seed=3)
    q, k, v, _, _ = _inputs(c, 3, False, (False, False))
    table = rope_table(128, 128)
    t = pkv.tokens(q, k, v, torch.empty_like(q), rope_cos_sin=table, rope_max_pos=128)
    pkv.paged_kv_append_norm(c.d, t, c.k16, c.v16, *c.rows)
    q2, k2, v2 = q.clone(), c.k16.clone(), c.v16.clone()
    k2.fill_(float("nan"))
    v2.fill_(float("nan"))
    pkv.paged_kv_append(c.d, q2, k, v, k2, v2, *c.rows, rope_cos_sin=table, rope_max_pos=128,
                        rope_q=True)
    for a, b in ((t.tensors[3], q2), (c.k16, k2), (c.v16, v2)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_in_place_and_without_queries():
    c = Cache([5, 33], 8, 4, 64, 16, seed=5)
    q, k, v, qw, kw = _inputs(c, 2, False, (True, True))
    table = rope_table(64, 64)
    q_out = torch.empty_like(q)
    rope = dict(rope_cos_sin=table, rope_max_pos=64)
    pkv.paged_kv_append_q8(c.d, pkv.tokens(q, k, v, q_out, qw, kw, **rope), *c.q8, *c.rows)
    first = [x.clone() for x in c.q8]
    pkv.paged_kv_append_q8(c.d, pkv.tokens(q, k, v, None, qw, kw, **rope), *c.q8, *c.rows)
    assert torch.equal(q.view(torch.int16), q_out.view(torch.int16))
    pkv.paged_kv_append_q8(c.d, pkv.tokens(None, k, v, None, None, kw, **rope), *c.q8, *c.rows)
    for a, b in zip(first, c.q8):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
def test_extreme_values(D):
    """Zeros, one element, subnormals, the largest bf16, a border of the scale,
    infinities and NaN."""
    big = float(torch.finfo(torch.bfloat16).max)
    vals = [torch.zeros(D), torch.full((D,), 1e-39), torch.full((D,), 448.0), torch.full((D,), 449.0),
            torch.full((D,), 2.0 ** -49), torch.full((D,), 2.0 ** -60), torch.full((D,), 447.0 * 2.0 ** 40),
            torch.full((D,), big), torch.linspace(-1, 1, D) * 7 * 2.0 ** -30]
    one = torch.zeros(D)
    one[D - 1] = -3.0
    x = torch.stack(vals + [one]).to(torch.bfloat16)[:, None, :]
    T = x.shape[0]
    c = Cache([1] * T, 1, 1, D, 16, seed=1)
    k = x.to(DEV)
    v = x.flip(0).contiguous().to(DEV)
    pkv.paged_kv_append_q8(c.d, pkv.tokens(None, k, v), *c.q8, *c.rows, status=c.status)
    assert int(c.status.item()) == 0
    zero = torch.zeros(1, 1, D).double()
    for b in range(T):
        check_stored(c, "k", k[b:b + 1].cpu().double(), zero, b, 0, 1)
        check_stored(c, "v", v[b:b + 1].cpu().double(), zero, b, 0, 1)
    # infinities and NaN become NaN, the other elements of the vector do not
    bad = torch.ones(2, 1, D)
    bad[0, 0, 3], bad[0, 0, 5], bad[1, 0, D - 1] = math.inf, -math.inf, math.nan
    bad = bad.to(torch.bfloat16).to(DEV)
    c = Cache([1, 1], 1, 1, D, 16, seed=2)
    pkv.paged_kv_append_q8(c.d, pkv.tokens(None, bad, bad), *c.q8, *c.rows)
    for b, where in ((0, [3, 5]), (1, [D - 1])):
        for got in c.held(b):
            assert torch.isnan(got[0, 0]).nonzero().flatten().tolist() == where
    # a zero vector stays zero through the norm
    c = Cache([1], 1, 1, D, 16, seed=2)
    z = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    pkv.paged_kv_append_norm(c.d, pkv.tokens(z, z, z, None, w, w), c.k16, c.v16, *c.rows)
    assert float(z.abs().max()) == 0 and float(c.k16[c.table[0].item(), 0].abs().max()) == 0


@pytest.mark.parametrize("q8", [False, True])
def test_flags(q8):
    """A bad row sets its flag and writes nothing; the others are written."""
    c = Cache([5, 9, 20, 3], 4, 2, 64, 4, seed=6, max_seq_len=16)
    table = rope_table(8, 64)

    def write(lens=None, indices=None, rope=None):
        for x in (c.k16, c.v16):
            x.fill_(float("nan"))
        for x, f in ((c.kc, 0x7F), (c.vc, 0x7F), (c.ks, 255), (c.vs, 255)):
            x.fill_(f)
        c.status.zero_()
        q, k, v, _, _ = _inputs(c, 4, False, (False, False))
        q_out = torch.full_like(q, float("nan"))
        t = pkv.tokens(q, k, v, q_out, rope_cos_sin=rope, rope_max_pos=0 if rope is None else 8)
        rows = (c.kv_indices if indices is None else indices, c.kv_indptr,
                c.seq_lens if lens is None else lens)
        if q8:
            pkv.paged_kv_append_q8(c.d, t, *c.q8, *rows, status=c.status)
        else:
            pkv.paged_kv_append_norm(c.d, t, c.k16, c.v16, *rows, status=c.status)
        live = [not bool(torch.isnan(q_out[b].float()).any()) for b in range(4)]
        return int(c.status.item()), live, c.kc if q8 else c.k16

    assert write()[:2] == (pkv.FLAG_BAD_LEN, [True, True, False, True])
    minus = c.seq_lens.clone()
    minus[2] = -1
    assert write(lens=minus)[:2] == (pkv.FLAG_BAD_LEN, [True, True, False, True])
    ok = c.seq_lens.clone()
    ok[2] = 10
    for bad in (-1, c.n_pool, 2 ** 31 - 1):
        ind = c.kv_indices.clone()
        ind[c.starts[1] + 2] = bad                          # row 1's token 8
        assert write(lens=ok, indices=ind)[:2] == (pkv.FLAG_BAD_PAGE, [True, False, True, True])
    status, live, _ = write(lens=ok, rope=table)             # positions 8 and 9 are past the table
    assert (status, live) == (pkv.FLAG_BAD_POS, [True, False, False, True])


def test_extend_flags():
    c = Cache([5, 9, 3], 4, 2, 64, 4, seed=7)
    q, k, v, _, _ = _inputs(c, 12, False, (False, False))

    def write(qo):
        c.status.zero_()
        q_out = torch.full_like(q, float("nan"))
        t = pkv.tokens(q, k, v, q_out)
        pkv.paged_kv_extend_q8(c.d, t, torch.tensor(qo, dtype=torch.int32, device=DEV), *c.q8,
                               *c.rows, status=c.status)
        return int(c.status.item()), (~torch.isnan(q_out.float()).flatten(1).any(1)).tolist()

    assert write([0, 4, 10, 12]) == (0, [True] * 12)
    # row 0's chunk is longer than the row
    assert write([0, 6, 10, 12]) == (pkv.FLAG_BAD_LEN, [False] * 6 + [True] * 6)
    # tokens before the first row and behind the last
    assert write([1, 4, 9, 11]) == (pkv.FLAG_BAD_LEN, [False] + [True] * 10 + [False])
    # chunks that leave the tokens given
    assert write([-1, 4, 10, 12]) == (pkv.FLAG_BAD_LEN, [False] * 4 + [True] * 8)
    assert write([0, 4, 10, 13]) == (pkv.FLAG_BAD_LEN, [True] * 10 + [False] * 2)


def test_rows_of_one_projection_and_64_bit_offsets():
    """Row strides far past the heads' own width."""
    c = Cache([3, 12], 2, 1, 64, 8, seed=8)
    wide = torch.zeros(2, 1 << 14, dtype=torch.bfloat16, device=DEV)
    wide[:, :256] = c.randn(2, 256).to(torch.bfloat16).to(DEV)
    q, k, v = wide[:, :128].unflatten(1, (2, 64)), wide[:, 128:192].unflatten(1, (1, 64)), wide[:, 192:256].unflatten(1, (1, 64))
    q_out = torch.empty(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    pkv.paged_kv_append_norm(c.d, pkv.tokens(q, k, v, q_out), c.k16, c.v16, *c.rows)
    assert torch.equal(q_out, q)
    for b, L in enumerate(c.lens):
        at = c.places(b, L - 1, L)
        assert torch.equal(c.k16.cpu()[at][0], k[b].cpu()) and torch.equal(c.v16.cpu()[at][0], v[b].cpu())
