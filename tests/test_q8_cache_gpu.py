"""paged_kv_read_q8 and paged_decode_attn_q8 against the definition in 64 bits,
and the operators run together as a serving loop runs them."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import pkv
from q8_cases import DEV, Cache, attention, norm_rotate, rope_table

pytestmark = pytest.mark.gpu


def _q(c, gain=1.0):
    return (c.randn(len(c.lens), c.Hq, c.D) * gain).to(torch.bfloat16).to(DEV)


# --------------------------------------------------------------------- reading
@pytest.mark.parametrize("Hkv,D,ps,lens", [
    (8, 128, 16, [1, 16, 17, 0, 100]), (2, 64, 16, [37, 100]), (1, 64, 1, [3, 0, 5]),
    (3, 128, 7, [50, 7, 8, 6]), (5, 64, 128, [200, 1, 127, 128, 129]), (16, 128, 24, [70])])
def test_read(Hkv, D, ps, lens):
    c = Cache(lens, Hkv, Hkv, D, ps, seed=D + ps).fill()
    k, v = (torch.full((c.n_ref, ps, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV)
            for _ in range(2))
    pkv.paged_kv_read_q8(c.d, *c.q8, *c.rows, k, v, status=c.status)
    assert int(c.status.item()) == 0
    left = torch.ones(c.n_ref * ps, dtype=torch.bool)
    k, v = k.cpu().view(-1, Hkv, D), v.cpu().view(-1, Hkv, D)
    for b, L in enumerate(lens):
        if L:
            at = slice(c.starts[b] * ps, c.starts[b] * ps + L)
            left[at] = False
            want = c.held(b)
            assert torch.equal(k[at].double(), want[0]) and torch.equal(v[at].double(), want[1])
    # slots behind a row's length keep what they held
    assert bool(torch.isnan(k[left]).all()) and bool(torch.isnan(v[left]).all())


@pytest.mark.parametrize("Hkv,D,ps", [(1, 64, 1), (3, 64, 7), (1, 128, 16), (2, 64, 5)])
def test_read_of_many_slots(Hkv, D, ps):
    """Enough slots that a warp takes several, with odd shares and rows that end inside one."""
    test_read(Hkv, D, ps, [9001, 0, 1, 13, 40007, 3, 0, 5 * 4864 + 2])


def test_read_flags():
    c = Cache([9, 30, 5], 2, 2, 64, 4, seed=1, max_seq_len=20).fill()
    k, v = (torch.zeros(c.n_ref, 4, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def read(indices=None, indptr=None, lens=None):
        k.fill_(-1.0)
        v.fill_(-1.0)
        c.status.zero_()
        pkv.paged_kv_read_q8(c.d, *c.q8, c.kv_indices if indices is None else indices,
                             c.kv_indptr if indptr is None else indptr,
                             c.seq_lens if lens is None else lens, k, v, status=c.status)
        there = (k.view(-1, 128) != -1).any(1)
        return int(c.status.item()), [int(there[c.starts[b] * 4:c.starts[b + 1] * 4].sum()) for b in range(3)]

    assert read() == (pkv.FLAG_BAD_LEN, [9, 0, 5])                # 30 is over max_seq_len
    lens = c.seq_lens.clone()
    lens[1] = -4
    assert read(lens=lens) == (pkv.FLAG_BAD_LEN, [9, 0, 5])
    lens[1] = 20
    ind = c.kv_indices.clone()
    ind[c.starts[0] + 1] = c.n_pool
    assert read(ind, lens=lens) == (pkv.FLAG_BAD_PAGE, [5, 20, 5])
    short = c.kv_indptr.clone()
    short[2] -= 4                                                  # row 1's table: 16 tokens
    lens[2] = 0
    assert read(indptr=short, lens=lens) == (pkv.FLAG_BAD_PAGE, [9, 16, 0])
    short[2] = c.n_ref + 1                                         # past the table
    assert read(indptr=short, lens=lens)[0] == pkv.FLAG_BAD_PAGE


# -------------------------------------------------------------------- decoding
SHAPES = [
    # Hq, Hkv, D, page size
    (32, 8, 128, 16), (32, 8, 64, 16), (64, 8, 128, 16), (128, 8, 64, 8), (4, 2, 64, 16),
    (16, 1, 128, 16), (1, 1, 64, 1), (7, 1, 128, 5), (9, 3, 64, 3), (35, 5, 128, 24), (12, 4, 128, 64),
    (64, 4, 64, 32), (16, 16, 128, 16), (48, 16, 64, 128), (22, 2, 128, 1), (30, 6, 64, 17),
    (60, 12, 128, 16), (26, 2, 64, 16),
]


@pytest.mark.parametrize("Hq,Hkv,D,ps", SHAPES)
def test_decode(Hq, Hkv, D, ps):
    c = Cache([37, 1, 0, 300, 16, 129, 17, 1000], Hq, Hkv, D, ps, seed=Hq + D).fill()
    q = _q(c, 0.5)
    for splits in (None, 1, 5):
        out, status = c.decode(q, splits)
        assert status == 0
        c.check_decode(q, out)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (32, 8, 128), (8, 1, 128)])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 4099])
def test_decode_one_row_of_any_length(Hq, Hkv, D, L):
    c = Cache([L], Hq, Hkv, D, 16, seed=L).fill()
    q = _q(c)
    for splits in (None, 3):
        out, status = c.decode(q, splits)
        assert status == 0
        c.check_decode(q, out)


def test_decode_single_token_returns_its_value():
    c = Cache([1, 1, 1], 8, 2, 128, 16, seed=2).fill()
    out, _ = c.decode(_q(c))
    for b in range(3):
        want = c.held(b)[1][0].repeat_interleave(4, 0)
        assert torch.equal(out[b].cpu().double(), want)             # codes are exact in bf16


@pytest.mark.parametrize("D", [64, 128])
def test_decode_values_of_very_different_scales(D):
    """Zero vectors, sinks with small values under a large weight, scales 80
    powers of two apart, sharp and flat softmaxes."""
    c = Cache([200, 65, 40, 500], 8, 2, D, 16, seed=9).fill(v_gain=(-40, -12))
    vs, ks = c.vs.cpu(), c.ks.cpu()
    at = c.places(1, 0, 65)
    vs[at[0][::3], at[1][::3]] = 127 + 40
    at = c.places(2, 0, 40)
    vs[at[0][:20], at[1][:20]] = 127 - 40
    vc = c.vc.cpu()
    vc[at[0][:20], at[1][:20]] = 0                                  # half the row's values are zero
    vs[at[0][20:], at[1][20:]] = 127 + 5
    c.vc.copy_(vc)
    c.vs.copy_(vs)
    c.ks.copy_(ks)
    for gain in (0.0, 0.02, 1.0, 8.0):
        q = _q(c, gain)
        out, status = c.decode(q)
        assert status == 0
        c.check_decode(q, out)


def test_decode_queries_of_any_size():
    """Queries whose heads are 2^-60 to 2^60 in size (the scores stay in range
    through the scale of their keys)."""
    c = Cache([100, 50], 8, 2, 64, 16, seed=4).fill(k_gain=(-40, -36))
    q = _q(c, 1.0)
    q[:, ::2] *= 2.0 ** 30
    q[0, 1] *= 2.0 ** -60
    q[1, 3] = 0
    out, status = c.decode(q)
    assert status == 0
    c.check_decode(q, out)


def test_decode_flags():
    c = Cache([40, 90, 64], 8, 2, 64, 16, seed=5, max_seq_len=80).fill()
    q = _q(c)
    out, status = c.decode(q)                                        # row 1 is cut to 80 tokens
    assert status == pkv.FLAG_BAD_LEN
    c.lens[1] = 80
    c.check_decode(q, out)
    c.seq_lens[1] = -7
    out, status = c.decode(q)
    assert status == pkv.FLAG_BAD_LEN and float(out[1].float().abs().max()) == 0
    c.seq_lens[1] = 80
    keep = c.kv_indices.clone()
    c.kv_indices[c.starts[0]] = c.n_pool                              # read as page 0
    out, status = c.decode(q)
    assert status == pkv.FLAG_BAD_PAGE
    c.kv_indices.copy_(keep)
    c.kv_indptr[1] -= 1                                               # row 0's table covers 32 tokens
    c.starts[1] -= 1
    out, status = c.decode(q)
    assert status & pkv.FLAG_BAD_PAGE
    want, bound = attention(q[0].cpu(), *c.held(0, 32), c.scale)
    assert bool(((out[0].cpu().double() - want).abs() <= bound).all())


def test_decode_more_rows_than_one_launch_serves():
    lens = [(i * 7) % 40 for i in range(4100)]
    c = Cache(lens, 4, 1, 64, 16, seed=6).fill()
    q = _q(c)
    out, status = c.decode(q)
    assert status == 0
    c.check_decode(q, out)


def test_decode_is_the_same_from_call_to_call():
    c = Cache([700, 33, 2000, 64], 32, 8, 128, 16, seed=7).fill()
    q = _q(c)
    first, _ = c.decode(q)
    for _ in range(3):
        again, _ = c.decode(q)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))


def test_cache_past_32_bit_offsets():
    """A pool of more than 2^32 code bytes: rows in its last pages."""
    P, ps, Hkv, D = 300_000, 16, 8, 128
    c = Cache([100, 37], 16, Hkv, D, ps, seed=11).fill()
    high = torch.arange(P - c.n_ref, P, dtype=torch.int32).flip(0)
    big = [torch.empty(P, *x.shape[1:], dtype=torch.uint8, device=DEV) for x in c.q8]
    for x, y in zip(big, c.q8):
        x[high.long().to(DEV)] = y[c.table.long().to(DEV)]
    d = pkv.dims(2, 16, Hkv, D, ps, P, c.n_ref, c.d.max_seq_len)
    q = _q(c)
    want, _ = c.decode(q)
    rows = (high.to(DEV), c.kv_indptr, c.seq_lens)
    S = pkv.plan(d)[0]
    ws, out = pkv.alloc_workspace(d, S, DEV), torch.empty_like(want)
    pkv.paged_decode_attn_q8(d, q, *big, *rows, S, ws, out)
    assert pkv.status_word(ws) == 0 and torch.equal(out, want)
    k, v, k2, v2 = (torch.zeros(c.n_ref, ps, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(4))
    pkv.paged_kv_read_q8(d, *big, *rows, k, v)
    pkv.paged_kv_read_q8(c.d, *c.q8, *c.rows, k2, v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    new = c.randn(2, Hkv, D).to(torch.bfloat16).to(DEV)
    pkv.paged_kv_append_q8(d, pkv.tokens(None, new, new), *big, *rows)
    pkv.paged_kv_append_q8(c.d, pkv.tokens(None, new, new), *c.q8, *c.rows)
    for x, y in zip(big, c.q8):
        assert torch.equal(x[high.long().to(DEV)], y[c.table.long().to(DEV)])


# -------------------------------------------------------------------- together
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 64, 16), (32, 8, 128, 16), (10, 5, 128, 8)])
def test_prompt_then_decode_steps_captured(Hq, Hkv, D, ps):
    """A prompt written into the 8-bit cache, its attention through the
    read-back pools and the prefill, then decode steps (append + attention),
    the last two of them replays of one captured graph."""
    lens, steps = [33, 1, 150], 4
    c = Cache(lens, Hq, Hkv, D, ps, seed=21, room=steps)
    B, T = 3, sum(lens)
    table = rope_table(200, D)
    qw, kw = ((1 + 0.2 * c.randn(D)).to(torch.bfloat16).to(DEV) for _ in range(2))
    new = lambda n, H: c.randn(n, H, D).to(torch.bfloat16).to(DEV)  # noqa: E731
    q, k, v = new(T, Hq), new(T, Hkv), new(T, Hkv)
    qo = torch.tensor([0, 33, 34, 184], dtype=torch.int32, device=DEV)
    how = dict(q_norm=qw, k_norm=kw, rope_cos_sin=table, rope_max_pos=200)
    q_out = torch.empty_like(q)
    pkv.paged_kv_extend_q8(c.d, pkv.tokens(q, k, v, q_out, **how), qo, *c.q8, *c.rows, status=c.status)
    k16, v16 = (torch.full((c.n_ref, ps, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV)
                for _ in range(2))
    pkv.paged_kv_read_q8(c.d, *c.q8, *c.rows, k16, v16, status=c.status)
    flat = pkv.dims(B, Hq, Hkv, D, ps, c.n_ref, c.n_ref, c.d.max_seq_len)
    out = torch.empty_like(q)
    ids = torch.arange(c.n_ref, dtype=torch.int32, device=DEV)
    pkv.paged_prefill_attn(flat, q_out, qo, k16, v16, ids, c.kv_indptr, c.seq_lens, out, status=c.status,
                           max_q_len=150)
    assert int(c.status.item()) == 0
    for b, L in enumerate(lens):                        # a row's last query sees all of it
        at = int(qo[b + 1]) - 1
        want, bound = attention(q_out[at].cpu(), *c.held(b), c.scale)
        # the prefill rounds its weights to bf16: 2^-8 of them
        kk, vv = c.held(b)
        w = torch.softmax(torch.einsum("grd,lgd->grl", q_out[at].cpu().double().view(Hkv, -1, D), kk) * c.scale, -1)
        size = torch.einsum("grl,lgd->grd", w, vv.abs()).reshape(Hq, D)
        assert bool(((out[at].cpu().double() - want).abs() <= bound + size * 2.0 ** -7).all())

    q1, k1, v1 = new(B, Hq), new(B, Hkv), new(B, Hkv)
    q_out1, out1 = torch.empty_like(q1), torch.empty_like(q1)
    S = pkv.plan(c.d)[0]
    ws = pkv.alloc_workspace(c.d, S, DEV)

    def step():
        c.seq_lens.add_(1)
        pkv.paged_kv_append_q8(c.d, pkv.tokens(q1, k1, v1, q_out1, **how), *c.q8, *c.rows,
                               status=ws[:4].view(torch.int32))
        pkv.paged_decode_attn_q8(c.d, q_out1, *c.q8, *c.rows, S, ws, out1)

    def check():
        assert torch.equal(c.seq_lens.cpu(), torch.tensor(c.lens, dtype=torch.int32))
        assert pkv.status_word(ws) == 0
        c.check_decode(q_out1, out1)
        for b, L in enumerate(c.lens):
            want, off = norm_rotate(q1[b:b + 1].cpu(), qw.cpu(), table[L - 1:L].cpu())
            assert bool(((q_out1[b].cpu().double() - want[0]).abs() <= want[0].abs() * 2.0 ** -8 + off[0] * 1.01).all())

    for i in range(steps):
        for x, H in ((q1, Hq), (k1, Hkv), (v1, Hkv)):
            x.copy_(new(B, H))
        c.lens = [L + 1 for L in c.lens]
        if i == 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if i < 2:
            step()
        else:
            graph.replay()
        check()


def test_norm_write_then_bf16_decode_step():
    """paged_kv_append_norm before paged_decode_attn: a decode step of a model
    with normed queries and keys on the bf16 cache."""
    c = Cache([40, 129, 1], 8, 2, 128, 16, seed=31)
    table = rope_table(256, 128)
    qw, kw = ((1 + 0.2 * c.randn(128)).to(torch.bfloat16).to(DEV) for _ in range(2))
    new = lambda n, H: c.randn(n, H, 128).to(torch.bfloat16).to(DEV)  # noqa: E731
    how = dict(q_norm=qw, k_norm=kw, rope_cos_sin=table, rope_max_pos=256)
    qo = torch.tensor([0, 39, 167, 167], dtype=torch.int32, device=DEV)
    before = torch.tensor([39, 128, 0], dtype=torch.int32, device=DEV)
    q, k, v = new(167, 8), new(167, 2), new(167, 2)
    pkv.paged_kv_extend_norm(c.d, pkv.tokens(None, k, v, k_norm=kw, rope_cos_sin=table, rope_max_pos=256),
                             qo, c.k16, c.v16, c.kv_indices, c.kv_indptr, before, status=c.status)
    q, k, v = new(3, 8), new(3, 2), new(3, 2)
    q_out, out = torch.empty_like(q), torch.empty_like(q)
    pkv.paged_kv_append_norm(c.d, pkv.tokens(q, k, v, q_out, **how), c.k16, c.v16, *c.rows, status=c.status)
    S = pkv.plan(c.d)[0]
    ws = pkv.alloc_workspace(c.d, S, DEV)
    pkv.paged_decode_attn(c.d, q_out, c.k16, c.v16, *c.rows, S, ws, out)
    assert int(c.status.item()) == 0 and pkv.status_word(ws) == 0
    for b, L in enumerate(c.lens):
        at = c.places(b, 0, L)
        kk, vv = c.k16.cpu()[at].double(), c.v16.cpu()[at].double()
        want, bound = attention(q_out[b].cpu(), kk, vv, c.scale)
        # paged_decode_attn rounds its weights to bf16: 2^-8 of them
        w = torch.softmax(torch.einsum("grd,lgd->grl", q_out[b].cpu().double().view(2, 4, 128), kk) * c.scale, -1)
        size = torch.einsum("grl,lgd->grd", w, vv.abs()).reshape(8, 128)
        assert bool(((out[b].cpu().double() - want).abs() <= bound + size * 2.0 ** -7).all())


# ------------------------------------------------------------- plans and errors
def _ws(c, S):
    return pkv.alloc_workspace(c.d, S, DEV)


@pytest.mark.parametrize("Hq,Hkv,D,ps", [(32, 8, 128, 16), (8, 2, 64, 16), (5, 1, 64, 7), (48, 16, 128, 16)])
def test_planned_calls_give_the_same_bits(Hq, Hkv, D, ps):
    """On a plan of its own making, and on one that the bf16 decode made (which it
    does not use); the bf16 decode on either."""
    c = Cache([700, 0, 33, 64, 1, 2000], Hq, Hkv, D, ps, seed=D + Hkv).fill()
    c.k16.normal_()
    c.v16.normal_()
    q = _q(c)
    for S in (pkv.plan(c.d)[0], 3, 1):
        want, _ = c.decode(q, S)
        want16 = torch.empty_like(want)
        ws = _ws(c, S)
        pkv.paged_decode_attn(c.d, q, c.k16, c.v16, *c.rows, S, ws, want16)
        for make in ("bf16", "plan", "plan_q8", "q8"):
            ws = _ws(c, S)
            out = torch.full_like(want, float("nan"))
            if make == "bf16":
                pkv.paged_decode_attn(c.d, q, c.k16, c.v16, *c.rows, S, ws, out)
            elif make == "plan":
                pkv.paged_decode_plan(c.d, *c.rows, S, ws)
            elif make == "plan_q8":
                pkv.paged_decode_plan_q8(c.d, *c.rows, S, ws)
            else:
                pkv.paged_decode_attn_q8(c.d, q, *c.q8, *c.rows, S, ws, out)
            out.fill_(float("nan"))
            pkv.paged_decode_attn_q8_planned(c.d, q, *c.q8, *c.rows, S, ws, out)
            assert torch.equal(out.view(torch.int16), want.view(torch.int16)), make
            out.fill_(float("nan"))
            pkv.paged_decode_attn_planned(c.d, q, c.k16, c.v16, *c.rows, S, ws, out)
            assert torch.equal(out.view(torch.int16), want16.view(torch.int16)), make
            assert pkv.status_word(ws) == 0


def test_planned_call_on_another_shapes_plan():
    """A plan for another grid or batch is not used, nor what it left for the
    join of the pieces."""
    c, other = (Cache(lens, 8, 2, 64, 16, seed=3).fill() for lens in ([300, 40], [10, 500, 77]))
    c.k16.normal_()
    c.v16.normal_()
    S = pkv.plan(c.d)[0]
    q = _q(c)
    want, _ = c.decode(q, S)
    ws, want16 = _ws(c, S), torch.empty_like(want)
    pkv.paged_decode_attn(c.d, q, c.k16, c.v16, *c.rows, S, ws, want16)
    for splits in (S, 64):
        ws, out = pkv.alloc_workspace(other.d, 64, DEV), torch.empty_like(want)
        pkv.paged_decode_plan_q8(other.d, *other.rows, splits, ws)
        pkv.paged_decode_attn_q8_planned(c.d, q, *c.q8, *c.rows, S, ws, out)
        assert torch.equal(out, want)
        ws = pkv.alloc_workspace(other.d, 64, DEV)
        pkv.paged_decode_plan(other.d, *other.rows, splits, ws)
        pkv.paged_decode_attn_planned(c.d, q, c.k16, c.v16, *c.rows, S, ws, out)
        assert torch.equal(out, want16)


def test_not_a_number_is_not_lost_in_the_join():
    """A NaN key or value in one piece of a row that many blocks share."""
    c = Cache([3000, 50], 8, 2, 64, 16, seed=12).fill()
    q = _q(c)
    ok, _ = c.decode(q)
    at = c.places(0, 1234, 1235)
    c.kc[at[0][0], at[1][0], 1, 7] = 0x7F
    bad, _ = c.decode(q)
    assert bool(torch.isnan(bad[0, 4:].float()).all())                # kv head 1 serves heads 4-7
    assert torch.equal(bad[0, :4], ok[0, :4]) and torch.equal(bad[1], ok[1])
    c.kc[at[0][0], at[1][0], 1, 7] = 0
    c.vc[at[0][0], at[1][0], 0, 9] = 0xFF
    bad, _ = c.decode(q)
    nan = torch.isnan(bad[0, :4].float())
    assert bool(nan[:, 9].all()) and int(nan.sum()) == 4
    # an infinite query makes its own head NaN and no other
    c.vc[at[0][0], at[1][0], 0, 9] = 0
    ok, _ = c.decode(q)
    q[0, 2, 5] = float("inf")
    bad, _ = c.decode(q)
    assert bool(torch.isnan(bad[0, 2].float()).all())
    assert torch.equal(bad[0, [0, 1, 3]], ok[0, [0, 1, 3]]) and torch.equal(bad[1], ok[1])


def test_handoff_timeout_sets_flag_and_the_next_call_is_right():
    c = Cache([5000, 100], 32, 8, 128, 16, seed=13).fill()
    q = _q(c)
    want, _ = c.decode(q)
    try:
        pkv.testing_set_handoff_wait_ns(0)
        _, status = c.decode(q)
        assert status & pkv.FLAG_TIMEOUT
    finally:
        pkv.testing_set_handoff_wait_ns(pkv.DEFAULT_HANDOFF_WAIT_NS)
    out, status = c.decode(q)
    assert status == 0 and torch.equal(out, want)


def test_two_streams_at_once():
    """Two caches written and read on two streams, each with its own workspace."""
    cases = [Cache([900, 41, 7], 16, 4, 128, 16, seed=s).fill() for s in (1, 2)]
    qs = [_q(c) for c in cases]
    want = [c.decode(q)[0] for c, q in zip(cases, qs)]
    streams = [torch.cuda.Stream() for _ in cases]
    S = [pkv.plan(c.d)[0] for c in cases]
    ws = [_ws(c, s) for c, s in zip(cases, S)]
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for i in range(20):
        for n, c in enumerate(cases):
            pkv.paged_decode_attn_q8(c.d, qs[n], *c.q8, *c.rows, S[n], ws[n], outs[n][i], stream=streams[n])
    torch.cuda.synchronize()
    for n in range(2):
        assert all(torch.equal(o, want[n]) for o in outs[n])


def test_two_graphs_share_a_workspace():
    c = Cache([900, 41, 7], 16, 4, 64, 16, seed=5).fill()
    S = pkv.plan(c.d)[0]
    ws = _ws(c, S)
    q = [_q(c), _q(c)]
    want = [c.decode(x)[0] for x in q]
    out = [torch.empty_like(w) for w in want]
    graphs = []
    for x, o in zip(q, out):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_decode_attn_q8(c.d, x, *c.q8, *c.rows, S, ws, o)
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, out):
            o.zero_()
            g.replay()
    assert all(torch.equal(o, w) for o, w in zip(out, want))


def test_shared_pages_and_the_same_page_twice():
    """Rows that share a prefix's pages, and a row that names one page twice."""
    c = Cache([64, 64, 48], 8, 2, 64, 16, seed=8).fill()
    c.kv_indices[4:6] = c.kv_indices[0:2]
    c.kv_indices[10] = c.kv_indices[9]
    c.table.copy_(c.kv_indices.cpu())
    q = _q(c)
    out, status = c.decode(q)
    assert status == 0
    c.check_decode(q, out)


@pytest.mark.parametrize("Hq,Hkv,D,ps", [(4, 2, 64, 16), (32, 8, 128, 16), (5, 1, 64, 1), (48, 3, 128, 7),
                                         (64, 16, 64, 32)])
@pytest.mark.parametrize("most", [1, 16, 128, 257])
def test_decode_short_rows(Hq, Hkv, D, ps, most):
    """Short rows are not split (the limit is in bytes of a group of heads: 256
    tokens and more here); more rows than blocks, empty ones among them, planned
    and not, whatever the split count."""
    lens = [(i * 37) % (most + 1) for i in range(331)]
    c = Cache(lens, Hq, Hkv, D, ps, seed=most, max_seq_len=most).fill()
    q = _q(c)
    for S in (pkv.plan(c.d)[0], 1):
        ws, out = _ws(c, S), torch.full((331, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        pkv.paged_decode_attn_q8(c.d, q, *c.q8, *c.rows, S, ws, out)
        assert pkv.status_word(ws) == 0
        c.check_decode(q, out)
        again = torch.full_like(out, float("nan"))
        pkv.paged_decode_attn_q8_planned(c.d, q, *c.q8, *c.rows, S, ws, again)
        assert torch.equal(out, again)


def test_decode_short_rows_flags():
    c = Cache([40, 90, 64], 8, 2, 64, 16, seed=5, max_seq_len=80).fill()
    c.seq_lens[0] = -3
    c.kv_indices[c.starts[2]] = -1
    q = _q(c)
    out, status = c.decode(q)
    assert status == pkv.FLAG_BAD_LEN | pkv.FLAG_BAD_PAGE
    assert float(out[0].float().abs().max()) == 0
    want, bound = attention(q[1].cpu(), *c.held(1, 80), c.scale)        # cut to 80 tokens
    assert bool(((out[1].cpu().double() - want).abs() <= bound).all())
