"""The 8-bit decode's split path (partition, plan, join of the pieces): every case
here has a max_seq_len that keeps its rows off the whole-row path, and says so."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import pkv
from q8_cases import DEV, Cache
from test_q8_precision_gpu import _reference

pytestmark = pytest.mark.gpu

LONG = 1 << 14                     # over any group of heads' limit for whole rows
HEADER = 256


def _q(c):
    return c.randn(len(c.lens), c.Hq, c.D).to(torch.bfloat16).to(DEV)


def _words_written(ws, first, last, call):
    """32-bit words of ws[first:last] that `call` writes (bytes)."""
    ws[first:last] = 0x5A
    call()
    return int((ws[first:last].view(torch.int32) != 0x5A5A5A5A).sum())


@pytest.mark.parametrize("Hq,Hkv,D,lens", [(32, 8, 128, [700, 0, 3, 4000]), (5, 1, 64, [9000]),
                                           (6, 3, 64, [70] * 100)])
def test_a_plan_is_the_partition_and_nothing_else(Hq, Hkv, D, lens):
    """No block's entry is left in the workspace: no call over an 8-bit cache reads one."""
    c = Cache(lens, Hq, Hkv, D, 16, seed=2, max_seq_len=LONG).fill()
    S = pkv.plan(c.d)[0]
    ws = pkv.alloc_workspace(c.d, S, DEV)
    parts = pkv.workspace_layout(c.d, S)[0]
    rows = len(lens) * (Hkv // next(h for h in (8, 4, 2, 1) if Hkv % h == 0))
    most = 7 + rows + 1 + 2 * rows                # a header, the prefix sums, two words a row
    q, out = _q(c), torch.empty(len(lens), Hq, D, dtype=torch.bfloat16, device=DEV)
    plan = lambda: pkv.paged_decode_plan_q8(c.d, *c.rows, S, ws)  # noqa: E731
    call = lambda: pkv.paged_decode_attn_q8(c.d, q, *c.q8, *c.rows, S, ws, out)  # noqa: E731
    for make in (plan, call):
        n = _words_written(ws, HEADER, parts, make)
        assert 7 + rows < n <= most, (n, most)
    c.check_decode(q, out)
    want = out.clone()
    for make in (plan, call):
        make()
        out.fill_(float("nan"))
        pkv.paged_decode_attn_q8_planned(c.d, q, *c.q8, *c.rows, S, ws, out)
        assert torch.equal(out, want)
    assert pkv.status_word(ws) == 0


def _path_splits(c, q, S, d=None):
    """Whether the call cuts rows: it then leaves partials in the workspace."""
    d = d or c.d
    ws = pkv.alloc_workspace(d, S, DEV)
    out = torch.empty(d.B, c.Hq, c.D, dtype=torch.bfloat16, device=DEV)
    call = lambda: pkv.paged_decode_attn_q8(d, q, *c.q8, *c.rows, S, ws, out)  # noqa: E731
    return _words_written(ws, HEADER, pkv.workspace_layout(d, S)[0], call) > 0


def _splits_and_is_right(c, splits=(None, 1, 5)):
    q = _q(c)
    for S in splits:
        assert _path_splits(c, q, S or pkv.plan(c.d)[0])
        out, status = c.decode(q, S)
        assert status == 0
        c.check_decode(q, out)


@pytest.mark.parametrize("Hq,Hkv,D,ps", [
    (16, 1, 128, 16), (1, 1, 64, 1), (7, 1, 128, 5), (9, 3, 64, 3), (35, 5, 128, 24), (22, 2, 128, 1), (30, 6, 64, 17),
    (26, 2, 64, 16), (4, 2, 64, 16), (64, 4, 64, 32), (60, 12, 128, 16), (48, 16, 64, 128), (128, 8, 128, 16)])
def test_every_group_of_heads(Hq, Hkv, D, ps):
    _splits_and_is_right(Cache([37, 1, 0, 300, 16, 129, 17, 1000], Hq, Hkv, D, ps, seed=Hq + D,
                               max_seq_len=LONG).fill())


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (1, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 257, 4099])
def test_one_row_of_any_length(Hq, Hkv, D, L):
    _splits_and_is_right(Cache([L], Hq, Hkv, D, 16, seed=L, max_seq_len=LONG).fill(), (None, 3))


@pytest.mark.parametrize("Hq,Hkv,B", [(4, 1, 1100), (6, 3, 700), (5, 5, 2100)])
def test_more_rows_than_one_launch_takes(Hq, Hkv, B):
    """Two and more pairs of launches, one after the other, with one set of partials;
    no plan, so a planned call gives the same."""
    c = Cache([(i * 7) % 190 for i in range(B)], Hq, Hkv, 64, 16, seed=6, max_seq_len=LONG).fill()
    assert B * Hkv > 1024
    q = _q(c)
    S = pkv.plan(c.d)[0]
    assert _path_splits(c, q, S)
    ws = pkv.alloc_workspace(c.d, S, DEV)
    first, again = (torch.full((B, Hq, 64), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pkv.paged_decode_plan_q8(c.d, *c.rows, S, ws)
    for out, call in ((first, pkv.paged_decode_attn_q8), (again, pkv.paged_decode_attn_q8_planned)):
        call(c.d, q, *c.q8, *c.rows, S, ws, out)
        assert pkv.status_word(ws) == 0
        c.check_decode(q, out)
    assert torch.equal(first, again)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S", [None, 7])
def test_pieces_whose_values_are_of_very_different_scales(D, S):
    """Rows cut into pieces of which some hold values 50 powers of two larger, some
    only zeros: their bases lie far apart when they are joined.

    The bound has a term for weights under f16's normal range: a weight w 2^e that is
    at most 2^15 above and 7 under base is rounded to a step of 2^-24, so it is off by
    at most 2^-25 2^base <= 2^-25 2^-7 of the row's largest w 2^e, times its code.
    Where the tokens of a row's largest weights hold zeros (row 1 at the highest gain,
    whose output is 2^-30 of its values) this is all there is."""
    c = Cache([5000, 650, 2000], 8, 2, D, 16, seed=9, max_seq_len=LONG).fill(v_gain=(-40, -30))
    vs, vc = c.vs.cpu(), c.vc.cpu()
    at = c.places(0, 1000, 1400)
    vs[at[0], at[1]] = 127 + 20
    at = c.places(1, 0, 300)
    vc[at[0], at[1]] = 0
    at = c.places(2, 1999, 2000)
    vs[at[0], at[1]] = 127 + 40
    c.vc.copy_(vc)
    c.vs.copy_(vs)
    for gain in (0.0, 0.02, 1.0, 8.0):
        q = (c.randn(3, 8, D) * gain).to(torch.bfloat16).to(DEV)
        assert _path_splits(c, q, S or pkv.plan(c.d)[0])
        out, status = c.decode(q, S)
        assert status == 0
        for b in range(3):
            want, bound = _reference(c, b, q[b].cpu())
            off = (out[b].cpu().double() - want).abs()
            assert bool((off <= bound).all()), (gain, b, float((off / bound.clamp(min=1e-300)).max()))


def test_flags_of_rows_that_are_cut():
    c = Cache([400, 900, 640], 8, 2, 64, 16, seed=5, max_seq_len=LONG).fill()
    q = _q(c)
    want, _ = c.decode(q)
    d = pkv.dims(3, 8, 2, 64, 16, c.n_pool, c.n_ref, LONG)
    c.seq_lens[1] = LONG + 1                       # cut to what the table covers: 57 pages
    out, status = c.decode(q)
    assert status == pkv.FLAG_BAD_LEN | pkv.FLAG_BAD_PAGE
    for b in (0, 2):                                # the other rows' pieces lie elsewhere now
        right, bound = _reference(c, b, q[b].cpu())
        assert bool(((out[b].cpu().double() - right).abs() <= bound).all())
    c.seq_lens[1] = -7
    out, status = c.decode(q)
    assert status == pkv.FLAG_BAD_LEN and float(out[1].float().abs().max()) == 0
    c.seq_lens[1] = 900
    keep = c.kv_indices.clone()
    c.kv_indices[c.starts[0] + 3] = c.n_pool                          # read as page 0
    out, status = c.decode(q, d=d)
    assert status == pkv.FLAG_BAD_PAGE
    c.kv_indices.copy_(keep)
    out, status = c.decode(q)
    assert status == 0 and torch.equal(out, want)


def test_planned_call_on_another_shapes_split_plan():
    c, other = (Cache(lens, 8, 2, 64, 16, seed=3, max_seq_len=LONG).fill()
                for lens in ([3000, 40], [10, 5000, 77]))
    S = pkv.plan(c.d)[0]
    q = _q(c)
    assert _path_splits(c, q, S)
    want, _ = c.decode(q, S)
    for splits in (S, 64):
        ws, out = pkv.alloc_workspace(other.d, max(S, 64), DEV), torch.empty_like(want)
        pkv.paged_decode_plan_q8(other.d, *other.rows, splits, ws)
        pkv.paged_decode_attn_q8_planned(c.d, q, *c.q8, *c.rows, S, ws, out)
        assert torch.equal(out, want)


@pytest.mark.parametrize("Hq,Hkv,D,ps", [(5, 1, 64, 7), (8, 2, 64, 16), (16, 1, 128, 16)])
def test_planned_calls_on_split_rows_give_the_same_bits(Hq, Hkv, D, ps):
    c = Cache([700, 0, 33, 64, 1, 2000], Hq, Hkv, D, ps, seed=D + Hkv, max_seq_len=LONG).fill()
    q = _q(c)
    for S in (pkv.plan(c.d)[0], 3, 1):
        assert _path_splits(c, q, S)
        want, _ = c.decode(q, S)
        ws = pkv.alloc_workspace(c.d, S, DEV)
        pkv.paged_decode_plan_q8(c.d, *c.rows, S, ws)
        for _ in range(3):                        # a step's layers on one plan
            out = torch.full_like(want, float("nan"))
            pkv.paged_decode_attn_q8_planned(c.d, q, *c.q8, *c.rows, S, ws, out)
            assert torch.equal(out, want)
        assert pkv.status_word(ws) == 0


def test_a_plan_and_its_planned_calls_in_one_graph():
    """The plan is made anew in every replay, so a graph holds while lengths grow."""
    c = Cache([900, 41, 7, 3000], 16, 4, 64, 16, seed=5, room=64, max_seq_len=LONG).fill()
    for pool in c.q8[2:]:
        pool.clamp_(max=127)                      # room behind the lengths: finite scales and codes
    for pool in c.q8[:2]:
        pool[pool == 0x7F] = 0x30
    S = pkv.plan(c.d)[0]
    q, ws = _q(c), pkv.alloc_workspace(c.d, S, DEV)
    outs = [torch.empty(4, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(3)]

    def step():
        pkv.paged_decode_plan_q8(c.d, *c.rows, S, ws)
        for o in outs:
            pkv.paged_decode_attn_q8_planned(c.d, q, *c.q8, *c.rows, S, ws, o)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for grow in (0, 5, 59):
        c.seq_lens.add_(grow)
        c.lens = [L + grow for L in c.lens]
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            c.check_decode(q, o)
    assert pkv.status_word(ws) == 0
