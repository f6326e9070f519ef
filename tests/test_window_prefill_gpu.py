"""GPU tests of paged_prefill_attn_window against 64 bits."""

import math

import pytest
import torch

from paged_kv_gqa_16_gb300 import pkv
from q4_cases import Cache, fill16
from q8_cases import DEV

pytestmark = pytest.mark.gpu


def _case(Hq, Hkv, D, ps, lens, chunks, seed=0, **kw):
    c = fill16(Cache(lens, Hq, Hkv, D, ps, seed=seed, **kw))
    ends = torch.tensor([0] + list(chunks)).cumsum(0)
    q = c.randn(int(ends[-1]), Hq, D).to(torch.bfloat16).to(DEV)
    return c, q, ends


def _seen(L, n, window, sinks):
    """[n, L]: what the row's last n tokens see."""
    p, t = torch.arange(L - n, L)[:, None], torch.arange(L)
    m = t <= p
    return m if window == 0 else m & ((t > p - window) | (t < sinks))


def _unread(c, chunks, window, sinks):
    """The table with ids outside the pool at pages that no query sees."""
    table = c.table.clone()
    for b, (L, n) in enumerate(zip(c.lens, chunks)):
        some = _seen(L, n, window, sinks).any(0) if n else torch.zeros(L, dtype=torch.bool)
        for i in range(-(-L // c.ps)):
            if not bool(some[i * c.ps:(i + 1) * c.ps].any()):
                table[c.starts[b] + i] = (-7, c.n_pool, 1 << 30)[i % 3]
    return table.to(DEV)


def _run(c, q, ends, window, sinks, rows=None, ws=None, max_q=None, d=None, status=None):
    out = torch.full_like(q, float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device=DEV) if status is None else status
    pkv.paged_prefill_attn_window(d or c.d, q, ends.to(torch.int32).to(DEV), c.k16, c.v16, *(rows or c.rows), window,
                                  sinks, out, status=status, max_q_len=max_q, workspace=ws)
    return out, int(status)


def _check(c, q, out, ends, window, sinks):
    """Bound: the output's rounding (2^-8), the weights' (2^-8 of each, in the sum
    too), a part's of a key split (2^-8), and the scores' error (128 products and
    sums of 2^-23 each at most, so under 2^-16 of sum |q k|, twice)."""
    for b, L in enumerate(c.lens):
        a, e = int(ends[b]), int(ends[b + 1])
        n = e - a
        if n == 0:
            continue
        at = c.places(b, 0, L)
        k, v = (x.cpu()[at].double().to(DEV) for x in (c.k16, c.v16))
        qq = q[a:e].double().view(n, c.Hkv, -1, c.D)
        x = torch.einsum("ngrd,lgd->grnl", qq, k) * c.scale
        m = _seen(L, n, window, sinks).to(DEV)
        w = torch.softmax(x.masked_fill(~m, -math.inf), -1)
        want = torch.einsum("grnl,lgd->ngrd", w, v).reshape(n, c.Hq, c.D)
        size = torch.einsum("grnl,lgd->ngrd", w, v.abs()).reshape(n, c.Hq, c.D)
        far = float(torch.einsum("ngrd,lgd->grnl", qq.abs(), k.abs()).max()) * c.scale * 2.0 ** -16
        bound = want.abs() * 2.0 ** -8 + size * (3 * 2.0 ** -8 + 2 * far)
        off = (out[a:e].double() - want).abs()
        assert bool((off <= bound).all()), (b, L, n, float((off / bound).max()))


def _workspace(D):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return torch.empty(pkv.prefill_workspace_bytes(D, sms), dtype=torch.uint8, device=DEV)


SHAPES = [  # Hq, Hkv, D, page size
    (32, 8, 128, 16), (8, 2, 64, 16), (4, 4, 128, 64), (6, 2, 64, 24), (16, 1, 128, 8), (7, 1, 64, 256),
    (5, 1, 128, 3),
]
ROWS = [  # lengths, chunks
    ([700, 300, 1, 0, 64, 513], [700, 129, 1, 0, 64, 40]),
    ([2050, 40], [3, 17]),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rows", [0, 1])
@pytest.mark.parametrize("split", [False, True])
def test_against_64_bits(shape, rows, split):
    lens, chunks = ROWS[rows]
    c, q, ends = _case(*shape, lens, chunks)
    ws = _workspace(shape[2]) if split else None
    for window, sinks in [(0, 0), (1, 0), (1, 1), (7, 130), (64, 4), (128, 0), (129, 128), (300, 5), (1500, 300),
                          (9000, 4)]:
        table = (_unread(c, chunks, window, sinks), c.kv_indptr, c.seq_lens)
        out, status = _run(c, q, ends, window, sinks, rows=table, ws=ws, max_q=max(chunks))
        assert status == 0, (window, sinks, status)
        _check(c, q, out, ends, window, sinks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [3, 24, 40, 136, 384, 1000])
def test_page_sizes(ps, D):
    """Sizes with a power-of-two part are copied by its boxes, others key by key; the keys
    and their blocks, so the sums, are those of any page size."""
    lens, chunks = [700, 300, 1, 0, 64, 513, 2050], [700, 129, 1, 0, 64, 40, 130]
    ref, q, ends = _case(8, 2, D, 16, lens, chunks, seed=2)
    c, _, _ = _case(8, 2, D, ps, lens, chunks, seed=3)
    for b, L in enumerate(lens):
        if L:
            for of, to in ((ref.k16, c.k16), (ref.v16, c.v16)):
                to[tuple(x.to(DEV) for x in c.places(b, 0, L))] = of[tuple(x.to(DEV) for x in ref.places(b, 0, L))]
    want, status = _run(ref, q, ends, 0, 0)
    assert status == 0
    out, status = _run(c, q, ends, 0, 0)
    assert status == 0 and torch.equal(out, want)
    for window, sinks in [(1, 1), (64, 4), (129, 0), (300, 130)]:
        table = (_unread(c, chunks, window, sinks), c.kv_indptr, c.seq_lens)
        out, status = _run(c, q, ends, window, sinks, rows=table)
        assert status == 0
        _check(c, q, out, ends, window, sinks)


def test_no_window_is_the_prefill():
    c, q, ends = _case(16, 4, 128, 16, [500, 77], [200, 77], seed=1)
    for window, sinks in ((0, 0), (0, 9), (c.d.max_seq_len, 0), (c.d.max_seq_len - 4, 4)):
        out, _ = _run(c, q, ends, window, sinks)
        want = torch.empty_like(q)
        pkv.paged_prefill_attn(c.d, q, ends.to(torch.int32).to(DEV), c.k16, c.v16, *c.rows, want)
        assert torch.equal(out, want)


@pytest.mark.parametrize("ps", [16, 24])
def test_unseen_pages_may_hold_anything(ps):
    """NaN in every page and slot that no query of a row sees (the table still names
    them), with and without the copy engine."""
    lens, chunks, window, sinks = [900, 400], [50, 33], 200, 5
    c, q, ends = _case(8, 2, 128, ps, lens, chunks, seed=2)
    for b, (L, n) in enumerate(zip(lens, chunks)):
        some = _seen(L, n, window, sinks).any(0)
        for i in range(-(-L // ps)):
            if not bool(some[i * ps:(i + 1) * ps].any()):
                page = int(c.table[c.starts[b] + i])
                c.k16[page] = float("inf")
                c.v16[page] = float("nan")
    for ws in (None, _workspace(128)):
        out, status = _run(c, q, ends, window, sinks, ws=ws, max_q=50)
        assert status == 0
        # (the reference reads them: zeros there)
        keep = c.k16.clone(), c.v16.clone()
        c.k16.nan_to_num_(0.0, 0.0, 0.0)
        c.v16.nan_to_num_(0.0)
        _check(c, q, out, ends, window, sinks)
        c.k16.copy_(keep[0])
        c.v16.copy_(keep[1])


def test_flags_and_unwritten_rows():
    lens, chunks = [300, 40, 90], [100, 40, 10]
    c, q, ends = _case(8, 2, 64, 16, lens, chunks, seed=3)
    table = c.kv_indices.clone()
    table[c.starts[0] + 18] = c.n_pool              # seen by row 0's last queries
    out, status = _run(c, q, ends, 64, 4, rows=(table, c.kv_indptr, c.seq_lens))
    assert status == pkv.FLAG_BAD_PAGE
    bad = c.seq_lens.clone()
    bad[1] = 39                                     # a chunk longer than its row
    out, status = _run(c, q, ends, 64, 4, rows=(c.kv_indices, c.kv_indptr, bad))
    assert status == pkv.FLAG_BAD_LEN
    a, e = int(ends[1]), int(ends[2])
    assert bool(out[a:e].isnan().all()) and not bool(out[:a].isnan().any()) and not bool(out[e:].isnan().any())


def test_graph_and_repeats():
    c, q, ends = _case(32, 8, 128, 16, [1500, 800, 300], [256, 256, 256], seed=4)
    ws = _workspace(128)
    first, status = _run(c, q, ends, 333, 4, ws=ws, max_q=256)
    assert status == 0
    _check(c, q, first, ends, 333, 4)
    out, qo = torch.empty_like(q), ends.to(torch.int32).to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_prefill_attn_window(c.d, q, qo, c.k16, c.v16, *c.rows, 333, 4, out, max_q_len=256, workspace=ws)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, _ = _run(c, q, ends, 333, 4, ws=ws, max_q=256)
    torch.cuda.synchronize()
    assert torch.equal(other, first)


def test_long_row_past_a_window():
    """A chunk at the end of a long row: the list leaves out most blocks."""
    c, q, ends = _case(8, 1, 128, 128, [70000], [130], seed=5, spare=3)
    for window, sinks in ((1, 0), (4096, 4), (50000, 1000)):
        out, status = _run(c, q, ends, window, sinks, ws=_workspace(128), max_q=130)
        assert status == 0
        _check(c, q, out, ends, window, sinks)


def test_rows_behind_the_last_chunk_stay():
    c, q, ends = _case(8, 2, 128, 16, [300, 200], [70, 33], seed=6)
    more = torch.cat([q, torch.full((9, 8, 128), float("nan"), dtype=torch.bfloat16, device=DEV)])
    out, status = _run(c, more, ends, 64, 4)
    assert status == 0 and bool(out[-9:].isnan().all())
    _check(c, q, out[:-9], ends, 64, 4)
