"""GPU tests of the decode over the 4-bit cache and through sliding windows,
against 64 bits."""

import pytest
import torch

import q4_cases
from paged_kv_gqa_16_gb300 import pkv
from q4_cases import Cache, check, decode, fill16, unread
from q8_cases import DEV

pytestmark = pytest.mark.gpu

SHAPES = [  # Hq, Hkv, D, page size
    (32, 8, 128, 16), (16, 16, 64, 16), (4, 4, 128, 24), (8, 1, 64, 1), (8, 2, 64, 17), (12, 2, 128, 8),
    (7, 1, 128, 128), (16, 1, 64, 32), (32, 2, 128, 16), (64, 4, 64, 64), (15, 5, 64, 3), (160, 10, 64, 16),
]
WINDOWS = [(0, 0), (1, 0), (1, 3), (16, 4), (33, 17), (200, 130), (5000, 4)]
LENS = [1, 0, 2, 15, 16, 17, 37, 64, 100, 300, 513]


def _cache(shape, lens, bits, seed=0, **kw):
    c = Cache(lens, *shape, seed=seed, **kw)
    return c.fill() if bits == 4 else fill16(c)


def _q(c, seed=1, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(len(c.lens), c.Hq, c.D, generator=g) * gain).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("shape", SHAPES)
def test_whole_rows(shape, bits):
    """Short rows: one kernel, every window; entries of unseen pages are bad ids."""
    c = _cache(shape, LENS, bits)
    q = _q(c)
    for window, sinks in WINDOWS:
        rows = (unread(c, window, sinks), c.kv_indptr, c.seq_lens)
        out, status = decode(c, q, bits, window, sinks, rows=rows)
        assert status == 0, (window, sinks, status)
        check(c, q, out, bits, window, sinks)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (4097, 4), (2500, 1700)])
def test_split_rows(shape, window, sinks, bits):
    """Rows that the length bound lets split: pieces and their join, by several counts."""
    lens = [0, 4700, 1, 33, 900]
    c = _cache(shape, lens, bits, seed=2, max_seq_len=40000)
    q = _q(c, 3)
    rows = (unread(c, window, sinks), c.kv_indptr, c.seq_lens)
    for splits in (1, 3, 40, 152):
        out, status = decode(c, q, bits, window, sinks, splits=splits, rows=rows)
        assert status == 0
        check(c, q, out, bits, window, sinks)


@pytest.mark.parametrize("bits", [4, 16])
def test_more_rows_than_a_launch_takes(bits):
    lens = [(i * 7) % 40 for i in range(300)]
    c = _cache((10, 5, 64, 8), lens, bits, seed=4, max_seq_len=60000)
    q = _q(c, 5)
    for window, sinks in ((0, 0), (20000, 5)):
        out, status = decode(c, q, bits, window, sinks, splits=64)
        assert status == 0
        check(c, q, out, bits, window, sinks)


@pytest.mark.parametrize("bits", [4, 16])
def test_large_and_tiny_scores(bits):
    """Scores over hundreds of octaves: the running base moves."""
    c = _cache((8, 2, 128, 16), [400, 90], bits, seed=6)
    for gain in (1e-20, 30.0, 1000.0):
        q = _q(c, 7, gain)
        out, status = decode(c, q, bits, 64, 4)
        assert status == 0
        check(c, q, out, bits, 64, 4)


def test_unlike_scales_of_a_value():
    """V's scales differ by 2^20 within a token and between tokens."""
    c = Cache([200, 31], 8, 2, 128, 16, seed=8).fill(v_gain=(-12, 8))
    q = _q(c, 9)
    out, status = decode(c, q)
    assert status == 0
    check(c, q, out)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("split", [False, True])
def test_not_a_number_stays_with_its_heads(bits, split):
    """An infinite or NaN key or value that is seen reaches its kv head's outputs;
    one that is not seen reaches nothing."""
    lens = [300, 40, 77]
    c = _cache((8, 4, 64, 16), lens, bits, seed=10, max_seq_len=40000 if split else None)
    window, sinks = (6000, 4) if split else (32, 4)

    def poison(b, t, head, of_k):
        at = c.places(b, t, t + 1)
        at = int(at[0]), int(at[1])
        if bits == 4:
            (c.ks if of_k else c.vs)[at[0], at[1], head, 0] = 255
            (c.kc if of_k else c.vc)[at[0], at[1], head, :16] = 0
        else:
            (c.k16 if of_k else c.v16)[at[0], at[1], head, 5] = float("nan")

    if not split:
        poison(0, 100, 0, True)                     # unseen
        poison(0, 5, 1, False)
    poison(1, 39, 2, True)
    poison(2, 76, 3, False)
    q = _q(c, 11)
    out, status = decode(c, q, bits, window, sinks)
    assert status == 0
    out = out.cpu().view(3, 4, 2, 64)
    want_nan = torch.zeros(3, 4, dtype=torch.bool)
    want_nan[1, 2] = want_nan[2, 3] = True
    if bits == 4:
        assert torch.equal(out.isnan().all(-1).all(-1), want_nan) and torch.equal(out.isnan().any(-1).any(-1), want_nan)
    else:
        got = out.isnan().any(-1).any(-1)
        assert torch.equal(got, want_nan) and bool(out[1, 2].isnan().all())
    inf = q.clone()
    inf[0, 0, 0] = float("inf")
    out, _ = decode(c, inf, bits, window, sinks)
    assert bool(out[0, 0].isnan().all()) and not bool(out[0, 2:].isnan().any())


def test_unseen_slots_may_hold_anything():
    """Slots behind the rows' ends are NaN in every test here; here all unseen ones are."""
    c = fill16(Cache([120, 47], 8, 2, 128, 16, seed=12))
    window, sinks = 20, 3
    for b, L in enumerate(c.lens):
        for t in set(range(L)) - set(q4_cases.seen(L, window, sinks).tolist()):
            at = c.places(b, t, t + 1)
            c.k16[int(at[0]), int(at[1])] = float("inf")
            c.v16[int(at[0]), int(at[1])] = float("nan")
    q = _q(c, 13)
    out, status = decode(c, q, 16, window, sinks)
    assert status == 0
    check(c, q, out, 16, window, sinks)


@pytest.mark.parametrize("bits", [4, 16])
def test_bad_tables_are_flagged(bits):
    c = _cache((8, 2, 64, 16), [40, 70, 33], bits, seed=14)
    q = _q(c, 15)
    rows = [c.kv_indices.clone(), c.kv_indptr, c.seq_lens.clone()]
    rows[0][c.starts[1] + 4] = c.n_pool             # seen by row 1's window
    out, status = decode(c, q, bits, 32, 2, rows=rows)
    assert status == pkv.FLAG_BAD_PAGE
    rows = [c.kv_indices, c.kv_indptr, c.seq_lens.clone()]
    rows[2][0], rows[2][2] = -3, 10 ** 6
    out, status = decode(c, q, bits, 32, 2, rows=rows)
    assert status == pkv.FLAG_BAD_LEN | pkv.FLAG_BAD_PAGE
    assert bool((out[0] == 0).all())
    # the row that is in order has its output
    want, bound = q4_cases.attention(q[1].cpu(), *((x[q4_cases.seen(70, 32, 2)] for x in c.held(1)) if bits == 4 else
                                     (x.cpu()[c.places(1, 0, 70)][q4_cases.seen(70, 32, 2)].double()
                                      for x in (c.k16, c.v16))), c.scale,
                                     q4_cases.F16_EPS if bits == 4 else q4_cases.BF16_EPS)
    assert bool(((out[1].cpu().double() - want).abs() <= bound).all())


@pytest.mark.parametrize("bits", [4, 16])
def test_graph_streams_and_repeats(bits):
    """A captured call replayed on changed lengths, a call on another stream, and the
    same bits every time."""
    c = _cache((32, 8, 128, 16), [500, 3000, 60, 0], bits, seed=16, max_seq_len=20000)
    q = _q(c, 17)
    window, sinks = 6000, 4
    S = pkv.plan(c.d)[0]
    ws = pkv.alloc_workspace(c.d, S, DEV)
    first, status = decode(c, q, bits, window, sinks, splits=S, ws=ws)
    assert status == 0
    first = first.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = torch.empty_like(first)
        decode(c, q, bits, window, sinks, splits=S, ws=ws, out=other)
    torch.cuda.synchronize()
    assert torch.equal(first, other)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(first)
    args = (q, *c.q4) if bits == 4 else (q, c.k16, c.v16)
    call = ((lambda: pkv.paged_decode_attn_q4(c.d, *args, *c.rows, S, ws, out, window=window, sinks=sinks))
            if bits == 4 else
            (lambda: pkv.paged_decode_attn_window(c.d, *args, *c.rows, window, sinks, S, ws, out)))
    with torch.cuda.graph(graph):
        call()
    for lens in ([500, 3000, 60, 0], [500, 17, 0, 0], [1, 2999, 60, 0]):
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        full = c.lens
        c.lens = lens
        check(c, q, out, bits, window, sinks)
        if lens == full:
            assert torch.equal(out, first)
        c.lens = full
    assert pkv.status_word(ws) == 0


@pytest.mark.parametrize("bits", [4, 16])
def test_a_plan_of_the_bf16_decode_stays(bits):
    """The calls share a workspace with a step whose bf16 layers run on its plan."""
    c = fill16(Cache([700, 90, 2100], 16, 4, 128, 16, seed=18, max_seq_len=9000)).fill()
    q = _q(c, 19)
    S = pkv.plan(c.d)[0]
    ws = pkv.alloc_workspace(c.d, S, DEV)
    a, b = torch.empty_like(q), torch.empty_like(q)
    pkv.paged_decode_attn(c.d, q, c.k16, c.v16, *c.rows, S, ws, a)
    out, status = decode(c, q, bits, 64 if bits == 16 else 0, 4, splits=S, ws=ws)
    pkv.paged_decode_attn_planned(c.d, q, c.k16, c.v16, *c.rows, S, ws, b)
    assert torch.equal(a, b) and status == 0
    check(c, q, out, bits, 64 if bits == 16 else 0, 4)


def test_a_wait_that_runs_out_is_reported():
    c = _cache((32, 8, 128, 16), [3000] * 4, 4, seed=20, max_seq_len=20000)
    q = _q(c, 21)
    try:
        pkv.testing_set_handoff_wait_ns(0)
        _, status = decode(c, q)
    finally:
        pkv.testing_set_handoff_wait_ns(pkv.DEFAULT_HANDOFF_WAIT_NS)
    assert status == pkv.FLAG_TIMEOUT
    out, status = decode(c, q)
    assert status == 0
    check(c, q, out)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("shape", [(32, 8, 64, 16), (32, 8, 128, 16), (16, 1, 128, 16), (128, 8, 128, 16), (4, 4, 64, 3)])
def test_waits_that_run_out_on_shared_stages(shape, bits):
    """Warps that fill a stage together, and one each: all of them end, and the next call is right."""
    c = _cache(shape, [3000] * 4, bits, seed=26, max_seq_len=20000)
    q = _q(c, 27)
    try:
        pkv.testing_set_handoff_wait_ns(0)
        _, status = decode(c, q, bits)
    finally:
        pkv.testing_set_handoff_wait_ns(pkv.DEFAULT_HANDOFF_WAIT_NS)
    assert status == pkv.FLAG_TIMEOUT
    out, status = decode(c, q, bits)
    assert status == 0
    check(c, q, out, bits)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("bound", [20000, 1 << 28, (1 << 30) - 1000])
def test_a_wide_length_bound_splits_rows(bound, bits):
    """The bytes of a row of 2^28 tokens and more pass 31 bits: it is not a short one. Pieces of a
    split row are left in the workspace, a whole row leaves none."""
    c = _cache((8, 8, 64, 16), [3000], bits, seed=28, max_seq_len=bound)
    q = _q(c, 29)
    ws = pkv.alloc_workspace(c.d, 8, DEV)
    pkv.workspace_init(ws)
    ws[256:] = 0x5a
    out, status = decode(c, q, bits, splits=8, ws=ws)
    assert status == 0
    check(c, q, out, bits)
    assert bool((ws[256:] != 0x5a).any())


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("shape", [(16, 4, 128, 16), (1, 1, 64, 16)])
def test_a_plan_of_the_8_bit_decode_stays(shape, bits):
    """A step whose 8-bit layers run on their plan, with other layers between them."""
    import q8_cases
    lens = [30000, 90, 21000, 4]
    c8 = q8_cases.Cache(lens, *shape, seed=22, max_seq_len=50000).fill()
    c = _cache(shape, [700, 0, 33000, 900], bits, seed=23, max_seq_len=50000)
    q = _q(c, 24)
    S = pkv.plan(c8.d)[0]
    ws = pkv.alloc_workspace(c8.d, S, DEV)
    a, b = torch.empty_like(q), torch.empty_like(q)
    pkv.paged_decode_attn_q8(c8.d, q, *c8.q8, *c8.rows, S, ws, a)
    window = 0 if bits == 4 else 32000
    out, status = decode(c, q, bits, window, 4, splits=S, ws=ws)
    pkv.paged_decode_attn_q8_planned(c8.d, q, *c8.q8, *c8.rows, S, ws, b)
    assert torch.equal(a, b) and status == 0
    check(c, q, out, bits, window, 4)


def test_offsets_past_2_31_bytes():
    """Rows in the last pages of pools of more than 2^31 bytes each."""
    Hq, Hkv, D, ps, L = 16, 8, 128, 16, 40
    pages = (1 << 31) // (ps * Hkv * D // 2) + 1000
    c = Cache([L, 3], Hq, Hkv, D, ps, seed=25)
    small = [x.clone() for x in c.q4]
    big = [torch.empty(pages, *x.shape[1:], dtype=torch.uint8, device=DEV) for x in c.q4]
    c.kc, c.vc, c.ks, c.vs = big
    at = pages - len(small[0])
    for x, y in zip(big, small):
        x[at:] = y
    table = c.kv_indices + at
    d = pkv.dims(2, Hq, Hkv, D, ps, pages, c.n_ref, 64)
    rows = (table, c.kv_indptr, c.seq_lens)
    k, v = (c.randn(L + 3, Hkv, D).to(torch.bfloat16).to(DEV) for _ in range(2))
    ends = torch.tensor([0, L, L + 3], dtype=torch.int32, device=DEV)
    pkv.paged_kv_extend_q4(d, pkv.tokens(None, k, v), ends, *big, *rows, status=c.status)
    k16, v16 = (torch.zeros(c.n_ref, ps, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pkv.paged_kv_read_q4(d, *big, *rows, k16, v16, status=c.status)
    q = _q(c, 26)
    out, status = decode(c, q, 4, rows=rows, d=d)
    assert int(c.status) == 0 and status == 0
    for x, y in zip(big, small):
        y.copy_(x[at:])
    c.kc, c.vc, c.ks, c.vs = small
    for b, (a, e) in enumerate(((0, L), (L, L + 3))):
        for got, want in zip(c.held(b), (k, v)):
            code, scale = q4_cases.quantise(want[a:e].cpu())
            assert torch.equal(got, q4_cases.values(code, scale))
    check(c, q, out)
    flat = k16.cpu().flatten(0, 1)
    assert torch.equal(flat[:L], q4_cases.bf16_of(c.held(0)[0]))
    # bf16 pools, through a window
    pages = (1 << 30) // (ps * Hkv * D) + 1000
    big = [torch.empty(pages, ps, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    at = pages - c.n_pool
    fill16(c)
    for x, y in zip(big, (c.k16, c.v16)):
        x[at:] = y
    d = pkv.dims(2, Hq, Hkv, D, ps, pages, c.n_ref, 64)
    rows = (c.kv_indices + at, c.kv_indptr, c.seq_lens)
    S = pkv.plan(d)[0]
    ws = pkv.alloc_workspace(d, S, DEV)
    out = torch.empty_like(q)
    pkv.paged_decode_attn_window(d, q, *big, *rows, 20, 3, S, ws, out)
    check(c, q, out, 16, 20, 3)
    assert pkv.status_word(ws) == 0
    chunk = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    pkv.paged_prefill_attn_window(d, q, chunk, *big, *rows, 20, 3, out, status=c.status, max_q_len=1)
    check(c, q, out, 16, 20, 3)
    assert int(c.status) == 0
