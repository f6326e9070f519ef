"""GPU tests of the stream decode's kernels that have a pipeline of their own: many query heads
over eight kv heads, bulk copies from pages of any size, and every kernel's way out when a wait
runs out."""

import pytest
import torch

import test_stream_decode_gpu as stream
from paged_kv_gqa_16_gb300 import pkv
from q4_cases import check, decode

pytestmark = pytest.mark.gpu

# Hq, Hkv, D, page size: two tiles of query heads over eight kv heads, at D = 64 (at 4 bits stages
# of one tile, a warp each) and 128 (bulk copies at 16); bulk copies from pages of 17 and 24
SHAPES = [(128, 8, 64, 16), (128, 8, 128, 24), (32, 8, 128, 17)]


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("shape", SHAPES)
def test_whole_rows(shape, bits):
    stream.test_whole_rows(shape, bits)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (4097, 4), (2500, 1700)])
def test_split_rows(shape, window, sinks, bits):
    stream.test_split_rows(shape, window, sinks, bits)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 2, 4, 8])
@pytest.mark.parametrize("n_rep", [3, 12])
def test_every_kernel_ends_when_waits_run_out(n_rep, Hkv, D, bits):
    """Time limits at which all, some or none of the warps give up, each call with an ordinary one
    right behind it, which takes over the blocks' shared memory: its bits are those of a call
    by itself."""
    c = stream._cache((n_rep * Hkv, Hkv, D, 16), [3000, 40, 2500, 3000], bits, seed=30, max_seq_len=20000)
    q = stream._q(c, 31)
    S = pkv.plan(c.d)[0]
    first, status = decode(c, q, bits, splits=S)
    assert status == 0
    check(c, q, first, bits)
    ws, other = (pkv.alloc_workspace(c.d, S, q.device) for _ in range(2))
    late, out = torch.empty_like(q), torch.empty_like(q)
    call = ((lambda ws, out: pkv.paged_decode_attn_q4(c.d, q, *c.q4, *c.rows, S, ws, out)) if bits == 4 else
            (lambda ws, out: pkv.paged_decode_attn_window(c.d, q, c.k16, c.v16, *c.rows, 0, 0, S, ws, out)))
    for limit in (0, 200, 1000, 3000, 10000, 0):
        pkv.workspace_init(ws)
        try:
            pkv.testing_set_handoff_wait_ns(limit)
            call(ws, late)
        finally:
            pkv.testing_set_handoff_wait_ns(pkv.DEFAULT_HANDOFF_WAIT_NS)
        out.fill_(float("nan"))
        call(other, out)
        torch.cuda.synchronize()
        status = pkv.status_word(ws)
        assert status in (0, pkv.FLAG_TIMEOUT)
        assert limit > 0 or status == pkv.FLAG_TIMEOUT
        if status == 0:
            assert torch.equal(late, first)
        assert pkv.status_word(other) == 0 and torch.equal(out, first)
