"""The 8-bit decode's split path (partition, plan, join of the pieces): every case
here has a max_seq_len that keeps its rows off the whole-row path, and says so."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import pkv
from q8_cases import DEV, Cache

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
