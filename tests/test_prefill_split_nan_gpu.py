"""GPU tests of the prefill's key split with keys and values that are not numbers."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import pkv
from q4_cases import Cache, fill16
from q8_cases import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3500, 4)])
@pytest.mark.parametrize("what", ["key", "value", "infinite key"])
@pytest.mark.parametrize("at", [0, 1700, 4090])
def test_a_part_that_is_not_a_number_is_kept(D, window, sinks, what, at):
    """A NaN key, or an infinite one that scores so, reaches every query that sees it, a NaN value
    their column, whichever part of the keys it is in: as without a split."""
    L, chunk, Hq, Hkv = 4096, 60, 8, 2
    c = fill16(Cache([L], Hq, Hkv, D, 16, seed=1))
    place = tuple(int(x) for x in c.places(0, at, at + 1))
    if what == "value":
        c.v16[place][1, 5] = float("nan")
    elif what == "key":
        c.k16[place][1, 5] = float("nan")
    else:
        c.k16[place][1, 5] = float("inf")
    q = c.randn(chunk, Hq, D).to(torch.bfloat16).to(DEV)
    q[..., 5] = q[..., 5].abs() + 0.5
    ends = torch.tensor([0, chunk], dtype=torch.int32, device=DEV)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.empty(pkv.prefill_workspace_bytes(D, sms), dtype=torch.uint8, device=DEV)
    assert pkv.prefill_plan(c.d, chunk, sms, ws.numel())["split"] > 1
    got = []
    for w in (ws, None):
        out, status = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device=DEV)
        pkv.paged_prefill_attn_window(c.d, q, ends, c.k16, c.v16, *c.rows, window, sinks, out, status=status,
                                      workspace=w)
        assert int(status) == 0
        got.append(out.isnan().cpu().view(chunk, Hkv, -1, D))
    # position p = L - chunk + i sees `at`
    p = torch.arange(L - chunk, L)
    sees = (at <= p) & ((at > p - window) | (at < sinks) | (window == 0))
    want = torch.zeros(chunk, Hkv, Hq // Hkv, D, dtype=torch.bool)
    if what == "value":
        want[sees, 1, :, 5] = True
    else:
        want[sees, 1] = True
    for x in got:
        # (who does not see it may get it from the tile's others: only those that do are compared,
        # and that the other kv head is untouched)
        assert bool(x[want].all()) and not bool(x[:, 0].any())
        if what == "value":
            assert not bool(x[:, 1, :, :5].any()) and not bool(x[:, 1, :, 6:].any())
