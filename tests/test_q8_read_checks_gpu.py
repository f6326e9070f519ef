"""paged_kv_read_q8's checks of the rows and scales that it is given."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import pkv
from q8_cases import DEV, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,want", [([0, 0], 0), ([3, 0], pkv.FLAG_BAD_PAGE), ([0, -1], pkv.FLAG_BAD_LEN),
                                       ([21, 0], pkv.FLAG_BAD_LEN),
                                       ([-5, 2], pkv.FLAG_BAD_LEN | pkv.FLAG_BAD_PAGE)])
def test_rows_are_checked_where_the_table_is_empty(lens, want):
    d = pkv.dims(2, 2, 2, 64, 4, 3, 0, 20)
    pools = [torch.zeros(3, 4, 2, 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
    pools += [torch.full((3, 4, 2), 127, dtype=torch.uint8, device=DEV) for _ in range(2)]
    ptr = torch.zeros(3, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    k, v = (torch.full((1, 4, 2, 64), -1.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pkv.paged_kv_read_q8(d, *pools, None, ptr, torch.tensor(lens, dtype=torch.int32, device=DEV), k, v,
                         status=status)
    assert int(status.item()) == want
    assert bool((k == -1).all()) and bool((v == -1).all())


def test_a_table_that_decreases_is_flagged_by_idle_rows_too():
    """Offsets that decrease hide other rows' entries from the search for a slot's row,
    so the row that makes them decrease is reported even if it has no tokens."""
    c = Cache([12, 0, 0, 9], 2, 2, 64, 4, seed=1).fill()
    k, v = (torch.zeros(c.n_ref, 4, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    indptr = c.kv_indptr.clone()

    def read():
        c.status.zero_()
        pkv.paged_kv_read_q8(c.d, *c.q8, c.kv_indices, indptr, c.seq_lens, k, v, status=c.status)
        return int(c.status.item())

    assert read() == 0
    for bad in (1000, -3):
        indptr[2] = bad                                            # ends row 1, starts row 2: both idle
        assert read() == pkv.FLAG_BAD_PAGE, bad
    indptr[2] = c.kv_indptr[2]
    indptr[4] = c.n_ref + 1                                        # the last row's end is past the table
    c.seq_lens[3] = 0
    assert read() == pkv.FLAG_BAD_PAGE


@pytest.mark.parametrize("D", [64, 128])
def test_scales_at_the_ends_of_their_type(D):
    """e8m0 byte 0 is 2^-127 and 255 is NaN; where a bf16 does not hold the product it is
    the nearest one."""
    sizes = [0, 1, 2, 5, 10, 126, 127, 128, 240, 246, 253, 254, 255]
    c = Cache([len(sizes)], 1, 1, D, 16, seed=5).fill()
    at = c.places(0, 0, len(sizes))
    for scale in (c.ks, c.vs):
        scale[at[0], at[1], 0] = torch.tensor(sizes, dtype=torch.uint8, device=DEV)
    k, v = (torch.zeros(c.n_ref, 16, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pkv.paged_kv_read_q8(c.d, *c.q8, *c.rows, k, v, status=c.status)
    assert int(c.status.item()) == 0
    for got, codes in ((k, c.kc), (v, c.vc)):
        got = got.cpu().view(-1, D)[:len(sizes)].double()
        want = codes.cpu()[at][:, 0].view(torch.float8_e4m3fn).double()
        want = want * torch.exp2(torch.tensor(sizes).double() - 127)[:, None]
        # (fp32 holds every product under its largest, so that is the one rounding to bf16)
        want[sizes.index(255)] = float("nan")
        want = want.float().to(torch.bfloat16).double()
        assert torch.equal(got.nan_to_num(nan=1e300, posinf=1e301, neginf=-1e301),
                           want.nan_to_num(nan=1e300, posinf=1e301, neginf=-1e301))
