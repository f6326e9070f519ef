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
