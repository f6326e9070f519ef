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
