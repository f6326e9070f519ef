"""GPU tests of paged_prefill_attn_window at page sizes whose pages are found in other ways: 1 (a
shift by nothing, where the product in place of the division has no meaning) and 17 (key by key)."""

import pytest

import test_window_prefill_gpu as windows

pytestmark = windows.pytestmark


@pytest.mark.parametrize("shape", [(8, 1, 64, 1), (6, 2, 128, 1), (8, 2, 64, 17), (16, 4, 128, 17)])
@pytest.mark.parametrize("rows", [0, 1])
@pytest.mark.parametrize("split", [False, True])
def test_against_64_bits(shape, rows, split):
    windows.test_against_64_bits(shape, rows, split)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [1, 17])
def test_page_sizes(ps, D):
    windows.test_page_sizes(ps, D)
