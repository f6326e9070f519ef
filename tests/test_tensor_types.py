"""The types of the tensors that the normalising writes and the 8-bit cache's calls
take: others are refused before anything is launched, so no GPU is needed."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import build as pkv_build
from paged_kv_gqa_16_gb300 import pkv

BF16, F16, I16 = torch.bfloat16, torch.float16, torch.int16


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


@pytest.mark.parametrize("other", [F16, I16, torch.float32, torch.uint8])
@pytest.mark.parametrize("which", ["q", "k", "v", "q_out", "q_norm", "k_norm"])
def test_tokens_are_bf16(which, other):
    a = dict(q=torch.zeros(3, 4, 64, dtype=BF16), k=torch.zeros(3, 2, 64, dtype=BF16),
             v=torch.zeros(3, 2, 64, dtype=BF16), q_out=torch.zeros(3, 4, 64, dtype=BF16),
             q_norm=torch.ones(64, dtype=BF16), k_norm=torch.ones(64, dtype=BF16))
    assert pkv.tokens(**a).shape == (3, 4, 2, 64)
    a[which] = a[which].to(other)
    with pytest.raises(ValueError):
        pkv.tokens(**a)


@pytest.mark.parametrize("other", [F16, BF16, I16, torch.float64, torch.int32])
def test_the_rotation_table_is_fp32(other):
    """A table of the same elements in two bytes each would be read past its end."""
    q, k = torch.zeros(3, 4, 64, dtype=BF16), torch.zeros(3, 2, 64, dtype=BF16)
    rope = torch.zeros(5, 32, 2)
    assert pkv.tokens(q, k, k, rope_cos_sin=rope, rope_max_pos=5).rope_cos_sin == rope.data_ptr()
    with pytest.raises(ValueError):
        pkv.tokens(q, k, k, rope_cos_sin=rope.to(other), rope_max_pos=5)
