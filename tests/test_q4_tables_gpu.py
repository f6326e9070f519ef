"""GPU tests of the 4-bit writes with tables that are no rotations: a pair's two factors of any
size, sums that cancel, values on a border. Codes are the exact value's."""

import pytest
import torch

import q4_cases
from paged_kv_gqa_16_gb300 import pkv
from q4_cases import quantise
from q8_cases import DEV, EPS, norm_rotate

pytestmark = pytest.mark.gpu


def _table(kind, n, D, g):
    if kind == "any":
        size = torch.exp2(torch.randint(-9, 10, (n, D // 2, 2), generator=g).float())
        return torch.randn(n, D // 2, 2, generator=g) * size
    if kind == "equal":                                 # a c - b s cancels where a and b are near
        return (torch.randn(n, D // 2, 1, generator=g)).expand(n, D // 2, 2).contiguous()
    return torch.randint(-2, 3, (n, D // 2, 2), generator=g).float()      # small whole numbers: ties


@pytest.mark.parametrize("kind", ["any", "equal", "whole"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_codes_with_any_table(D, norm, kind):
    L, Hkv = 900, 4
    c = q4_cases.Cache([L], 8, Hkv, D, 16, seed=1)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(L, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    if kind == "equal":                                 # pairs a bf16 step or a few apart, or equal
        step = 1 + torch.randint(0, 4, (L, Hkv, D // 2), generator=g) * 2.0 ** -7
        k[..., 1::2] = (k[..., 0::2].float() * step).to(torch.bfloat16)
    if kind == "whole":
        k = torch.randint(-8, 9, (L, Hkv, D), generator=g).to(torch.bfloat16) / 4
    table = _table(kind, L, D, g).to(DEV)
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) if norm else None
    ends = torch.tensor([0, L], dtype=torch.int32, device=DEV)
    t = pkv.tokens(None, k.to(DEV), v.to(DEV), k_norm=w, norm_eps=EPS, rope_cos_sin=table, rope_max_pos=L)
    pkv.paged_kv_extend_q4(c.d, t, ends, *c.q4, *c.rows, status=c.status)
    assert int(c.status) == 0
    want, _ = norm_rotate(k, None if w is None else w.cpu(), table.cpu())
    kc, ks, _, _ = c.stored(0, 0, L)
    code, scale = quantise(want)
    assert torch.equal(ks, scale)
    assert torch.equal(kc & 7, code & 7)
    assert torch.equal((kc >> 3)[code & 7 != 0], (code >> 3)[code & 7 != 0])
