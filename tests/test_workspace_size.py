"""The workspace is no larger than the bf16 decode's regions: shapes that the
no-allocation call took before there was an 8-bit cache still fit its array."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import build as pkv_build
from paged_kv_gqa_16_gb300 import pkv

# (Hq, Hkv, D, B, num_splits): at the array's last bytes
LARGEST = [(32, 8, 64, 159, 12), (16, 2, 128, 269, 7)]


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def _round(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("Hq,Hkv,D,B,S", LARGEST + [(32, 8, 128, 1, 152), (5, 5, 64, 1, 1), (1, 1, 64, 1, 1),
                                                    (48, 3, 128, 65535, 1), (16, 1, 64, 700, 33)])
def test_size_is_the_sum_of_the_bf16_regions(Hq, Hkv, D, B, S):
    d = pkv.dims(B, Hq, Hkv, D, 16, 1 << 16, 1 << 16, 400)
    hpc = next(h for h in (8, 4, 2, 1) if Hkv % h == 0)
    rows = B * (Hkv // hpc)
    plan = 4 * (16 + (rows + 1 + 3) // 4 * 4 + 72 * S) if rows <= 4096 else 0
    fixed = 256 + sum(map(_round, (8 * rows, plan, 2 * B * Hq * D, 4 * (2 * B + 1))))
    parts = max(_round(8 * n) + _round(4 * n * D) for n in (B * Hq * S, (S + rows) * hpc * (Hq // Hkv)))
    assert pkv.workspace_bytes(d, S) == fixed + parts


@pytest.mark.parametrize("Hq,Hkv,D,B,S", LARGEST)
def test_largest_shapes_fit_the_array(Hq, Hkv, D, B, S):
    d = pkv.dims(B, Hq, Hkv, D, 16, 1 << 16, 1 << 16, 400)
    assert pkv.workspace_bytes(d, S) <= pkv.NOALLOC_SCRATCH_BYTES


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,B,S", LARGEST)
def test_no_allocation_call_on_the_largest_shapes(Hq, Hkv, D, B, S):
    g = torch.Generator("cuda").manual_seed(B)
    pages = 3 * B
    d = pkv.dims(B, Hq, Hkv, D, 16, pages, pages, 48)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = randn(B, Hq, D), randn(pages, 16, Hkv, D), randn(pages, 16, Hkv, D)
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    ptr = torch.arange(0, pages + 1, 3, dtype=torch.int32, device="cuda")
    lens = torch.randint(0, 49, (B,), generator=g, device="cuda").to(torch.int32)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got, want = (torch.full((B, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.paged_decode_attn_noalloc(d, q, k, v, ids, ptr, lens, S, got, status=status)
    pkv.paged_decode_attn(d, q, k, v, ids, ptr, lens, S, pkv.alloc_workspace(d, S, "cuda"), want)
    assert int(status.item()) == 0 and torch.equal(got, want)


@pytest.mark.gpu
def test_a_bf16_step_leaves_the_8_bit_plan():
    """A planned call on the 8-bit cache after the bf16 calls that write no plan."""
    from q8_cases import Cache, rope_table
    c = Cache([3000, 0, 33, 64, 1, 7000], 8, 2, 64, 16, seed=3, max_seq_len=1 << 14).fill()
    c.k16.normal_()
    c.v16.normal_()
    S = pkv.plan(c.d)[0]
    q, k, v = (c.randn(6, H, 64).to(torch.bfloat16).cuda() for H in (8, 2, 2))
    want, _ = c.decode(q, S)
    ws, out, other = pkv.alloc_workspace(c.d, S, "cuda"), torch.empty_like(want), torch.empty_like(want)
    table = rope_table(7000, 64)
    for make in (lambda: pkv.paged_decode_plan_q8(c.d, *c.rows, S, ws),
                 lambda: pkv.paged_decode_attn_q8(c.d, q, *c.q8, *c.rows, S, ws, out)):
        make()
        pkv.paged_decode_attn_planned(c.d, q, c.k16, c.v16, *c.rows, S, ws, other)
        pkv.paged_decode_step_planned(c.d, q, k, v, c.k16, c.v16, *c.rows, table, 7000, S, ws, other)
        pkv.paged_decode_partials(c.d, q, c.k16, c.v16, *c.rows, S, ws)
        for _ in range(2):
            out.fill_(float("nan"))
            pkv.paged_decode_attn_q8_planned(c.d, q, *c.q8, *c.rows, S, ws, out)
            assert torch.equal(out, want)
    assert pkv.status_word(ws) == 0
