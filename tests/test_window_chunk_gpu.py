"""GPU tests of a chunk of a prompt attended through a window over a 4-bit or an 8-bit cache whose
old pages have been given away: written, the seen part read back, the windowed prefill over it."""

import pytest
import torch

import q4_cases
import q8_cases
from paged_kv_gqa_16_gb300 import pkv
from q4_cases import BF16_EPS, attention, bf16_of, seen
from q8_cases import DEV

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D,ps", [(128, 16), (64, 24), (64, 1)])
@pytest.mark.parametrize("window,sinks", [(100, 4), (33, 0), (64, 30)])
def test_a_chunk_behind_given_away_pages(window, sinks, D, ps, bits):
    Hq, Hkv = 8, 2
    lens, chunks = [700, 300, 0, 64, 1], [129, 40, 0, 64, 1]
    B = len(lens)
    if bits == 4:
        c = q4_cases.Cache(lens, Hq, Hkv, D, ps, seed=1).fill()
        cache, extend, read = c.q4, pkv.paged_kv_extend_q4, pkv.paged_kv_read_q4
    else:
        c = q8_cases.Cache(lens, Hq, Hkv, D, ps, seed=1).fill()
        cache, extend, read = c.q8, pkv.paged_kv_extend_q8, pkv.paged_kv_read_q8
    L, n = torch.tensor(lens), torch.tensor(chunks)
    ends = torch.tensor([0] + chunks).cumsum(0)
    # the first page with a token that the chunk's first query sees through its window
    skip = ((L - n - window + 1).clamp(min=0) // ps)
    table = c.table.clone()
    gone = 0
    for b in range(B):
        for i in range(-(-sinks // ps), int(skip[b])):
            table[c.starts[b] + i] = (-1, c.n_pool, 1 << 30)[i % 3]
            gone += 1
    assert gone > 3
    indices, indptr, seq = table.to(DEV), _i32(c.starts), _i32(lens)
    T = int(ends[-1])
    q, k, v = (c.randn(T, h, D).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
    status = _i32([0])
    extend(c.d, pkv.tokens(None, k, v), _i32(ends), *cache, indices, indptr, seq, status=status)
    # the read-back of the pages with a seen token: rows that begin at their window's first page, then
    # the sinks' pages (whole ones: the prefill takes whole pages, and one's NaN may reach its output)
    pools = [torch.full((c.n_ref, ps, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    begin = torch.tensor(c.starts)
    begin[:B] += skip
    read(c.d, *cache, indices, _i32(begin), _i32(L - skip * ps), *pools, status=status)
    if sinks:
        read(c.d, *cache, indices, indptr, _i32(L.clamp(max=-(-sinks // ps) * ps)), *pools, status=status)
    own = pkv.dims(B, Hq, Hkv, D, ps, c.n_ref, c.n_ref, c.d.max_seq_len)
    order = torch.arange(c.n_ref, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, float("nan"))
    pkv.paged_prefill_attn_window(own, q, _i32(ends), *pools, order, indptr, seq, window, sinks, out, status=status,
                                  max_q_len=max(chunks))
    assert int(status) == 0
    for b in range(B):
        if chunks[b] == 0:
            continue
        held = c.held(b)
        flat = [x.cpu().flatten(0, 1)[c.starts[b] * ps:c.starts[b] * ps + lens[b]] for x in pools]
        first, head = int(skip[b]) * ps, min(-(-sinks // ps) * ps, lens[b])
        for x, y in zip(flat, held):
            assert torch.equal(x[first:], bf16_of(y)[first:]) and torch.equal(x[:head], bf16_of(y)[:head])
            assert bool(x[head:first].isnan().all())
        for i in range(chunks[b]):
            at = seen(lens[b] - chunks[b] + i + 1, window, sinks)
            want, bound = attention(q[int(ends[b]) + i].cpu(), held[0][at], held[1][at], c.scale, 2 * BF16_EPS)
            assert bool(((out[int(ends[b]) + i].cpu().double() - want).abs() <= bound).all()), (b, i)
