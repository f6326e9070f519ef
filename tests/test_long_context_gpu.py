"""GPU tests of the 4-bit cache and of windows as a serving loop uses them: a prompt
written, read back and attended over, then captured steps that advance the tables,
write a token and attend, with the pages behind the window given away."""

import pytest
import torch

import q4_cases
from paged_kv_gqa_16_gb300 import pkv
from q4_cases import BF16_EPS, F16_EPS, attention, quantise, seen, values
from q8_cases import DEV, EPS, norm_rotate, rope_table

pytestmark = pytest.mark.gpu


class Rows:
    """B rows with room to grow, their tables and free pages on the device."""

    def __init__(self, lens, Hq, Hkv, D, ps, room, seed):
        self.g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.lens, self.Hq, self.Hkv, self.D, self.ps = list(lens), Hq, Hkv, D, ps
        cap = -(-(max(lens) + room) // ps)
        used = [-(-L // ps) for L in lens]
        n_pool = B * cap + 4
        pages = torch.randperm(n_pool, generator=self.g).to(torch.int32)
        table = torch.full((B, cap), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(used):
            table[b, :n] = pages[at:at + n]
            at += n
        self.cap, self.n_pool = cap, n_pool
        self.indices = table.flatten().to(DEV)
        self.indptr = (torch.arange(B + 1) * cap).to(torch.int32).to(DEV)
        self.seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.free = pages[at:].to(DEV)
        self.head = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.d = pkv.dims(B, Hq, Hkv, D, ps, n_pool, B * cap, max(lens) + room)
        self.S = pkv.plan(self.d)[0]
        self.ws = pkv.alloc_workspace(self.d, self.S, DEV)
        self.rope = rope_table(max(lens) + room, D)
        self.w = (1 + 0.2 * torch.randn(D, generator=self.g)).to(torch.bfloat16).to(DEV)

    @property
    def rows(self):
        return self.indices, self.indptr, self.seq

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g).to(torch.bfloat16)

    def key(self, k, first):
        """Keys [n, Hkv, D] as the writes form them, in 64 bits."""
        return norm_rotate(k, self.w.cpu(), self.rope.cpu()[first:first + len(k)])[0]

    def new(self, q, k, v, q_out):
        return pkv.tokens(q, k, v, q_out, q_norm=self.w, k_norm=self.w, norm_eps=EPS, rope_cos_sin=self.rope,
                          rope_max_pos=self.rope.shape[0])


@pytest.mark.parametrize("D,ps", [(128, 16), (64, 24)])
def test_a_prompt_and_captured_steps_on_a_4_bit_cache(D, ps):
    Hq, Hkv, window, sinks, steps = 8, 2, 40, 4, 20
    lens = [70, 5, 133]
    r = Rows(lens, Hq, Hkv, D, ps, steps + 2, seed=1)
    heads = (r.n_pool, ps, Hkv)
    cache = [torch.full((*heads, D // 2), 0x77, dtype=torch.uint8, device=DEV) for _ in range(2)]
    cache += [torch.full((*heads, D // 32), 255, dtype=torch.uint8, device=DEV) for _ in range(2)]
    # the prompts: written, read back, attended over through the window
    ends = torch.tensor([0] + lens).cumsum(0)
    T = int(ends[-1])
    q, k, v = r.randn(T, Hq, D), r.randn(T, Hkv, D), r.randn(T, Hkv, D)
    q_out = torch.empty_like(q, device=DEV)
    qo = ends.to(torch.int32).to(DEV)
    pkv.paged_kv_extend_q4(r.d, r.new(q.to(DEV), k.to(DEV), v.to(DEV), q_out), qo, *cache, *r.rows, status=r.status)
    pools = [torch.zeros(len(lens) * r.cap, ps, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pkv.paged_kv_read_q4(r.d, *cache, *r.rows, *pools, status=r.status)
    own = pkv.dims(3, Hq, Hkv, D, ps, len(lens) * r.cap, len(lens) * r.cap, r.d.max_seq_len)
    order = torch.arange(len(lens) * r.cap, dtype=torch.int32, device=DEV)
    out = torch.full_like(q_out, float("nan"))
    pkv.paged_prefill_attn_window(own, q_out, qo, *pools, order, r.indptr, r.seq, window, sinks, out, status=r.status,
                                  max_q_len=max(lens))
    assert int(r.status) == 0
    held = []
    for b, L in enumerate(lens):
        a, e = int(ends[b]), int(ends[b + 1])
        held.append([values(*quantise(x)) for x in (r.key(k[a:e], 0), v[a:e].double())])
        for i in range(L):
            at = seen(i + 1, window, sinks)
            want, bound = attention(q_out[a + i].cpu(), held[b][0][at], held[b][1][at], D ** -0.5, 2 * BF16_EPS)
            assert bool(((out[a + i].cpu().double() - want).abs() <= bound).all()), (b, i)
    # steps: one graph
    q1, k1, v1 = (torch.zeros(3, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    q2, wide, near = (torch.empty_like(q1) for _ in range(3))
    graph = torch.cuda.CUDAGraph()
    new = r.new(q1, k1, v1, q2)
    with torch.cuda.graph(graph):
        pkv.paged_kv_advance(r.d, r.seq, r.indptr, r.indices, r.free, r.head, status=r.status)
        pkv.paged_kv_append_q4(r.d, new, *cache, *r.rows, status=r.status)
        pkv.paged_decode_attn_q4(r.d, q2, *cache, *r.rows, r.S, r.ws, wide)
        pkv.paged_decode_attn_q4(r.d, q2, *cache, *r.rows, r.S, r.ws, near, window=window, sinks=sinks)
    for step in range(steps):
        for t in (q1, k1, v1):
            t.copy_(r.randn(*t.shape))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(3):
            L = lens[b] + step + 1
            held[b] = [torch.cat([x, values(*quantise(n))]) for x, n in
                       zip(held[b], (r.key(k1[b:b + 1].cpu(), L - 1), v1[b:b + 1].cpu().double()))]
            for got, at in ((wide, seen(L)), (near, seen(L, window, sinks))):
                want, bound = attention(q2[b].cpu(), held[b][0][at], held[b][1][at], D ** -0.5, F16_EPS)
                # (codes of zero: a step of f16 of the row's largest weight, as q4_cases says)
                bound = bound + 2.0 ** -32 * 6 * len(at) * 2.0
                assert bool(((got[b].cpu().double() - want).abs() <= bound).all()), (step, b)
    assert int(r.status) == 0 and pkv.status_word(r.ws) == 0
    assert r.seq.tolist() == [L + steps for L in lens]


def test_steps_through_a_window_whose_old_pages_are_given_away():
    """bf16 pools: before each step the pages that the window has left are poisoned and
    their entries replaced by ids outside the pool."""
    Hq, Hkv, D, ps, window, sinks, steps = 16, 4, 128, 16, 50, 4, 40
    lens = [90, 64, 200]
    r = Rows(lens, Hq, Hkv, D, ps, steps + 2, seed=2)
    pools = [torch.full((r.n_pool, ps, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    T = sum(lens)
    ends = torch.tensor([0] + lens).cumsum(0)
    k, v = r.randn(T, Hkv, D), r.randn(T, Hkv, D)
    pkv.paged_kv_extend_norm(r.d, r.new(None, k.to(DEV), v.to(DEV), None), ends.to(torch.int32).to(DEV), *pools, *r.rows,
                             status=r.status)
    table = r.indices.view(3, r.cap)
    held = []
    for b, L in enumerate(lens):
        t = torch.arange(L)
        held.append([x.cpu()[table[b].cpu().long()[t // ps], t % ps] for x in pools])
    q1, k1, v1 = (torch.zeros(3, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    q2, out = torch.empty_like(q1), torch.empty_like(q1)
    for step in range(steps):
        for t in (q1, k1, v1):
            t.copy_(r.randn(*t.shape))
        pkv.paged_kv_advance(r.d, r.seq, r.indptr, r.indices, r.free, r.head, status=r.status)
        pkv.paged_kv_append_norm(r.d, r.new(q1, k1, v1, q2), *pools, *r.rows, status=r.status)
        for b in range(3):
            L = lens[b] + step + 1
            page, slot = int(table[b, (L - 1) // ps]), (L - 1) % ps
            held[b] = [torch.cat([x, p[page, slot].cpu()[None]]) for x, p in zip(held[b], pools)]
            for i in range(-(-sinks // ps), (L - window) // ps):
                if int(table[b, i]) >= 0:
                    for p in pools:
                        p[int(table[b, i])] = float("nan")
                    table[b, i] = -1 - i
        pkv.paged_decode_attn_window(r.d, q2, *pools, *r.rows, window, sinks, r.S, r.ws, out)
        assert pkv.status_word(r.ws) == 0
        for b in range(3):
            at = seen(lens[b] + step + 1, window, sinks)
            want, bound = attention(q2[b].cpu(), held[b][0][at].double(), held[b][1][at].double(), D ** -0.5, BF16_EPS)
            assert bool(((out[b].cpu().double() - want).abs() <= bound).all()), (step, b)
    assert int(r.status) == 0
    assert int((table < 0).sum()) > 10


def test_two_graphs_with_workspaces_of_their_own():
    """Two captured decodes replayed at once on two streams."""
    cs, outs, graphs, want = [], [], [], []
    for i in range(2):
        c = q4_cases.fill16(q4_cases.Cache([3000, 200 + i], 16, 4, 128, 16, seed=30 + i, max_seq_len=9000)).fill()
        g = torch.Generator().manual_seed(i)
        q = torch.randn(2, 16, 128, generator=g).to(torch.bfloat16).to(DEV)
        S = pkv.plan(c.d)[0]
        ws = [pkv.alloc_workspace(c.d, S, DEV) for _ in range(2)]
        out = [torch.empty_like(q) for _ in range(2)]

        def call():
            pkv.paged_decode_attn_q4(c.d, q, *c.q4, *c.rows, S, ws[0], out[0])
            pkv.paged_decode_attn_window(c.d, q, c.k16, c.v16, *c.rows, 1500, 4, S, ws[1], out[1])

        call()
        torch.cuda.synchronize()
        want.append([o.clone() for o in out])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        cs.append((c, q, ws))
        outs.append(out)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for out in outs:
            for o in out:
                o.fill_(float("nan"))
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))
