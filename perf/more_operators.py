"""What is measured of the 4-bit key-value cache and of attention with a sliding window.

Around a paged cache (pools of [pages, page_size, Hkv, D], a page table per row,
D 64 or 128, grouped-query heads). The 4-bit cache holds e2m1 codes, two to a
byte, and one power-of-two scale (e8m0) for every 32 elements of a head vector.

* ``q4_extend``: ragged chunks of new tokens quantised into the cache (norms
  and rotation on the way), and the rows read back in bf16 for the prefill
  attention over them.
* ``q4_read``: the rows of such a cache read back alone.
* ``q4_step``: a layer of a decode step: each row's new token into the cache, then
  the attention of its query over the row.
* ``q4_decode``: the attention alone, over all tokens or through a window.
* ``window_decode``: one query a row that sees the last ``window`` tokens and the
  first ``sinks`` of a bf16 cache.
* ``window_prefill``: chunks of queries, each of which sees the last ``window``
  tokens up to its own and the first ``sinks``.

``run`` computes them in plain torch operations, or with ``own`` through the
library's calls.
"""

import itertools
import math
import random
import statistics

import torch

own = False

EPS = 1e-6
LOW, HIGH = -40, 40        # range of a scale's exponent
GROUP = 32                 # elements of a scale


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # prompts of odd lengths behind a cached prefix, head size 64, odd pages, keys normalised
        dict(name="q4_extend_odd_d64", op="q4_extend", B=32, Hq=32, Hkv=8, D=64, page=24, lo=301,
             hi=1021, shape="even", idle=0, q_lo=129, q_hi=509, norm=True, rope=True, packed=False),
        # sixteen extends of 256 tokens and more on longer contexts
        dict(name="q4_extend_b16", op="q4_extend", B=16, Hq=32, Hkv=8, D=128, page=16, lo=2048, hi=2048,
             shape="even", idle=0, q_lo=256, q_hi=2048, norm=False, rope=True, packed=True),
        # two short rows read back, the smallest call, and a ragged batch before a prefill over it
        dict(name="q4_read_tiny", op="q4_read", B=2, Hq=4, Hkv=2, D=64, page=16, lo=37, hi=100,
             shape="even", idle=0),
        dict(name="q4_read_ragged_b32", op="q4_read", B=32, Hq=32, Hkv=8, D=128, page=16, lo=512,
             hi=4096, shape="even", idle=0),
        # a layer of a decode step of a 1B-class model: latency
        dict(name="q4_step_1b_d64", op="q4_step", B=8, Hq=32, Hkv=8, D=64, page=16, lo=513, hi=1025,
             shape="even", idle=0, norm=True, rope=True, packed=False),
        # the same of a serving batch padded to a power of two, q, k, v in one projection's output
        dict(name="q4_step_serving_b128", op="q4_step", B=128, Hq=64, Hkv=8, D=128, page=16, lo=16,
             hi=8192, shape="lognormal", idle=32, norm=True, rope=True, packed=True),
        # one row of 32,768 tokens
        dict(name="q4_decode_long_32k", op="q4_decode", B=1, Hq=32, Hkv=8, D=128, page=16, lo=32768,
             hi=32768, shape="even", idle=0, window=0, sinks=0),
        # a ragged batch of which every layer but a few sees a window
        dict(name="q4_decode_window_b32", op="q4_decode", B=32, Hq=32, Hkv=8, D=128, page=16, lo=512,
             hi=4096, shape="even", idle=0, window=1024, sinks=4),
        # two short rows through a short window: the smallest call
        dict(name="window_decode_tiny", op="window_decode", B=2, Hq=4, Hkv=2, D=64, page=16, lo=37,
             hi=100, shape="even", idle=0, window=32, sinks=4),
        # a serving batch whose long rows keep their first tokens
        dict(name="window_decode_serving_b128", op="window_decode", B=128, Hq=64, Hkv=8, D=128, page=16,
             lo=16, hi=8192, shape="lognormal", idle=32, window=1024, sinks=4),
        # odd chunks behind cached contexts, head size 64, odd pages, a window shorter than the chunk
        dict(name="window_prefill_odd_d64", op="window_prefill", B=16, Hq=32, Hkv=8, D=64, page=24, lo=301,
             hi=2021, shape="even", idle=0, q_lo=129, q_hi=509, window=250, sinks=4),
        # four whole prompts of 4,096 tokens
        dict(name="window_prefill_4x4096", op="window_prefill", B=4, Hq=32, Hkv=8, D=128, page=16, lo=4096,
             hi=4096, shape="even", idle=0, q_lo=4096, q_hi=4096, window=1024, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["q4_extend", "q4_read", "q4_step", "q4_decode", "q4_decode", "window_decode",
                     "window_decode", "window_prefill"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    rep = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 16])
    B = _log_int(rng, 1, 16 if op == "window_prefill" else 128)
    idle = rng.choice([0, 0, B // 4])
    # no more cached values than the largest listed rows of the kind have
    budget = {"q4_read": 70e6, "q4_extend": 32e6, "window_prefill": 16e6}.get(op, 150e6)
    most = max(1, int(budget / (B * Hkv * D)))
    hi = _log_int(rng, 1, min(4096 if op == "window_prefill" else 32768, most))
    lo = _log_int(rng, 1, hi)
    case = dict(op=op, B=B, Hq=Hkv * rep, Hkv=Hkv, D=D, page=rng.choice([1, 8, 16, 16, 17, 32, 64, 128]),
                lo=lo, hi=hi, shape="lognormal" if hi > 16 * lo else "even", idle=idle)
    if op in ("q4_extend", "window_prefill"):
        most_q = max(1, int((48e6 if op == "q4_extend" else 32e6) / (B * (case["Hq"] + 2 * Hkv) * D)))
        # (the plain scores of a prefill, kept under 4 x 32 heads x 4,096 x 4,096)
        if op == "window_prefill":
            most_q = max(1, min(most_q, int(2e9 / (B * case["Hq"] * hi))))
        case["q_hi"] = _log_int(rng, 1, min(hi, most_q))
        case["q_lo"] = rng.randint(0, case["q_hi"])
    if op in ("q4_extend", "q4_step"):
        case.update(norm=rng.random() < 0.6, rope=rng.random() < 0.8, packed=rng.random() < 0.5)
    if op.startswith("window") or op == "q4_decode":
        case.update(window=_log_int(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 4, 4, 16, 17, 64, 130]))
        if op == "q4_decode" and rng.random() < 0.6:
            case.update(window=0, sinks=0)
    return case


def _lens(case):
    """The rows' lengths, idle rows last: they follow from the case alone."""
    n = case["B"] - case["idle"]
    lo, hi = case["lo"], case["hi"]
    got = []
    for i in range(n):
        u = (i + 0.5) / n
        if case["shape"] == "lognormal":
            x = math.exp(math.log(math.sqrt(lo * hi) if lo * 64 > hi else hi / 8)
                         + statistics.NormalDist().inv_cdf(u))
        else:
            x = lo + (hi - lo) * (u if n > 1 else 1.0) if n != 2 else (lo, hi)[i]
        got.append(max(lo, min(hi, int(round(x)))))
    return got


def _chunks(case, lens):
    """New tokens of each row of a chunked call (no more than its length)."""
    n = len(lens)
    return [min(L, case["q_lo"] + ((case["q_hi"] - case["q_lo"]) * (n - 1 - i)) // max(1, n - 1)
                if n > 1 else case["q_hi"]) for i, L in enumerate(lens)]


def _seen(case, L):
    """Tokens of a row of L that its last one sees."""
    return min(L, case["window"] + case["sinks"]) if case.get("window") else L


# ------------------------------------------------------------------ the inputs
def _quantise(x):
    """(codes [..., D/2], scales [..., D/32]) of head vectors x [..., D], in 64 bits:
    a group's scale is the smallest power of two that brings its largest value to
    6 or under, its codes the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the
    even code), two to a byte, the first in the low half."""
    x = x.double().unflatten(-1, (-1, GROUP))
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 3 + (m > 0.75).to(e.dtype), torch.full_like(e, LOW)).clamp(LOW, HIGH)
    y = torch.ldexp(x.abs(), -e.unsqueeze(-1)).clamp(max=6.0)
    step = torch.where(y >= 4, 2.0, torch.where(y >= 2, 1.0, 0.5))
    y = torch.round(y / step) * step
    code = torch.where(y <= 2, 2 * y, torch.where(y <= 4, y + 2, y / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(x).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """What codes and scales stand for, [..., D] in 32 bits."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    a = (both & 7).to(torch.float32)
    a = torch.where(a <= 4, a / 2, torch.where(a <= 6, a - 2, 6.0))
    a = torch.where(both > 7, -a, a).unflatten(-1, (-1, GROUP))
    return torch.ldexp(a, (scales.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    order = random.Random(seed)
    B, Hq, Hkv, D, ps, op = (case[k] for k in ("B", "Hq", "Hkv", "D", "page", "op"))
    live = _lens(case)
    rows = list(zip(live, _chunks(case, live) if case.get("q_hi") else live))
    order.shuffle(rows)
    lens = [L for L, _ in rows] + [0] * case["idle"]
    pages = [-(-L // ps) for L in lens]
    n_ref = sum(pages)
    n_pool = n_ref + n_ref // 4 + 1
    indptr = [0] + list(itertools.accumulate(pages))
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(case=case, lens=lens, kept={}, seq_lens=ints(lens), kv_indptr=ints(indptr),
             kv_indices=torch.randperm(n_pool, generator=g, device=dev)[:n_ref].to(torch.int32),
             max_len=max(case["hi"], 1))
    pool = (n_pool, ps, Hkv, D)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    # keys have a few large channels, as projections of trained models do
    loud = torch.exp(0.5 * randn(Hkv, D))
    for name, gain in (("k", loud), ("v", 1.0)):
        x = (randn(*pool) * gain * torch.exp(0.3 * randn(*pool[:3], 1))).to(torch.bfloat16)
        if op.startswith("q4"):
            s[name + "_pool"], s[name + "_scale"] = (torch.cat(t) for t in zip(
                *(_quantise(part) for part in x.split(1 + (1 << 25) // (ps * Hkv * D)))))
        else:
            s[name + "_pool"] = x
        del x
    T = B
    if case.get("q_hi"):
        s["chunks"] = [n for _, n in rows] + [0] * case["idle"]
        ends = list(itertools.accumulate(s["chunks"]))
        s["qo_indptr"] = ints([0] + ends)
        T = ends[-1]
    if op in ("q4_extend", "q4_step"):
        both = randn(T, Hq + 2 * Hkv, D)
        both[:, Hq:Hq + Hkv] *= loud
        both = both.to(torch.bfloat16)
        q, k, v = both[:, :Hq], both[:, Hq:Hq + Hkv], both[:, Hq + Hkv:]
        s["q"], s["k"], s["v"] = (q, k, v) if case["packed"] else (q.contiguous(), k.contiguous(), v.contiguous())
        s["q_out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
        if case["norm"]:
            s["q_norm"] = (1 + 0.2 * randn(D)).to(torch.bfloat16)
            s["k_norm"] = (1 + 0.2 * randn(D)).to(torch.bfloat16)
        if case["rope"]:
            at = torch.arange(s["max_len"], device=dev, dtype=torch.float64)
            turn = 10000.0 ** (-2.0 * torch.arange(D // 2, device=dev, dtype=torch.float64) / D)
            angle = at[:, None] * turn
            s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32).contiguous()
    if op in ("q4_extend", "q4_read"):
        shape = (max(1, n_ref), ps, Hkv, D)
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
        return s
    if op != "q4_step":
        s["q"] = randn(T, Hq, D).to(torch.bfloat16)
    s["out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------- the plain forms
def _of_rows(counts, device):
    """The row of each of the rows' `counts` things laid end to end, and its place in the row."""
    n = torch.tensor(counts, dtype=torch.int64, device=device)
    row = torch.repeat_interleave(torch.arange(len(counts), device=device), n, output_size=sum(counts))
    return row, torch.arange(sum(counts), device=device) - (n.cumsum(0) - n)[row]


def _slots(s, row, pos):
    """Flat pool slot of each (row, position)."""
    ps = s["case"]["page"]
    page = s["kv_indices"].long()[s["kv_indptr"].long()[row] + pos // ps]
    return page * ps + pos % ps


def _chunk_rows(s):
    """The row and the position of every new token."""
    dev = s["seq_lens"].device
    if "qo_indptr" not in s:
        row = torch.arange(s["case"]["B"] - s["case"]["idle"], device=dev)
        return row, s["seq_lens"].long()[row] - 1
    row, at = _of_rows(s["chunks"], dev)
    new = s["qo_indptr"].long()[1:] - s["qo_indptr"].long()[:-1]
    return row, s["seq_lens"].long()[row] - new[row] + at


def _normed_rotated(s, x, weight, pos, kind):
    x = x.to(kind)
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(kind)
    if "rope" in s:
        c, r = s["rope"][pos, :, 0].to(kind).unsqueeze(1), s["rope"][pos, :, 1].to(kind).unsqueeze(1)
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack([a * c - b * r, a * r + b * c], -1).flatten(-2)
    return x


def _plain_write(s):
    row, pos = _chunk_rows(s)
    n = row.numel()
    s["q_out"][:n] = _normed_rotated(s, s["q"][:n], s.get("q_norm"), pos, torch.float32).to(torch.bfloat16)
    Hkv, slot = s["case"]["Hkv"], _slots(s, row, pos)
    # (in 64 bits: a code next to a border goes by the value's last bits)
    for name, x in (("k", _normed_rotated(s, s["k"][:n], s.get("k_norm"), pos, torch.float64)), ("v", s["v"][:n])):
        codes, scales = _quantise(x)
        s[name + "_pool"].view(-1, Hkv, codes.shape[-1])[slot] = codes
        s[name + "_scale"].view(-1, Hkv, scales.shape[-1])[slot] = scales


def _gathered(s, name, slot):
    """Cached head vectors at flat slots, [..., Hkv, D] in 32 bits."""
    x = s[name + "_pool"].flatten(0, 1)[slot]
    if name + "_scale" not in s:
        return x.to(torch.float32)
    return _values(x, s[name + "_scale"].flatten(0, 1)[slot])


def _plain_read(s):
    Hkv, D, ps = s["case"]["Hkv"], s["case"]["D"], s["case"]["page"]
    row, pos = _of_rows(s["lens"], s["seq_lens"].device)
    slot = _slots(s, row, pos)
    to = s["kv_indptr"].long()[row] * ps + pos
    s["k_out"].view(-1, Hkv, D)[to] = _gathered(s, "k", slot).to(torch.bfloat16)
    s["v_out"].view(-1, Hkv, D)[to] = _gathered(s, "v", slot).to(torch.bfloat16)


def _slots_or_none(s, pos, there):
    """Flat slots of positions [B, L] where they are there, slot 0 elsewhere."""
    rows = torch.arange(s["case"]["B"], device=pos.device)[:, None].expand_as(there)
    entry = (s["kv_indptr"].long()[rows] + pos // s["case"]["page"]).clamp(max=s["kv_indices"].numel() - 1)
    return torch.where(there, s["kv_indices"].long()[entry] * s["case"]["page"] + pos % s["case"]["page"], 0)


def _softmax(x, there):
    x = torch.where(there, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_decode(s, q):
    case, dev = s["case"], q.device
    B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
    at = torch.arange(max(_seen(case, L) for L in s["lens"] + [1]), device=dev)
    L = s["seq_lens"].long()[:, None]
    seen = L.clamp(max=case["window"] + case["sinks"]) if case.get("window") else L
    there = at < seen                                                  # [B, seen]
    pos = torch.where(at < case.get("sinks", 0), at, at + L - seen) if case.get("window") else at.expand_as(there)
    slot = _slots_or_none(s, torch.where(there, pos, 0), there)
    k = _gathered(s, "k", slot).permute(0, 2, 3, 1)                    # [B, Hkv, D, seen]
    x = (q.to(torch.float32).view(B, Hkv, Hq // Hkv, D) @ k) * (1.0 / math.sqrt(D))
    del k
    o = _softmax(x, there[:, None, None]) @ _gathered(s, "v", slot).permute(0, 2, 1, 3)
    s["out"].copy_(o.reshape(B, Hq, D))


def _plain_prefill(s):
    case, dev = s["case"], s["q"].device
    B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
    row, pos = _chunk_rows(s)
    _, at = _of_rows(s["chunks"], dev)
    longest = max(s["chunks"] + [1])
    q = torch.zeros(B, longest, Hq, D, device=dev)
    q[row, at] = s["q"].to(torch.float32)
    mine = torch.full((B, longest), -1, device=dev)
    mine[row, at] = pos
    keys = torch.arange(max(s["lens"] + [1]), device=dev)
    there = keys < s["seq_lens"][:, None]
    slot = _slots_or_none(s, keys.expand_as(there), there)
    k = _gathered(s, "k", slot).permute(0, 2, 3, 1)                    # [B, Hkv, D, L]
    q = q.view(B, longest, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)   # [B, Hkv, rep, longest, D]
    mine = mine[:, :, None]
    seen = (keys <= mine) & ((keys > mine - case["window"]) | (keys < case["sinks"]))
    o = _softmax((q @ k[:, :, None]) * (1.0 / math.sqrt(D)), seen[:, None, None])
    o = o @ _gathered(s, "v", slot).permute(0, 2, 1, 3)[:, :, None]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, longest, Hq, D)[row, at])


def _plain(s):
    op = s["case"]["op"]
    if op in ("q4_extend", "q4_step"):
        _plain_write(s)
    if op in ("q4_extend", "q4_read"):
        _plain_read(s)
    elif op == "window_prefill":
        _plain_prefill(s)
    else:
        _plain_decode(s, s["q_out"] if op == "q4_step" else s["q"])


# ------------------------------------------------------------ the library's own
def _own(s):
    from paged_kv_gqa_16_gb300 import pkv
    c, kept, op = s["case"], s["kept"], s["case"]["op"]
    dev = s["seq_lens"].device
    if not kept:
        d = kept["dims"] = pkv.dims(c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], s["k_pool"].shape[0],
                                    s["kv_indices"].numel(), s["max_len"])
        kept["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        if op == "window_prefill":
            sms = torch.cuda.get_device_properties(dev).multi_processor_count
            kept["workspace"] = torch.empty(pkv.prefill_workspace_bytes(c["D"], sms), dtype=torch.uint8, device=dev)
        elif "out" in s:
            kept["splits"] = pkv.plan(d)[0]
            kept["workspace"] = pkv.alloc_workspace(d, kept["splits"], dev)
    d, status = kept["dims"], kept["status"]
    table = (s["kv_indices"], s["kv_indptr"], s["seq_lens"])
    if op == "window_prefill":
        pkv.paged_prefill_attn_window(d, s["q"], s["qo_indptr"], s["k_pool"], s["v_pool"], *table, c["window"],
                                      c["sinks"], s["out"], status=status, max_q_len=max(s["chunks"] + [1]),
                                      workspace=kept["workspace"])
        return
    if op == "window_decode":
        pkv.paged_decode_attn_window(d, s["q"], s["k_pool"], s["v_pool"], *table, c["window"], c["sinks"],
                                     kept["splits"], kept["workspace"], s["out"])
        return
    cache = (s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
    if op in ("q4_extend", "q4_step"):
        rope = s.get("rope")
        t = pkv.tokens(s["q"], s["k"], s["v"], q_out=s["q_out"], q_norm=s.get("q_norm"), k_norm=s.get("k_norm"),
                       norm_eps=EPS, rope_cos_sin=rope, rope_max_pos=0 if rope is None else rope.shape[0])
        if op == "q4_extend":
            pkv.paged_kv_extend_q4(d, t, s["qo_indptr"], *cache, *table, status=status)
        else:
            pkv.paged_kv_append_q4(d, t, *cache, *table, status=status)
    if op in ("q4_extend", "q4_read"):
        pkv.paged_kv_read_q4(d, *cache, *table, s["k_out"], s["v_out"], status=status)
    else:
        pkv.paged_decode_attn_q4(d, s["q_out"] if op == "q4_step" else s["q"], *cache, *table, kept["splits"],
                                 kept["workspace"], s["out"], window=c.get("window", 0), sinks=c.get("sinks", 0))


def run(s):
    if own:
        _own(s)
    else:
        _plain(s)
    return {n: s[m] for n, m in (("q", "q_out"), ("k", "k_out"), ("v", "v_out"), ("out", "out")) if m in s}


def work(case):
    """Each new or cached token's values read and written once, in the types they are held in."""
    lens = _lens(case)
    Hq, Hkv, D, op = case["Hq"], case["Hkv"], case["D"], case["op"]
    token = 2 * Hkv * (D // 2 + D // GROUP) if op.startswith("q4") else 2 * Hkv * D * 2
    tables = 4 * (2 * case["B"] + 1 + sum(-(-L // case["page"]) for L in lens))
    total = sum(_seen(case, L) for L in lens)
    bytes_, flops = tables, 0
    if op in ("q4_extend", "q4_step"):
        T = sum(_chunks(case, lens)) if op == "q4_extend" else len(lens)
        cos_sin = 4 * D * min(T, max(case["hi"], 1)) if case["rope"] else 0
        bytes_ += T * ((2 * Hq + 2 * Hkv) * D * 2 + token) + cos_sin
        flops += T * ((Hq + Hkv) * D * ((3 if case["rope"] else 0) + (4 if case["norm"] else 0)) + 4 * Hkv * D)
    if op in ("q4_extend", "q4_read"):
        # (a chunk's tokens come back from the codes just written)
        bytes_ += total * (token + 2 * Hkv * D * 2)
        flops += total * 2 * Hkv * D
    elif op == "window_prefill":
        pairs = span = 0
        for L, n in zip(lens, _chunks(case, lens)):
            # tokens seen by the queries at L - n .. L - 1: sum over p of min(p + 1, window + sinks)
            W = case["window"] + case["sinks"]
            full = max(0, L - max(L - n, W - 1))
            pairs += full * W + (n - full) * (2 * (L - n) + n - full + 1) // 2
            span += min(L, n - 1 + W) if n else 0
        T = sum(_chunks(case, lens))
        bytes_ += span * token + 2 * T * Hq * D * 2
        flops += pairs * 4 * Hq * D
    else:
        bytes_ += total * token + 2 * case["B"] * Hq * D * 2
        flops += total * 4 * Hq * D
    return {"bytes": bytes_, "flops": flops}


# --------------------------------------------------------------- in 64 bits
def _held(x):
    """x [..., D] in 64 bits as a 4-bit cache holds it: the nearest of the group's
    fifteen values, the one with an even code where two are as near."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    x = x.unflatten(-1, (-1, GROUP))
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 6.0)).clamp(LOW, HIGH))
    size = (x.abs() / scale).clamp(max=6.0).contiguous()
    half = (grid[1:] + grid[:-1]) / 2
    # a border belongs to the lower value where that one's code is even
    up, down = torch.bucketize(size, half, right=True), torch.bucketize(size, half, right=False)
    at = torch.where(down % 2 == 0, down, up)
    return (torch.sign(x) * grid[at] * scale).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    B, Hq, Hkv, D, ps, op = (case[k] for k in ("B", "Hq", "Hkv", "D", "page", "op"))
    lens, starts = s["lens"], s["kv_indptr"].tolist()
    table = s["kv_indices"].long()
    value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=table.device)
    value = torch.cat([value, -value])

    def cached(name, b, first, last):
        """Row b's cached K or V of tokens first .. last - 1, [n, Hkv, D]."""
        t = torch.arange(first, last, device=table.device)
        at = table[starts[b] + torch.div(t, ps, rounding_mode="floor")], torch.remainder(t, ps)
        x = s[name + "_pool"][at]
        if not op.startswith("q4"):
            return x.double()
        x = torch.stack([value[(x % 16).long()], value[torch.div(x, 16, rounding_mode="floor").long()]], -1).flatten(-2)
        scale = torch.exp2(s[name + "_scale"][at].double() - 127.0)
        return x * scale.repeat_interleave(GROUP, -1)

    def new(name, b, n, at, L):
        """Row b's n new heads, normalised and rotated, in 64 bits."""
        x = s[name][at:at + n].double()
        if case["norm"]:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * s[name + "_norm"].double()
        if case["rope"]:
            turn = torch.view_as_complex(s["rope"][L - n:L].double())[:, None]
            x = torch.view_as_real(torch.view_as_complex(x.reshape(n, -1, D // 2, 2).contiguous()) * turn).reshape(n, -1, D)
        return x

    def attend(q, k, v, seen=None):
        """q [n, Hq, D] over k and v [L, Hkv, D]; seen [n, L]."""
        n = q.shape[0]
        x = torch.einsum("ngrd,lgd->grnl", q.view(n, Hkv, Hq // Hkv, D), k) / math.sqrt(D)
        if seen is not None:
            x = x.masked_fill(~seen, -math.inf)
        return torch.einsum("grnl,lgd->ngrd", torch.softmax(x, -1), v).reshape(n, Hq, D)

    chunk = "qo_indptr" in s
    ends = s["qo_indptr"].tolist()[1:] if chunk else list(range(1, B + 1))
    got = {n: s[m].double() for n, m in (("q", "q_out"), ("k", "k_out"), ("v", "v_out"), ("out", "out")) if m in s}
    at = 0
    for b, L in enumerate(lens):
        n = ends[b] - at if chunk or op == "q4_step" else 0
        if L:
            if op == "window_prefill":
                for i in range(0, n, 512):
                    p = torch.arange(L - n + i, min(L - n + i + 512, L), device=table.device)[:, None]
                    # the keys that some of these queries see: the first ones, then a band
                    band = max(min(case["sinks"], L), int(p[0]) - case["window"] + 1)
                    j = torch.cat([torch.arange(min(case["sinks"], L), device=table.device),
                                   torch.arange(band, int(p[-1]) + 1, device=table.device)])
                    seen = (j <= p) & ((j > p - case["window"]) | (j < case["sinks"]))
                    k, v = (torch.cat([cached(m, b, 0, min(case["sinks"], L)), cached(m, b, band, int(p[-1]) + 1)])
                            for m in ("k", "v"))
                    got["out"][at + i:at + i + len(p)] = attend(s["q"][at + i:at + i + len(p)].double(), k, v, seen)
            else:
                seen = _seen(case, L)
                first = min(case.get("sinks", 0), seen)
                row = {m: torch.cat([cached(m, b, 0, first), cached(m, b, L - seen + first, L)]) for m in ("k", "v")}
                if op in ("q4_extend", "q4_step") and n:
                    got["q"][at:at + n] = new("q", b, n, at, L)
                    row["k"][L - n:] = _held(new("k", b, n, at, L))
                    row["v"][L - n:] = _held(s["v"][at:at + n].double())
                if op in ("q4_extend", "q4_read"):
                    for m in ("k", "v"):
                        got[m].view(-1, Hkv, D)[starts[b] * ps:starts[b] * ps + L] = row[m]
                else:
                    # (the step's query is held in bf16)
                    q = got["q"][b:b + 1].to(torch.bfloat16) if op == "q4_step" else s["q"][b:b + 1]
                    got["out"][b] = attend(q.double(), row["k"], row["v"])[0]
        at = ends[b]
    return got
