"""What is measured of the quantised key-value cache and the normalising cache writes.

Four operators around a paged cache (pools of [pages, page_size, Hkv, D], a
page table per row, D 64 or 128, grouped-query heads):

* ``norm_write``: the cache write of a step (one new token a row) or of ragged
  chunks, with an RMS norm of every query and key head before the rotation;
  bf16 pools.
* ``q8_write``: the same pass into a cache of e4m3 codes with one power-of-two
  scale (e8m0) for each token and kv head.
* ``q8_read``: the rows of such a cache back in bf16, in logical order.
* ``q8_decode``: attention of one new token a row over such a cache.

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


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step's cache write of a 1B-class model: the smallest call, all latency
        dict(name="norm_append_b8_d64", op="norm_write", B=8, Hq=32, Hkv=8, D=64, page=16, lo=513,
             hi=1025, shape="even", idle=0, q_lo=0, q_hi=0, norm=True, rope=True, packed=False),
        # the same of a serving batch padded to a power of two, q, k, v in one projection's output
        dict(name="norm_append_serving_b128", op="norm_write", B=128, Hq=64, Hkv=8, D=128, page=16,
             lo=16, hi=8192, shape="lognormal", idle=32, q_lo=0, q_hi=0, norm=True, rope=True,
             packed=True),
        # the write of four whole prompts of 4,096 tokens
        dict(name="norm_extend_4x4096", op="norm_write", B=4, Hq=32, Hkv=8, D=128, page=16, lo=4096,
             hi=4096, shape="even", idle=0, q_lo=4096, q_hi=4096, norm=True, rope=True, packed=True),
        # the quantising write of one step over ragged rows
        dict(name="q8_append_ragged_b32", op="q8_write", B=32, Hq=32, Hkv=8, D=128, page=16, lo=512,
             hi=4096, shape="even", idle=0, q_lo=0, q_hi=0, norm=False, rope=True, packed=True),
        # prompts of odd lengths behind a cached prefix, head size 64, odd pages, keys normalised
        dict(name="q8_extend_odd_d64", op="q8_write", B=32, Hq=32, Hkv=8, D=64, page=24, lo=301,
             hi=1021, shape="even", idle=0, q_lo=129, q_hi=509, norm=True, rope=True, packed=False),
        # sixteen extends of 256 tokens and more on longer contexts
        dict(name="q8_extend_b16", op="q8_write", B=16, Hq=32, Hkv=8, D=128, page=16, lo=2048, hi=2048,
             shape="even", idle=0, q_lo=256, q_hi=2048, norm=False, rope=True, packed=True),
        # two short rows read back: the smallest call
        dict(name="q8_read_tiny", op="q8_read", B=2, Hq=4, Hkv=2, D=64, page=16, lo=37, hi=100,
             shape="even", idle=0),
        # a ragged batch read back before a prefill over it
        dict(name="q8_read_ragged_b32", op="q8_read", B=32, Hq=32, Hkv=8, D=128, page=16, lo=512,
             hi=4096, shape="even", idle=0),
        # one decode step: two short rows; a 1B-class batch; one row of 32,768 tokens; a serving batch
        dict(name="q8_decode_tiny", op="q8_decode", B=2, Hq=4, Hkv=2, D=64, page=16, lo=37, hi=100,
             shape="even", idle=0),
        dict(name="q8_decode_1b_d64", op="q8_decode", B=8, Hq=32, Hkv=8, D=64, page=16, lo=513, hi=1025,
             shape="even", idle=0),
        dict(name="q8_decode_long_32k", op="q8_decode", B=1, Hq=32, Hkv=8, D=128, page=16, lo=32768,
             hi=32768, shape="even", idle=0),
        dict(name="q8_decode_serving_b128", op="q8_decode", B=128, Hq=64, Hkv=8, D=128, page=16, lo=16,
             hi=8192, shape="lognormal", idle=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm_write", "q8_write", "q8_read", "q8_decode", "q8_decode"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    rep = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 16])
    B = _log_int(rng, 1, 128)
    idle = rng.choice([0, 0, B // 4])
    # no more cached values than the largest listed rows of the kind have
    budget = 150e6 if op == "q8_decode" else 70e6 if op == "q8_read" else 16e6
    most = max(1, int(budget / (B * Hkv * D)))
    hi = _log_int(rng, 1, min(32768, most))
    lo = _log_int(rng, 1, hi)
    case = dict(op=op, B=B, Hq=Hkv * rep, Hkv=Hkv, D=D, page=rng.choice([1, 8, 16, 16, 17, 32, 64, 128]),
                lo=lo, hi=hi, shape="lognormal" if hi > 16 * lo else "even", idle=idle)
    if op.endswith("_write"):
        chunk = rng.random() < 0.6
        most_q = max(1, int(48e6 / (B * (case["Hq"] + 2 * Hkv) * D)))
        q_hi = _log_int(rng, 1, min(hi, most_q)) if chunk else 0
        q_lo = rng.randint(0, q_hi) if chunk else 0
        case.update(q_lo=q_lo, q_hi=q_hi, norm=rng.random() < 0.6, rope=rng.random() < 0.8,
                    packed=rng.random() < 0.5)
        case["norm"] = case["norm"] or (op == "norm_write" and not case["rope"])
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
    """New tokens of each row of a chunked write (no more than its length)."""
    n = len(lens)
    return [min(L, case["q_lo"] + ((case["q_hi"] - case["q_lo"]) * (n - 1 - i)) // max(1, n - 1)
                if n > 1 else case["q_hi"]) for i, L in enumerate(lens)]


# ------------------------------------------------------------------ the inputs
def _quantise(x):
    """(e4m3 codes, e8m0 scales) of head vectors x [..., D] in 32 bits: the
    smallest power of two that brings the largest value to 448 or under."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, LOW)).clamp(LOW, HIGH)
    codes = torch.ldexp(x, -e.unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(codes, scales):
    """What codes and scales stand for, in 32 bits."""
    e = scales.view(torch.uint8).to(torch.int32) - 127
    return torch.ldexp(codes.to(torch.float32), e.unsqueeze(-1))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    order = random.Random(seed)
    B, Hq, Hkv, D, ps = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
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
    if case["op"].endswith("_write"):
        T = B
        if case["q_hi"]:
            s["chunks"] = [n for _, n in rows] + [0] * case["idle"]
            ends = list(itertools.accumulate(s["chunks"]))
            s["qo_indptr"] = ints([0] + ends)
            T = ends[-1]
        # keys have a few large channels, as projections of trained models do
        loud = torch.exp(0.6 * randn(Hkv, D))
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
        kind = torch.bfloat16 if case["op"] == "norm_write" else torch.float8_e4m3fn
        s["k_pool"], s["v_pool"] = (torch.zeros(pool, dtype=kind, device=dev) for _ in range(2))
        if case["op"] == "q8_write":
            s["k_scale"], s["v_scale"] = (torch.full(pool[:3], 127, dtype=torch.uint8, device=dev)
                                          .view(torch.float8_e8m0fnu) for _ in range(2))
        return s
    loud = torch.exp(0.4 * randn(Hkv, D))
    for name, gain in (("k", loud), ("v", 1.0)):
        x = randn(*pool) * gain * torch.exp(0.5 * randn(*pool[:3], 1))
        s[name + "_pool"], s[name + "_scale"] = _quantise(x.to(torch.bfloat16).float())
        del x
    if case["op"] == "q8_read":
        shape = (max(1, n_ref), ps, Hkv, D)
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
    else:
        s["q"] = randn(B, Hq, D).to(torch.bfloat16)
        s["out"] = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=dev)
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


def _normed_rotated(s, x, weight, pos):
    x = x.to(torch.float32)
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(torch.float32)
    if "rope" in s:
        c, r = s["rope"][pos, :, 0].unsqueeze(1), s["rope"][pos, :, 1].unsqueeze(1)
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack([a * c - b * r, a * r + b * c], -1).flatten(-2)
    return x


def _plain_write(s):
    case, dev = s["case"], s["k"].device
    D, Hkv = case["D"], case["Hkv"]
    live = s["lens"][:case["B"] - case["idle"]]
    if "qo_indptr" in s:
        row, at = _of_rows(s["chunks"], dev)
        pos = s["seq_lens"].long()[row] - (s["qo_indptr"].long()[row + 1] - s["qo_indptr"].long()[row]) + at
    else:
        row = torch.arange(len(live), device=dev)
        pos = s["seq_lens"].long()[row] - 1
    n = row.numel()
    s["q_out"][:n] = _normed_rotated(s, s["q"][:n], s.get("q_norm"), pos).to(torch.bfloat16)
    slot = _slots(s, row, pos)
    k = _normed_rotated(s, s["k"][:n], s.get("k_norm"), pos)
    v = s["v"][:n].to(torch.float32)
    if case["op"] == "norm_write":
        s["k_pool"].view(-1, Hkv, D)[slot] = k.to(torch.bfloat16)
        s["v_pool"].view(-1, Hkv, D)[slot] = v.to(torch.bfloat16)
        return
    for name, x in (("k", k), ("v", v)):
        codes, scales = _quantise(x)
        s[name + "_pool"].view(torch.uint8).view(-1, Hkv, D)[slot] = codes.view(torch.uint8)
        s[name + "_scale"].view(torch.uint8).view(-1, Hkv)[slot] = scales.view(torch.uint8)


def _gathered(s, name, slot):
    """Dequantised head vectors at flat slots, [..., Hkv, D] in 32 bits."""
    Hkv, D = s["case"]["Hkv"], s["case"]["D"]
    codes = s[name + "_pool"].view(torch.uint8).view(-1, Hkv, D)[slot].view(torch.float8_e4m3fn)
    return _values(codes, s[name + "_scale"].view(torch.uint8).view(-1, Hkv)[slot])


def _plain_read(s):
    Hkv, D, ps = s["case"]["Hkv"], s["case"]["D"], s["case"]["page"]
    row, pos = _of_rows(s["lens"], s["seq_lens"].device)
    slot = _slots(s, row, pos)
    to = s["kv_indptr"].long()[row] * ps + pos
    s["k_out"].view(-1, Hkv, D)[to] = _gathered(s, "k", slot).to(torch.bfloat16)
    s["v_out"].view(-1, Hkv, D)[to] = _gathered(s, "v", slot).to(torch.bfloat16)


def _plain_decode(s):
    case, dev = s["case"], s["q"].device
    B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
    pos = torch.arange(max(s["lens"] + [1]), device=dev)
    there = pos < s["seq_lens"][:, None]                              # [B, L]
    rows = torch.arange(B, device=dev)[:, None].expand_as(there)
    entry = (s["kv_indptr"].long()[rows] + pos // case["page"]).clamp(max=s["kv_indices"].numel() - 1)
    slot = torch.where(there, s["kv_indices"].long()[entry] * case["page"] + pos % case["page"], 0)
    k = _gathered(s, "k", slot).permute(0, 2, 3, 1)                    # [B, Hkv, D, L]
    q = s["q"].to(torch.float32).view(B, Hkv, Hq // Hkv, D)
    x = (q @ k) * (1.0 / math.sqrt(D))                                 # [B, Hkv, rep, L]
    del k
    x = torch.where(there[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = p @ _gathered(s, "v", slot).permute(0, 2, 1, 3)                # [B, Hkv, rep, D]
    s["out"].copy_(o.reshape(B, Hq, D))


# ------------------------------------------------------------ the library's own
def _dims(s, pkv):
    c = s["case"]
    if "dims" not in s["kept"]:
        s["kept"]["dims"] = pkv.dims(c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], s["k_pool"].shape[0],
                                     s["kv_indices"].numel(), s["max_len"])
        s["kept"]["status"] = torch.zeros(1, dtype=torch.int32, device=s["seq_lens"].device)
    return s["kept"]["dims"], s["kept"]["status"]


def _own_write(s, pkv):
    d, status = _dims(s, pkv)
    rope = s.get("rope")
    t = pkv.tokens(s["q"], s["k"], s["v"], q_out=s["q_out"], q_norm=s.get("q_norm"),
                   k_norm=s.get("k_norm"), norm_eps=EPS, rope_cos_sin=rope,
                   rope_max_pos=0 if rope is None else rope.shape[0])
    table = (s["kv_indices"], s["kv_indptr"], s["seq_lens"])
    if s["case"]["op"] == "norm_write":
        if "qo_indptr" in s:
            pkv.paged_kv_extend_norm(d, t, s["qo_indptr"], s["k_pool"], s["v_pool"], *table, status=status)
        else:
            pkv.paged_kv_append_norm(d, t, s["k_pool"], s["v_pool"], *table, status=status)
        return
    cache = (s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
    if "qo_indptr" in s:
        pkv.paged_kv_extend_q8(d, t, s["qo_indptr"], *cache, *table, status=status)
    else:
        pkv.paged_kv_append_q8(d, t, *cache, *table, status=status)


def _own_read(s, pkv):
    d, status = _dims(s, pkv)
    pkv.paged_kv_read_q8(d, s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["kv_indices"],
                         s["kv_indptr"], s["seq_lens"], s["k_out"], s["v_out"], status=status)


def _own_decode(s, pkv):
    d, _ = _dims(s, pkv)
    if "workspace" not in s["kept"]:
        s["kept"]["splits"] = pkv.plan(d)[0]
        s["kept"]["workspace"] = pkv.alloc_workspace(d, s["kept"]["splits"], s["q"].device)
    pkv.paged_decode_attn_q8(d, s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                             s["kv_indices"], s["kv_indptr"], s["seq_lens"], s["kept"]["splits"],
                             s["kept"]["workspace"], s["out"])


def run(s):
    op = s["case"]["op"]
    if own:
        from paged_kv_gqa_16_gb300 import pkv
        {"norm_write": _own_write, "q8_write": _own_write, "q8_read": _own_read, "q8_decode": _own_decode}[op](s, pkv)
    else:
        {"norm_write": _plain_write, "q8_write": _plain_write, "q8_read": _plain_read, "q8_decode": _plain_decode}[op](s)
    if op == "norm_write":
        return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}
    if op == "q8_write":
        return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if op == "q8_read":
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"out": s["out"]}


def work(case):
    """Each new or cached token's values read and written once, in the types they are held in."""
    lens = _lens(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    tables = 4 * (2 * case["B"] + 1 + sum(-(-L // case["page"]) for L in lens))
    total = sum(lens)
    if case["op"].endswith("_write"):
        T = sum(_chunks(case, lens)) if case["q_hi"] else len(lens)
        kept = 2 * Hkv * D * 2 if case["op"] == "norm_write" else 2 * Hkv * (D + 1)
        cos_sin = 4 * D * min(T, max(case["hi"], 1)) if case["rope"] else 0
        per = (Hq + 2 * Hkv) * D * 2 + Hq * D * 2 + kept
        ops = (Hq + Hkv) * D * ((3 if case["rope"] else 0) + (4 if case["norm"] else 0)) + 4 * Hkv * D
        return {"bytes": T * per + cos_sin + 12 * case["B"] + 4 * T, "flops": T * ops}
    if case["op"] == "q8_read":
        return {"bytes": total * 2 * Hkv * (D + 1 + 2 * D) + tables, "flops": total * 2 * Hkv * D}
    return {"bytes": total * 2 * Hkv * (D + 1) + 2 * case["B"] * Hq * D * 2 + tables,
            "flops": total * 4 * Hq * D}


# --------------------------------------------------------------- in 64 bits
def _e4m3(x):
    """x, at most 448 in size, rounded to the nearest value of four significant
    bits (steps of 2^-9 under 2^-6), ties to even."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    Hq, Hkv, D, ps = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    lens, starts = s["lens"], s["kv_indptr"].tolist()
    table = s["kv_indices"].long()

    def places(b, first, last):
        t = torch.arange(first, last, device=table.device)
        return table[starts[b] + torch.div(t, ps, rounding_mode="floor")], torch.remainder(t, ps)

    def cached(name, at):
        scale = torch.exp2(s[name + "_scale"].view(torch.uint8)[at].double() - 127.0)
        return s[name + "_pool"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * scale[..., None]

    if case["op"] == "q8_decode":
        out = torch.zeros(case["B"], Hq, D, dtype=torch.float64, device=table.device)
        for b, L in enumerate(lens):
            if L:
                k, v = cached("k", places(b, 0, L)), cached("v", places(b, 0, L))
                q = s["q"][b].double().view(Hkv, Hq // Hkv, D)
                w = torch.softmax(torch.einsum("grd,lgd->grl", q, k) / math.sqrt(D), -1)
                out[b] = torch.einsum("grl,lgd->grd", w, v).reshape(Hq, D)
        return {"out": out}
    if case["op"] == "q8_read":
        got = {}
        for name in ("k", "v"):
            got[name] = s[name + "_out"].double()
            for b, L in enumerate(lens):
                if L:
                    flat = got[name].view(-1, Hkv, D)
                    flat[starts[b] * ps:starts[b] * ps + L] = cached(name, places(b, 0, L))
        return got
    got = {n: s[m].double() for n, m in (("q", "q_out"), ("k", "k_pool"), ("v", "v_pool"))}
    if case["op"] == "q8_write":
        got["k_scale"], got["v_scale"] = (torch.exp2(s[n].view(torch.uint8).double() - 127.0)
                                          for n in ("k_scale", "v_scale"))
    at = 0
    chunk = "qo_indptr" in s
    ends = s["qo_indptr"].tolist()[1:] if chunk else list(range(1, case["B"] + 1))
    for b, L in enumerate(lens):
        n = ends[b] - at
        if L and n:
            here = places(b, L - n, L)
            new = {"q": s["q"][at:ends[b]].double(), "k": s["k"][at:ends[b]].double(), "v": s["v"][at:ends[b]].double()}
            for name in ("q", "k"):
                x = new[name]
                if case["norm"]:
                    x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * s[name + "_norm"].double()
                if case["rope"]:
                    turn = torch.view_as_complex(s["rope"][L - n:L].double())[:, None]
                    x = torch.view_as_real(torch.view_as_complex(x.reshape(n, -1, D // 2, 2).contiguous()) * turn).reshape(n, -1, D)
                new[name] = x
            got["q"][at:ends[b]] = new["q"]
            for name in ("k", "v"):
                x = new[name]
                if case["op"] == "q8_write":
                    big = x.abs().amax(-1)
                    e = torch.ceil(torch.log2(big / 448.0)).clamp(LOW, HIGH)
                    got[name + "_scale"][here] = torch.exp2(e)
                    x = _e4m3(x * torch.exp2(-e)[..., None])
                got[name][here] = x
        at = ends[b]
    return got
