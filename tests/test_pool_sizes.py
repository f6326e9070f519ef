"""The sizes of the tensors that the 8-bit and 4-bit cache's calls, the normalising writes and the
calls through a window take: one too small for the dims is refused before anything is launched, so
no GPU is needed."""

import pytest
import torch

from paged_kv_gqa_16_gb300 import build as pkv_build
from paged_kv_gqa_16_gb300 import pkv

BF16, E4M3, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8
Hq, Hkv, PS, PAGES = 4, 2, 16, 3


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def _calls(D, B=0, indices=0):
    """name -> (call, its tensors); an empty batch, which launches nothing."""
    d = pkv.dims(B, Hq, Hkv, D, PS, PAGES, indices, 40)
    zeros = lambda t, *s: torch.zeros(*s, dtype=t)  # noqa: E731
    k = zeros(BF16, B, Hkv, D)
    t = pkv.tokens(None, k, k)
    none = (None, None, None)
    ws = torch.zeros(1 << 20, dtype=U8)
    ws = ws[-ws.data_ptr() % 256:]
    rows = lambda: zeros(BF16, B, Hq, D)  # noqa: E731
    pool = lambda kind, last: zeros(kind, PAGES, PS, Hkv, *last)  # noqa: E731
    bf16 = dict(k_pool=pool(BF16, [D]), v_pool=pool(BF16, [D]))
    q8 = dict(k_codes=pool(E4M3, [D]), v_codes=pool(E4M3, [D]), k_scale=pool(U8, []), v_scale=pool(U8, []))
    q4 = dict(k_codes=pool(U8, [D // 2]), v_codes=pool(U8, [D // 2]), k_scale=pool(U8, [D // 32]),
              v_scale=pool(U8, [D // 32]))
    read = lambda: dict(k_out=zeros(BF16, indices, PS, Hkv, D), v_out=zeros(BF16, indices, PS, Hkv, D))  # noqa: E731
    qo = lambda: dict(q=rows(), out=rows())  # noqa: E731
    four = lambda a: [a[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale")]  # noqa: E731
    two = lambda a: [a["k_pool"], a["v_pool"]]  # noqa: E731
    P = pkv
    return {
        "append_norm": (lambda a: P.paged_kv_append_norm(d, t, *two(a), *none, stream=0), bf16),
        "extend_norm": (lambda a: P.paged_kv_extend_norm(d, t, None, *two(a), *none, stream=0), bf16),
        "append_q8": (lambda a: P.paged_kv_append_q8(d, t, *four(a), *none, stream=0), q8),
        "extend_q8": (lambda a: P.paged_kv_extend_q8(d, t, None, *four(a), *none, stream=0), q8),
        "read_q8": (lambda a: P.paged_kv_read_q8(d, *four(a), *none, a["k_out"], a["v_out"], stream=0),
                    dict(q8, **read())),
        "decode_q8": (lambda a: P.paged_decode_attn_q8(d, a["q"], *four(a), *none, 1, ws, a["out"], stream=0),
                      dict(q8, **qo())),
        "decode_q8_planned": (lambda a: P.paged_decode_attn_q8_planned(d, a["q"], *four(a), *none, 1, ws, a["out"],
                                                                       stream=0), dict(q8, **qo())),
        "append_q4": (lambda a: P.paged_kv_append_q4(d, t, *four(a), *none, stream=0), q4),
        "extend_q4": (lambda a: P.paged_kv_extend_q4(d, t, None, *four(a), *none, stream=0), q4),
        "read_q4": (lambda a: P.paged_kv_read_q4(d, *four(a), *none, a["k_out"], a["v_out"], stream=0),
                    dict(q4, **read())),
        "decode_q4": (lambda a: P.paged_decode_attn_q4(d, a["q"], *four(a), *none, 1, ws, a["out"], stream=0),
                      dict(q4, **qo())),
        "decode_window": (lambda a: P.paged_decode_attn_window(d, a["q"], *two(a), *none, 8, 1, 1, ws, a["out"],
                                                               stream=0), dict(bf16, **qo())),
        "prefill_window": (lambda a: P.paged_prefill_attn_window(d, a["q"], None, *two(a), *none, 8, 1, a["out"],
                                                                 stream=0), dict(bf16, **qo())),
    }


NAMES = list(_calls(64))
POOLS = ("k_pool", "v_pool", "k_codes", "v_codes", "k_scale", "v_scale")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("D", [64, 128])
def test_a_pool_of_fewer_slots_is_refused(name, D):
    call, args = _calls(D)[name]
    call(args)
    for at, right in args.items():
        if at in POOLS:
            call(dict(args, **{n: torch.cat([x, x]) for n, x in args.items() if n in POOLS}))     # more are
            with pytest.raises(ValueError):
                call(dict(args, **{at: right[:-1].contiguous()}))
    with pytest.raises(ValueError):                    # all of them: the kinds agree with each other
        call(dict(args, **{n: x[:-1].contiguous() for n, x in args.items() if n in POOLS}))
    with pytest.raises(ValueError):
        call(dict(args, **{n: x[:0] for n, x in args.items() if n in POOLS}))


@pytest.mark.parametrize("name", NAMES)
def test_a_cache_of_smaller_heads_is_refused(name):
    """A cache of heads of 64 behind dims of heads of 128 would be read past its end."""
    call, args = _calls(128)[name]
    small = _calls(64)[name][1]
    with pytest.raises(ValueError):
        call(dict(args, **{n: x for n, x in small.items() if n in POOLS}))


@pytest.mark.parametrize("name", [n for n in NAMES if n.startswith(("decode", "prefill", "read"))])
def test_a_short_query_or_output_is_refused(name):
    call, args = _calls(64, B=3, indices=2)[name]
    for at in args:
        if at not in POOLS and not (name == "prefill_window" and at == "q"):   # (whose rows are counted from it)
            with pytest.raises(ValueError):
                call(dict(args, **{at: args[at][:-1].contiguous()}))
    if name == "prefill_window":
        with pytest.raises(ValueError):
            call(dict(args, q=args["q"][:, :-1].contiguous()))


@pytest.mark.parametrize("name", ["prefill", "prefill_window"])
def test_the_prefill_refuses_pools_past_its_offsets(name):
    """It keeps pool offsets in 16-byte units of 32 bits: fewer than 2^35 elements."""
    x = torch.zeros(1, 1, 64, dtype=BF16)
    some = torch.zeros(2, dtype=torch.int32)
    for pages in ((1 << 35) // (16 * 64), (1 << 31) // 16 * 2 - 1):
        d = pkv.dims(1, 1, 1, 64, 16, pages, 0, 1)
        with pytest.raises(pkv.PkvError) as e:
            if name == "prefill":
                pkv.paged_prefill_attn(d, x, some, 16, 16, None, some, some, x, stream=0)
            else:
                pkv.paged_prefill_attn_window(d, x, some, 16, 16, None, some, some, 4, 1, x, stream=0)
        assert e.value.code == pkv.PKV_ERR_UNSUPPORTED
