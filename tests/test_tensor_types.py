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


E4M3, E5M2, E8M0, U8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu, torch.uint8


def _calls():
    """name -> (call of an empty batch, which launches nothing, and its cache tensors' types)"""
    d = pkv.dims(0, 4, 2, 64, 16, 3, 0, 40)
    zeros = lambda t, *s: torch.zeros(*s, dtype=t)  # noqa: E731
    k, q = zeros(BF16, 0, 2, 64), zeros(BF16, 0, 4, 64)
    t = pkv.tokens(None, k, k)
    none = (None, None, None)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    pool = lambda kind: zeros(kind, 3, 16, 2, 64)  # noqa: E731
    bf16 = dict(k_pool=pool(BF16), v_pool=pool(BF16))
    q8 = dict(k_codes=pool(E4M3), v_codes=pool(E4M3), k_scale=zeros(U8, 3, 16, 2).view(E8M0),
              v_scale=zeros(U8, 3, 16, 2).view(E8M0))
    read = dict(q8, k_out=pool(BF16), v_out=pool(BF16))
    dec = dict(q8, q=q, out=q)
    four = lambda a: [a[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale")]  # noqa: E731
    return {
        "append_norm": (lambda a: pkv.paged_kv_append_norm(d, t, a["k_pool"], a["v_pool"], *none, stream=0), bf16),
        "extend_norm": (lambda a: pkv.paged_kv_extend_norm(d, t, None, a["k_pool"], a["v_pool"], *none, stream=0), bf16),
        "append_q8": (lambda a: pkv.paged_kv_append_q8(d, t, *four(a), *none, stream=0), q8),
        "extend_q8": (lambda a: pkv.paged_kv_extend_q8(d, t, None, *four(a), *none, stream=0), q8),
        "read_q8": (lambda a: pkv.paged_kv_read_q8(d, *four(a), *none, a["k_out"], a["v_out"], stream=0), read),
        "decode_q8": (lambda a: pkv.paged_decode_attn_q8(d, a["q"], *four(a), *none, 1, ws, a["out"], stream=0), dec),
        "decode_q8_planned": (lambda a: pkv.paged_decode_attn_q8_planned(d, a["q"], *four(a), *none, 1, ws, a["out"],
                                                                         stream=0), dec),
    }


@pytest.mark.parametrize("name", ["append_norm", "extend_norm", "append_q8", "extend_q8", "read_q8", "decode_q8",
                                  "decode_q8_planned"])
def test_a_cache_of_another_type_is_refused(name):
    """An 8-bit pool taken for bf16 would be written at twice its size."""
    call, args = _calls()[name]
    call(args)
    for at, right in args.items():
        for other in (F16, torch.float32, E5M2, U8, E4M3, E8M0, BF16):
            fits = (other is right.dtype or
                    (other is U8 and right.element_size() == 1))
            a = dict(args, **{at: torch.zeros(right.shape, dtype=other)})
            if fits:
                call(a)
            else:
                with pytest.raises(ValueError):
                    call(a)
        if right.dim() > 2 and right.numel():
            with pytest.raises(ValueError):
                call(dict(args, **{at: right.transpose(1, 2)}))


BF16_CALLS = {
    "append": lambda d, k, v, x, ws: pkv.paged_kv_append(d, x, x, x, k, v, *[None] * 3, stream=0),
    "extend": lambda d, k, v, x, ws: pkv.paged_kv_extend(d, x, x, x, None, k, v, *[None] * 3, stream=0),
    "decode": lambda d, k, v, x, ws: pkv.paged_decode_attn(d, x, k, v, *[None] * 3, 1, ws, x, stream=0),
    "planned": lambda d, k, v, x, ws: pkv.paged_decode_attn_planned(d, x, k, v, *[None] * 3, 1, ws, x, stream=0),
    "step": lambda d, k, v, x, ws: pkv.paged_decode_step(d, x, x, x, k, v, *[None] * 4, 0, 1, ws, x, stream=0),
    "step_planned": lambda d, k, v, x, ws: pkv.paged_decode_step_planned(d, x, x, x, k, v, *[None] * 4, 0, 1, ws, x,
                                                                         stream=0),
    "advance": lambda d, k, v, x, ws: pkv.paged_decode_step_advance(d, x, x, x, k, v, *[None] * 4, 0, 1, ws, x, None,
                                                                    None, stream=0),
    "contig": lambda d, k, v, x, ws: pkv.decode_attn_contig(d, x, k, v, None, 1, ws, x, stream=0),
    "partials": lambda d, k, v, x, ws: pkv.paged_decode_partials(d, x, k, v, *[None] * 3, 1, ws, stream=0),
    "noalloc": lambda d, k, v, x, ws: pkv.paged_decode_attn_noalloc(d, x, k, v, *[None] * 3, 1, x, stream=0),
    "prefill": lambda d, k, v, x, ws: pkv.paged_prefill_attn(d, x, None, k, v, *[None] * 3, x, stream=0),
    "prefill_ws": lambda d, k, v, x, ws: pkv.paged_prefill_attn(d, x, None, k, v, *[None] * 3, x, stream=0,
                                                                workspace=ws),
}


@pytest.mark.parametrize("name", BF16_CALLS)
def test_bf16_calls_refuse_the_codes_of_an_8_bit_cache(name):
    """They would be read at twice their size.  (An empty batch: nothing is launched.)"""
    d = pkv.dims(0, 4, 2, 64, 16, 3, 0, 40)
    x, ws = torch.zeros(0, 4, 64, dtype=BF16), torch.zeros(1 << 20, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    right = torch.zeros(3, 16, 2, 64, dtype=BF16)
    call = BF16_CALLS[name]
    call(d, right, right, x, ws)
    raw = right.view(U8)                              # bytes with room for bf16 pass as before
    call(d, raw, raw, x, ws)
    for kind in (U8, E4M3):
        codes = torch.zeros(3, 16, 2, 64, dtype=kind)
        for k, v in ((codes, right), (right, codes)):
            with pytest.raises(ValueError, match="too small"):
                call(d, k, v, x, ws)
