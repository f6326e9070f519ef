"""Host-side checks of the 4-bit cache's calls: every case fails before a
launch, so no GPU is needed and no pointer is followed."""

import ctypes

import pytest
import torch

from paged_kv_gqa_16_gb300 import build as pkv_build
from paged_kv_gqa_16_gb300 import pkv

FAKE = 1 << 32
BAD, UNSUP = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def _d(**kw):
    base = dict(B=4, Hq=32, Hkv=8, D=128, page_size=16, num_pages=64, num_indices=50, max_seq_len=400)
    return pkv.dims(**dict(base, **kw))


def _t(**kw):
    base = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE + 4096, norm_eps=1e-6)
    return pkv.Tokens(**dict(base, **kw))


@pytest.mark.parametrize("extend", [False, True])
def test_write_refusals(extend):
    def call(d=None, t="", total_q=8, **kw):
        a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, ind=FAKE, ptr=FAKE, sl=FAKE, st=None)
        a.update({k: v for k, v in kw.items() if k in a})
        t = _t() if t == "" else t
        args = [ctypes.byref(d or _d()), None if t is None else ctypes.byref(t)]
        if extend:
            args += [kw.get("qo", FAKE), total_q]
        name = "paged_kv_extend_q4" if extend else "paged_kv_append_q4"
        return getattr(pkv.lib(), name)(*args, *a.values(), None)

    assert call(t=None) == BAD
    for field in ("k", "v", "q_out"):
        assert call(t=_t(**{field: None})) == BAD, field
    for field in ("q", "k", "v", "q_out", "q_norm", "k_norm"):
        assert call(t=_t(**{field: FAKE + 8})) == BAD, field
    for field in ("kc", "vc", "ks", "vs", "ptr", "sl", "ind") + (("qo",) if extend else ()):
        assert call(**{field: None}) == BAD, field
        assert call(**{field: FAKE + 2}) == BAD, field
    assert call(ks=FAKE + 8) == BAD and call(st=FAKE + 1) == BAD
    assert call(t=_t(k_norm=FAKE, norm_eps=-1.0)) == BAD
    assert call(t=_t(rope_cos_sin=FAKE, rope_max_pos=0)) == BAD
    assert call(d=_d(D=96)) == UNSUP and call(d=_d(Hq=30)) == BAD
    assert call(d=_d(B=0)) == pkv.PKV_OK
    if extend:
        assert call(total_q=-1) == BAD and call(total_q=0) == pkv.PKV_OK


def test_read_refusals():
    def call(d=None, **kw):
        a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, ind=FAKE, ptr=FAKE, sl=FAKE, ko=FAKE, vo=FAKE, st=None)
        a.update(kw)
        return pkv.lib().paged_kv_read_q4(ctypes.byref(d or _d()), *a.values(), None)

    for name in ("kc", "vc", "ks", "vs", "ptr", "sl", "ko", "vo", "ind"):
        assert call(**{name: None}) == BAD, name
        assert call(**{name: FAKE + 2}) == BAD, name
    assert call(st=FAKE + 1) == BAD and call(kc=FAKE + 8) == BAD and call(ko=FAKE + 8) == BAD
    assert call(d=_d(D=32)) == UNSUP
    assert call(d=_d(B=0)) == pkv.PKV_OK


def test_tensors_of_another_cache_are_refused():
    """An 8-bit cache has byte tensors too, and one scale for a head vector: too few."""
    codes = torch.zeros(2, 16, 8, 64, dtype=torch.uint8)
    scale = torch.zeros(2, 16, 8, 4, dtype=torch.uint8)
    want = (codes.data_ptr(),) * 2 + (scale.data_ptr(),) * 2
    assert pkv._q4_ptrs(codes, codes, scale, scale) == want
    e8m0 = scale.view(torch.float8_e8m0fnu)
    assert pkv._q4_ptrs(codes, codes, e8m0, e8m0) == want
    assert pkv._q4_ptrs(FAKE, FAKE, FAKE, None) == (FAKE, FAKE, FAKE, None)
    for bad in ([codes, codes, scale[..., 0].contiguous(), scale], [codes[:1], codes, scale, scale],
                [codes.to(torch.bfloat16), codes, scale, scale], [codes, codes.transpose(1, 2), scale, scale],
                [codes.view(torch.float8_e4m3fn), codes, scale, scale], [codes, None, scale, scale],
                [codes, codes, scale, FAKE]):
        with pytest.raises(ValueError):
            pkv._q4_ptrs(*bad)


@pytest.mark.parametrize("name", ["paged_decode_attn_q4", "paged_decode_attn_window"])
def test_decode_refusals(name):
    d = _d()
    need = pkv.workspace_bytes(d, 8)
    q4 = name.endswith("q4")

    def call(d=d, splits=8, ws_bytes=need, window=64, sinks=4, **kw):
        a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, ind=FAKE, ptr=FAKE, sl=FAKE)
        if not q4:
            del a["ks"], a["vs"]
        a.update({k: v for k, v in kw.items() if k in a})
        return getattr(pkv.lib(), name)(ctypes.byref(d), *a.values(), window, sinks, splits, kw.get("ws", FAKE),
                                        ws_bytes, kw.get("out", FAKE), None)

    for field in ("q", "kc", "vc", "ind", "ptr", "sl", "ws", "out") + (("ks", "vs") if q4 else ()):
        assert call(**{field: None}) == BAD, field
        assert call(**{field: FAKE + 2}) == BAD, field
    assert call(ws=FAKE + 16) == BAD and call(q=FAKE + 8) == BAD
    assert call(splits=0) == BAD and call(splits=70000) == BAD
    assert call(window=-1) == BAD and call(sinks=-1) == BAD
    assert call(ws_bytes=need - 1) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    assert call(d=_d(D=96)) == UNSUP and call(d=_d(Hq=8 * 17)) == UNSUP
    assert call(d=_d(B=0)) == pkv.PKV_OK
    big = _d(num_pages=1 << 28)
    assert call(d=big, ws_bytes=pkv.workspace_bytes(big, 8)) == UNSUP


def test_window_prefill_refusals():
    def call(d=None, total_q=8, max_q=8, window=64, sinks=4, **kw):
        a = dict(q=FAKE, qo=FAKE, k=FAKE, v=FAKE, ind=FAKE, ptr=FAKE, sl=FAKE, ws=FAKE, out=FAKE, st=None)
        a.update(kw)
        return pkv.lib().paged_prefill_attn_window(
            ctypes.byref(d or _d()), a["q"], a["qo"], total_q, max_q, a["k"], a["v"], a["ind"], a["ptr"], a["sl"],
            window, sinks, a["ws"], 1 << 20, a["out"], a["st"], None)

    for field in ("q", "qo", "k", "v", "ind", "ptr", "sl", "out"):
        assert call(**{field: None}) == BAD, field
        assert call(**{field: FAKE + 2}) == BAD, field
    assert call(ws=FAKE + 16) == BAD and call(st=FAKE + 1) == BAD
    assert call(window=-1) == BAD and call(sinks=-1) == BAD
    assert call(total_q=-1) == BAD and call(max_q=-1) == BAD
    assert call(d=_d(D=96)) == UNSUP and call(d=_d(B=0)) == pkv.PKV_OK and call(total_q=0) == pkv.PKV_OK
