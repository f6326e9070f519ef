"""Host-side checks of the normalising writes and the 8-bit cache's calls: every
case fails before a launch, so no GPU is needed and no pointer is followed."""

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


def _write(q8, extend, d=None, t=None, total_q=8, **kw):
    a = dict(qo=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, ind=FAKE, ptr=FAKE, sl=FAKE, st=None)
    a.update(kw)
    args = [ctypes.byref(d or _d()), None if t is None else ctypes.byref(t)]
    if extend:
        args += [a["qo"], total_q]
    args += [a["k"], a["v"]]
    if q8:
        args += [a["ks"], a["vs"]]
    args += [a["ind"], a["ptr"], a["sl"], a["st"], None]
    name = "paged_kv_%s_%s" % ("extend" if extend else "append", "q8" if q8 else "norm")
    return getattr(pkv.lib(), name)(*args)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("extend", [False, True])
def test_write_refusals(q8, extend):
    call = lambda **kw: _write(q8, extend, **dict(dict(t=_t()), **kw))  # noqa: E731
    assert call(t=None) == BAD
    for field in ("k", "v", "q_out"):
        assert call(t=_t(**{field: None})) == BAD, field
    for field in ("q", "k", "v", "q_out", "q_norm", "k_norm"):
        assert call(t=_t(**{field: FAKE + 8})) == BAD, field
    for field in ("q_stride", "k_stride", "v_stride"):
        heads = 32 if field[0] == "q" else 8
        for stride in (heads * 128 - 8, heads * 128 + 4, -heads * 128, 8):
            assert call(t=_t(**{field: stride})) == BAD, (field, stride)
    # in place needs a packed q
    assert call(t=_t(q_out=FAKE, q_stride=48 * 128)) == BAD
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(t=_t(k_norm=FAKE, norm_eps=eps)) == BAD
        assert call(t=_t(q_norm=FAKE, norm_eps=eps)) == BAD
    assert call(t=_t(rope_cos_sin=FAKE, rope_max_pos=0)) == BAD
    assert call(t=_t(rope_cos_sin=FAKE + 4, rope_max_pos=9)) == BAD
    for name in ("k", "v", "ptr", "sl") + (("ks", "vs") if q8 else ()) + (("qo",) if extend else ()):
        assert call(**{name: None}) == BAD, name
        assert call(**{name: FAKE + 2}) == BAD, name
    assert call(ind=None) == BAD and call(st=FAKE + 1) == BAD
    assert call(d=_d(D=96)) == UNSUP and call(d=_d(Hq=30)) == BAD
    assert call(d=_d(Hq=1 << 25, Hkv=1 << 21)) in (BAD, UNSUP)
    # nothing to do
    assert call(d=_d(B=0)) == pkv.PKV_OK
    if extend:
        assert call(total_q=-1) == BAD and call(total_q=0) == pkv.PKV_OK


def test_read_refusals():
    def call(d=None, **kw):
        a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, ind=FAKE, ptr=FAKE, sl=FAKE, ko=FAKE, vo=FAKE, st=None)
        a.update(kw)
        return pkv.lib().paged_kv_read_q8(ctypes.byref(d or _d()), *a.values(), None)

    for name in ("kc", "vc", "ks", "vs", "ptr", "sl", "ko", "vo", "ind"):
        assert call(**{name: None}) == BAD, name
        assert call(**{name: FAKE + 2}) == BAD, name
    assert call(st=FAKE + 1) == BAD and call(kc=FAKE + 8) == BAD and call(ko=FAKE + 8) == BAD
    assert call(d=_d(D=32)) == UNSUP
    assert call(d=_d(B=0)) == pkv.PKV_OK


def test_decode_refusals():
    d = _d()
    need = pkv.workspace_bytes(d, 8)

    def call(d=d, splits=8, ws_bytes=need, **kw):
        a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, ind=FAKE, ptr=FAKE, sl=FAKE)
        a.update({k: v for k, v in kw.items() if k in a})
        return pkv.lib().paged_decode_attn_q8(ctypes.byref(d), *a.values(), splits, kw.get("ws", FAKE),
                                              ws_bytes, kw.get("out", FAKE), None)

    for name in ("q", "kc", "vc", "ks", "vs", "ind", "ptr", "sl", "ws", "out"):
        assert call(**{name: None}) == BAD, name
        assert call(**{name: FAKE + 2}) == BAD, name
    assert call(ks=FAKE + 8) == BAD and call(ws=FAKE + 16) == BAD
    assert call(splits=0) == BAD and call(splits=70000) == BAD
    assert call(ws_bytes=need - 1) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    assert call(d=_d(D=96)) == UNSUP and call(d=_d(Hq=8 * 17)) == UNSUP
    assert call(d=_d(B=0)) == pkv.PKV_OK


def test_plan_refusals():
    d = _d()
    need = pkv.workspace_bytes(d, 8)
    call = lambda d=d, ind=FAKE, ptr=FAKE, sl=FAKE, S=8, ws=FAKE, n=need: pkv.lib().paged_decode_plan_q8(  # noqa: E731
        ctypes.byref(d), ind, ptr, sl, S, ws, n, None)
    assert call(ind=None) == BAD and call(ptr=None) == BAD and call(sl=FAKE + 2) == BAD
    assert call(S=0) == BAD and call(ws=None) == BAD and call(ws=FAKE + 16) == BAD
    assert call(n=need - 1) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    assert call(d=_d(B=0)) == pkv.PKV_OK
    # a batch of several launches has no plan: nothing is launched
    d = _d(B=1025)
    assert call(d=d, n=pkv.workspace_bytes(d, 8)) == pkv.PKV_OK


def test_decode_limits():
    """Shapes that the kernel cannot count are refused, the largest that it can are not."""
    def call(**kw):
        d = _d(**kw)
        return pkv.lib().paged_decode_attn_q8(ctypes.byref(d), *[FAKE] * 8, 1, FAKE, 1 << 40, FAKE, None)

    assert call(B=1, Hq=1031, Hkv=1031) == UNSUP                       # 1031 groups of one head
    assert call(B=1, num_pages=1 << 27, page_size=16) == UNSUP         # 2^31 token slots
    assert call(B=1, Hq=24, Hkv=24, max_seq_len=1 << 30) == UNSUP      # 3 groups of 2^30 tokens


def test_tokens_of_torch_rows():
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    both = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    t = pkv.tokens(both[:, :4], both[:, 4:6], both[:, 6:], q)
    assert (t.q_stride, t.k_stride, t.v_stride) == (512, 512, 512) and t.k == both.data_ptr() + 512
    assert pkv.tokens(q, k, k).q_out == q.data_ptr()
    assert pkv.tokens(None, k, k).q is None
    one = both[:1, :4]
    assert pkv.tokens(one, both[:1, 4:6], both[:1, 6:], q).q_stride == 0      # a single row is packed
    with pytest.raises(ValueError):
        pkv.tokens(q, k, torch.zeros(2, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        pkv.tokens(q, both[:, ::2][:, :2], k)                                  # heads not packed
    with pytest.raises(ValueError):
        pkv.tokens(q[..., ::2], k, k)
    with pytest.raises(ValueError):
        pkv.tokens(q.float(), k, k)
    with pytest.raises(ValueError):
        pkv._token_count(_d(B=3), pkv.tokens(q, k, k))                         # other heads
    with pytest.raises(ValueError):
        pkv._token_count(_d(B=4, Hq=4, Hkv=2, D=64), pkv.tokens(q, k, k), per_row=True)


def test_tokens_refuse_expanded_rows_and_short_tensors():
    """A row stride of 0 stands for packed rows in the C call: rows that share memory would
    be read past their end."""
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    for bad in ((q[:1].expand(3, 4, 64), k, k), (q, k[:1].expand(3, 2, 64), k),
                (q, k, k[:1].expand(3, 2, 64))):
        with pytest.raises(ValueError):
            pkv.tokens(*bad, torch.empty_like(q))
    assert pkv.tokens(q[:1], k[:1].expand(1, 2, 64), k[:1], torch.empty_like(q)).k_stride == 0
    with pytest.raises(ValueError):
        pkv.tokens(q, k, k, torch.empty_like(q[:2]))
    for kw in (dict(q_norm=w[:32]), dict(q_norm=w.float()), dict(k_norm=w[:32]), dict(k_norm=w.float())):
        with pytest.raises(ValueError):
            pkv.tokens(q, k, k, torch.empty_like(q), **kw)
    assert pkv.tokens(q, k, k, torch.empty_like(q), w, w).k_norm == w.data_ptr()
    rope = torch.zeros(5, 32, 2)
    assert pkv.tokens(q, k, k, rope_cos_sin=rope, rope_max_pos=5).rope_cos_sin == rope.data_ptr()
    for bad in (dict(rope_cos_sin=rope, rope_max_pos=6), dict(rope_cos_sin=rope[..., :1], rope_max_pos=1),
                dict(k_norm=torch.zeros(128, dtype=torch.bfloat16)[::2]),
                dict(q_out=torch.zeros(3, 4, 128, dtype=torch.bfloat16)[..., ::2])):
        with pytest.raises(ValueError):
            pkv.tokens(q, k, k, **bad)
