"""Refusals of the sink-window attention and the norm + rotation: every case fails the
argument checks, which come before any CUDA call (CPU only)."""

import ctypes
import os

import pytest
import torch

import linear_attention_sequence_causal_b200 as based
from linear_attention_sequence_causal_b200 import binding

FAKE = ctypes.c_void_p(1 << 20)        # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
INVALID, UNSUPPORTED = binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from linear_attention_sequence_causal_b200 import build
        build.build()
    return based.lib()


SIZES = dict(B=2, Hq=4, Hkv=2, N=16, d=64, w=8, s=4, scale=0.125, dt=1)
BAD_SIZES = [
    (dict(B=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=3), INVALID), (dict(w=0), INVALID),
    (dict(w=-1), INVALID), (dict(s=-1), INVALID), (dict(scale=-0.1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(dt=2), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
    (dict(s=65), UNSUPPORTED), (dict(B=1 << 24), UNSUPPORTED), (dict(w=(1 << 29) + 1), UNSUPPORTED),
]


def _strides(*s):
    return ctypes.byref(binding.Strides(*s))


BAD_STRIDES = [
    (4 * 16 * 64, 16 * 64, 60),            # a token stride that is no multiple of 16 bytes
    (4 * 16 * 64, 16 * 64, 0),             # broadcast rows overlap
    (4 * 16 * 64, 16 * 64, 32),            # rows overlap
    (4 * 16 * 64, 8 * 64, 64),             # heads overlap
    (0, 16 * 64, 64), (4 * 16 * 64, -16 * 64, 64), (1 << 39, 16 * 64, 64),
]


def test_prefill_refusals(lib):
    def call(q=FAKE, sq=None, lse=None, kc=None, vc=None, ln=None, **kw):
        a = dict(SIZES, **kw)
        return lib.based_swa_sink_prefill(q, sq, FAKE, None, FAKE, None, FAKE, None, lse, kc, vc, ln, a["B"], a["Hq"],
                                          a["Hkv"], a["N"], a["d"], a["w"], a["s"], a["scale"], a["dt"], None)

    for kw, want in BAD_SIZES + [(dict(N=0), INVALID), (dict(N=(1 << 29) + 1), UNSUPPORTED)]:
        assert call(**kw) == want, kw
    assert call(q=None) == INVALID and call(q=ODD) == INVALID
    assert call(lse=ODD) == INVALID and call(kc=FAKE) == INVALID and call(vc=FAKE) == INVALID
    assert call(kc=FAKE, vc=ODD) == INVALID
    assert call(ln=ctypes.c_void_p((1 << 20) + 4)) == INVALID
    for s in BAD_STRIDES:
        assert call(sq=_strides(*s)) == INVALID, s


def test_decode_refusals(lib):
    def call(kc=FAKE, pos=FAKE, q=FAKE, y=FAKE, **kw):
        a = dict(SIZES, **kw)
        return lib.based_swa_sink_decode(kc, FAKE, pos, q, FAKE, FAKE, y, a["B"], a["Hq"], a["Hkv"], a["d"], a["w"],
                                         a["s"], a["scale"], a["dt"], None)

    for kw, want in BAD_SIZES:
        assert call(**kw) == want, kw
    for kw in (dict(kc=None), dict(pos=None), dict(q=ODD), dict(y=None), dict(pos=ctypes.c_void_p((1 << 20) + 4))):
        assert call(**kw) == INVALID, kw


def test_backward_refusals(lib):
    need = lib.based_swa_sink_backward_workspace(2, 4, 2, 16, 64, 8, 4, 1)
    assert need > 0

    def call(q=FAKE, sdq=None, lse=FAKE, dq=FAKE, ws=FAKE, n=need, **kw):
        a = dict(SIZES, **kw)
        return lib.based_swa_sink_backward(q, None, FAKE, None, FAKE, None, FAKE, None, lse, FAKE, None, dq, sdq, FAKE,
                                           None, FAKE, None, None, a["B"], a["Hq"], a["Hkv"], a["N"], a["d"], a["w"],
                                           a["s"], a["scale"], a["dt"], ws, n, None)

    for kw, want in BAD_SIZES + [(dict(N=0), INVALID)]:
        assert call(**kw) == want, kw
        if "scale" not in kw:
            a = dict(SIZES, **kw)
            assert lib.based_swa_sink_backward_workspace(a["B"], a["Hq"], a["Hkv"], a["N"], a["d"], a["w"], a["s"],
                                                         a["dt"]) == 0
    for kw in (dict(q=None), dict(lse=None), dict(dq=ODD), dict(ws=None), dict(ws=ODD), dict(n=need - 1)):
        assert call(**kw) == INVALID, kw
    for s in BAD_STRIDES:
        assert call(sdq=_strides(*s)) == INVALID, s


ROPE = dict(mp=32, B=2, Hq=4, Hkv=2, N=16, d=64, rot=32, eps=1e-6, dt=1, psb=16)
BAD_ROPE = [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(N=-1), INVALID), (dict(rot=-16), INVALID), (dict(rot=80), INVALID),
    (dict(mp=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(dt=9), INVALID),
    (dict(psb=15), INVALID), (dict(psb=-16), INVALID), (dict(d=72), UNSUPPORTED), (dict(d=272), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED),
]


def test_norm_rope_refusals(lib):
    def call(q=FAKE, so=None, wq=None, table=FAKE, pos=FAKE, **kw):
        a = dict(ROPE, **kw)
        return lib.based_qk_norm_rope(q, None, FAKE, None, FAKE, so, FAKE, None, wq, None, table, a["mp"], pos, a["psb"],
                                      a["B"], a["Hq"], a["Hkv"], a["N"], a["d"], a["rot"], 0, a["eps"], a["dt"], None)

    for kw, want in BAD_ROPE:
        assert call(**kw) == want, kw
    for kw in (dict(q=None), dict(wq=ODD), dict(table=None), dict(table=ODD), dict(pos=ctypes.c_void_p(4))):
        assert call(**kw) == INVALID, kw
    for s in BAD_STRIDES:
        assert call(so=_strides(*s)) == INVALID, s

    def back(dq=FAKE, dqw=None, ws=None, n=0, **kw):
        a = dict(ROPE, **kw)
        return lib.based_qk_norm_rope_backward(FAKE, None, FAKE, None, FAKE, None, FAKE, None, dq, None, FAKE, None, dqw,
                                               None, None, None, FAKE, a["mp"], FAKE, a["psb"], a["B"], a["Hq"],
                                               a["Hkv"], a["N"], a["d"], a["rot"], 0, a["eps"], a["dt"], ws, n, None)

    for kw, want in BAD_ROPE:
        assert back(**kw) == want, kw
    assert back(dq=None) == INVALID and back(dqw=ODD) == INVALID


def test_rope_table_refusals(lib):
    f = lib.based_rope_table
    assert f(None, 8, 16, 1e4, None) == INVALID and f(FAKE, 0, 16, 1e4, None) == INVALID
    assert f(FAKE, 8, 0, 1e4, None) == INVALID and f(FAKE, 8, 16, -1.0, None) == INVALID
    assert f(FAKE, 8, 16, float("inf"), None) == INVALID
    assert f(FAKE, 8, 24, 1e4, None) == UNSUPPORTED and f(FAKE, 8, 512, 1e4, None) == UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 3, 8, 64)
    with pytest.raises(based.BasedError):
        based.swa_sink_prefill(q, q, q, 4, 0)                  # host tensors
    with pytest.raises(based.BasedError):
        based.swa_sink_prefill(q, k, k, 4, 0)                  # 4 heads over 3
    for w, sinks in ((0, 0), (-1, 0), (4, -1), (4, 65), ((1 << 32) + 4, 0)):
        with pytest.raises(based.BasedError):
            binding._window(w, sinks)
    with pytest.raises(based.BasedError):
        based.swa_sink_decode(q, q, None, q[:, :, 0], k[:, :, 0], k[:, :, 0], 4)
    with pytest.raises(based.BasedError):
        based.qk_norm_rope(q, q)
    with pytest.raises(based.BasedError):
        based.rope_table(0, 16)
