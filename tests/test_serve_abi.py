"""Refusals of the serving operators: every argument error comes back before any launch (fake pointers, no GPU)."""
import ctypes

import pytest
import torch

from mxfp4_microscaled_quantization_b200 import build as build_mod
from mxfp4_microscaled_quantization_b200 import mxattn as mx

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 1 << 20
F = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return mx.lib()


def _strides(values):
    return None if values is None else (ctypes.c_int64 * len(values))(*values)


def test_prompt_refusals(L):
    base = dict(q=FAKE, k=FAKE, v=FAKE, dt=0, qo=FAKE, ko=FAKE, B=2, tq=10, tk=10, Hq=8, Hkv=2, d=64, st=None, causal=1,
                o=FAKE, lse=FAKE, ls=10, ws=FAKE, wb=256)

    def call(**kw):
        a = {**base, **kw}
        return L.mxattn_prompt(a["q"], a["k"], a["v"], a["dt"], a["qo"], a["ko"], a["B"], a["tq"], a["tk"], a["Hq"],
                               a["Hkv"], a["d"], _strides(a["st"]), a["causal"], F(0), a["o"], a["lse"], a["ls"], a["ws"],
                               a["wb"], None)
    assert L.mxattn_prompt_workspace_size(2047, 128) == 256 and L.mxattn_prompt_workspace_size(0, 64) == 256
    assert 256 < L.mxattn_prompt_workspace_size(2048, 64) < L.mxattn_prompt_workspace_size(1 << 30, 128) < 1 << 26
    assert L.mxattn_prompt_workspace_size(100, 96) == 0 and L.mxattn_prompt_workspace_size(-1, 64) == 0
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(qo=None), dict(ko=None), dict(ws=None),
               dict(dt=2), dict(dt=-1), dict(B=-1), dict(Hq=7), dict(Hq=0), dict(Hkv=0), dict(tq=-1), dict(tk=-1),
               dict(causal=2), dict(wb=255), dict(ws=FAKE + 16), dict(q=FAKE + 8), dict(k=FAKE + 8), dict(v=FAKE + 2),
               dict(o=FAKE + 8), dict(ls=9), dict(lse=FAKE + 2), dict(qo=FAKE + 2),
               dict(st=[512, 64, 128, 64, 128, 64, 512, 60]), dict(st=[512, 64, 128, 32, 128, 64, 512, 64]),
               dict(st=[508, 64, 128, 64, 128, 64, 512, 64]), dict(st=[-512, 64, 128, 64, 128, 64, 512, 64])):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=96), dict(d=256), dict(tq=(1 << 30) + 1, ls=1 << 40), dict(tk=(1 << 30) + 1), dict(Hq=65536, Hkv=1)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(B=0, q=None, k=None, v=None, o=None, qo=None, ko=None) == OK     # nothing to do
    assert call(tq=0, q=None, o=None) == OK


def test_store_refusals(L):
    base = dict(k=FAKE, v=FAKE, dt=0, n=4, of=FAKE, held=FAKE, B=4, Hkv=2, d=64, st=None, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE,
                pages=9, page=16, tab=FAKE, ts=3, most=3, status=None)

    def call(**kw):
        a = {**base, **kw}
        return L.mxattn_cache_store(a["k"], a["v"], a["dt"], a["n"], a["of"], a["held"], a["B"], a["Hkv"], a["d"],
                                    _strides(a["st"]), a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["page"], a["tab"],
                                    a["ts"], a["most"], a["status"], None)
    for kw in (dict(k=None), dict(v=None), dict(of=None), dict(held=None), dict(kc=None), dict(vc=None), dict(ks=None),
               dict(vs=None), dict(tab=None), dict(dt=5), dict(n=-1), dict(B=-1), dict(Hkv=0), dict(pages=-1),
               dict(most=-1), dict(ts=2), dict(k=FAKE + 8), dict(kc=FAKE + 8), dict(vc=FAKE + 4), dict(held=FAKE + 1),
               dict(status=FAKE + 2), dict(st=[128, 64, 128, 63]), dict(st=[128, 64, 32, 64])):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=32), dict(page=8), dict(page=48), dict(page=256), dict(n=(1 << 30) + 1), dict(most=1 << 27, ts=1 << 27)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(n=0, k=None, v=None) == OK
    assert call(B=0, of=None, held=None) == OK


def test_attend_refusals(L):
    need = L.mxattn_cache_attend_workspace_size(8, 2, 64)
    assert need >= 256
    for bad in ((7, 2, 64), (8, 0, 64), (0, 1, 64), (8, 2, 96)):
        assert L.mxattn_cache_attend_workspace_size(*bad) == 0
    base = dict(q=FAKE, dt=1, B=3, Hq=8, Hkv=2, d=64, st=None, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pages=9, page=16,
                tab=FAKE, ts=3, most=3, lens=FAKE, o=FAKE, lse=FAKE, ws=FAKE, wb=need)

    def call(**kw):
        a = {**base, **kw}
        return L.mxattn_cache_attend(a["q"], a["dt"], a["B"], a["Hq"], a["Hkv"], a["d"], _strides(a["st"]), a["kc"], a["vc"],
                                     a["ks"], a["vs"], a["pages"], a["page"], a["tab"], a["ts"], a["most"], a["lens"], F(0),
                                     a["o"], a["lse"], a["ws"], a["wb"], None)
    for kw in (dict(q=None), dict(o=None), dict(lens=None), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None),
               dict(tab=None), dict(ws=None), dict(wb=need - 1), dict(ws=FAKE + 128), dict(dt=3), dict(B=-2), dict(Hq=9),
               dict(pages=-1), dict(most=-1), dict(ts=2), dict(q=FAKE + 8), dict(o=FAKE + 8), dict(kc=FAKE + 8),
               dict(lse=FAKE + 1), dict(st=[512, 64, 512, 8]), dict(st=[512, 68, 512, 64])):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=192, wb=1 << 40), dict(page=12), dict(most=1 << 27, ts=1 << 27)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(B=0, q=None, o=None, lens=None) == OK


def test_bindings_refuse_what_is_not_on_the_gpu():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mx.mxattn_prompt(x, x, x, i)
    with pytest.raises(ValueError, match="CUDA"):
        mx.mxattn_cache_attend(x, *mx.new_cache(2, 2, 16, 64, device="cpu"), i.view(1, 3), i)
    with pytest.raises(ValueError, match="CUDA"):
        mx.mxattn_cache_store(x, x, *mx.new_cache(2, 2, 16, 64, device="cpu"), i.view(1, 3), i, i)
