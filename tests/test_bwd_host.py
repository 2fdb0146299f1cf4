"""fa_bwd: what is refused before any CUDA call, and the workspace size."""
import ctypes
import math

import pytest
import torch

from attention_attn_fwd_11_b200 import fa


def params(**kw):
    p = fa.BwdParams()
    base = dict(q=16, k=32, v=48, o=64, dout=80, lse=96, gq=112, gk=128, gv=144, B=1, Hq=2, Hkv=2, Sq=128, Sk=128,
                dk=128, dv=128, scale=0.088, causal=1, o_dtype=0, g_dtype=1, workspace=256, workspace_bytes=1 << 20)
    for t in ("q", "k", "v", "o", "do", "gq", "gk", "gv"):
        base.update({t + "_sb": 2 * 128 * 128, t + "_sh": 128 * 128, t + "_ss": 128})
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(dk=96, dv=96), fa.FA_ERR_UNSUPPORTED), (dict(dk=256, dv=256), fa.FA_ERR_UNSUPPORTED),
    (dict(dk=128, dv=64), fa.FA_ERR_UNSUPPORTED), (dict(Hq=3), fa.FA_ERR_INVALID_ARG),
    (dict(B=-1), fa.FA_ERR_INVALID_ARG), (dict(Sk=-1), fa.FA_ERR_INVALID_ARG), (dict(scale=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=math.inf), fa.FA_ERR_INVALID_ARG), (dict(o_dtype=3), fa.FA_ERR_INVALID_ARG),
    (dict(g_dtype=3), fa.FA_ERR_INVALID_ARG), (dict(softcap=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(max_bias=math.nan), fa.FA_ERR_INVALID_ARG), (dict(gsinks=16), fa.FA_ERR_INVALID_ARG),
    (dict(q=0), fa.FA_ERR_INVALID_ARG), (dict(k=0), fa.FA_ERR_INVALID_ARG), (dict(lse=0), fa.FA_ERR_INVALID_ARG),
    (dict(lse=98), fa.FA_ERR_INVALID_ARG), (dict(dlse=98), fa.FA_ERR_INVALID_ARG), (dict(o=0), fa.FA_ERR_INVALID_ARG),
    (dict(dout=88), fa.FA_ERR_INVALID_ARG), (dict(o_ss=130), fa.FA_ERR_INVALID_ARG), (dict(gq=0), fa.FA_ERR_INVALID_ARG),
    (dict(gk_ss=124), fa.FA_ERR_INVALID_ARG), (dict(gv_ss=64), fa.FA_ERR_INVALID_ARG),
    (dict(gq_sh=4), fa.FA_ERR_INVALID_ARG), (dict(mask=16, m_ss=120), fa.FA_ERR_INVALID_ARG),
    (dict(mask=8, m_ss=128), fa.FA_ERR_INVALID_ARG), (dict(mask=16, m_ss=132), fa.FA_ERR_INVALID_ARG),
    (dict(workspace=0), fa.FA_ERR_WORKSPACE), (dict(workspace=128), fa.FA_ERR_WORKSPACE),
    (dict(workspace_bytes=2047), fa.FA_ERR_WORKSPACE), (dict(Sq=(1 << 30) + 1), fa.FA_ERR_INVALID_ARG),
    (dict(B=1 << 24, Hq=64, Hkv=64), fa.FA_ERR_INVALID_ARG), (dict(B=0), fa.FA_OK),
    (dict(Sq=0, Sk=0, workspace=0), fa.FA_OK)])
def test_refused(kw, status):
    assert fa.load().fa_bwd(ctypes.byref(params(**kw)), None) == status


def test_workspace_size():
    n = ctypes.c_size_t(0)
    for B, Hq, Sq, rows in ((1, 2, 128, 128), (3, 4, 129, 256), (2, 2, 1, 128), (1, 2, 0, 0)):
        p = params(B=B, Hq=Hq, Hkv=2, Sq=Sq)
        assert fa.load().fa_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == fa.FA_OK
        assert n.value >= 2 * B * Hq * rows * 4
    assert fa.load().fa_bwd_workspace_size(ctypes.byref(params(dk=80)), ctypes.byref(n)) == fa.FA_ERR_UNSUPPORTED
    assert fa.load().fa_bwd_workspace_size(ctypes.byref(params()), None) == fa.FA_ERR_INVALID_ARG


def test_cpu_tensors_are_refused():
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.bwd(x, x, x, x, torch.zeros(1, 1, 2), x)


# Outputs that would overwrite themselves, each other or an input.
@pytest.mark.parametrize("kw", [
    dict(gk_sh=0), dict(gq_sb=0, B=2), dict(gv_ss=128, gv_sh=128), dict(gq_ss=128, gq_sh=64 * 128),
    dict(gq=16), dict(gk=32), dict(gk=112), dict(gv=128), dict(gv=80), dict(gq=64)])
def test_overlapping_gradients_are_refused(kw):
    assert fa.load().fa_bwd(ctypes.byref(params(**kw)), None) == fa.FA_ERR_INVALID_ARG
    assert b"overlap" in fa.load().fa_last_error() or b"apart" in fa.load().fa_last_error()


# A stride that no second element uses may be anything: what stops these calls
# is the check that comes after (the workspace).
@pytest.mark.parametrize("kw", [
    dict(gq_sb=3, gk_sb=0, gv_sb=-1, o_sb=5), dict(Sq=1, gq_ss=1, o_ss=1), dict(Hq=1, Hkv=1, gq_sh=0, gk_sh=7, o_sh=3),
    dict(gq_ss=2 * 128, gq_sh=128), dict(gk_ss=3 * 256, gk_sh=128, gv_ss=3 * 256, gv_sh=128)])
def test_layouts_of_gradients(kw):
    assert fa.load().fa_bwd(ctypes.byref(params(workspace=0, **kw)), None) == fa.FA_ERR_WORKSPACE
