"""fa_bwd: what it writes may share memory neither with itself nor with what it reads."""
import ctypes

import pytest

from attention_attn_fwd_11_b200 import fa

MB = 1 << 20
NAMES = ("q", "k", "v", "o", "dout", "lse", "gq", "gk", "gv", "dlse", "sinks", "gsinks", "mask", "workspace")
AT = {n: (i + 1) * 16 * MB for i, n in enumerate(NAMES)}  # 128 KB or less each, but for the workspace


def call(**kw):
    base = dict(AT, B=1, Hq=2, Hkv=2, Sq=128, Sk=128, dk=128, dv=128, scale=0.088, causal=1, o_dtype=0, g_dtype=1, m_ss=128,
                workspace_bytes=16 * MB)
    for t in ("q", "k", "v", "o", "do", "gq", "gk", "gv"):
        base.update({t + "_sb": 2 * 128 * 128, t + "_sh": 128 * 128, t + "_ss": 128})
    p = fa.BwdParams()
    for n, v in {**base, **kw}.items():
        setattr(p, n, v)
    return fa.load().fa_bwd(ctypes.byref(p), None), fa.load().fa_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(gq=AT["q"] + 256), dict(gk=AT["k"] - 256), dict(gv=AT["gk"] + 4096), dict(gq=AT["lse"] + 64 - 65536),
    dict(gk=AT["dlse"] + 16), dict(gv=AT["mask"] + 128), dict(gq=AT["workspace"] + 1024), dict(gsinks=AT["sinks"] + 4),
    dict(gsinks=AT["gv"] + 65532), dict(gsinks=AT["workspace"] + 2048), dict(workspace=AT["o"] + 131072 - 256),
    dict(workspace=AT["lse"] - 1024), dict(gq=AT["dout"] + 65536 - 16), dict(gq=AT["v"] + 16, g_dtype=0)])
def test_refused(kw):
    status, message = call(**kw)
    assert status == fa.FA_ERR_INVALID_ARG and "must be apart from" in message, message


# Rows [gq | gk | gv] of one buffer whose heads meet.
def test_views_of_one_buffer_that_meet():
    kw = {}
    for n, at in (("gq", 0), ("gk", 256), ("gv", 1024)):
        kw.update({n: (1 << 30) + 2 * at, n + "_ss": 768, n + "_sh": 128, n + "_sb": 768 * 128})
    kw["gk"] -= 256  # gk's first head on gq's second
    status, message = call(**kw)
    assert status == fa.FA_ERR_INVALID_ARG and "gq must be apart from gk" in message
