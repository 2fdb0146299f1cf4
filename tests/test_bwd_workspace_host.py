"""How much memory the backward asks for: no GPU needed."""
import ctypes
import random

import pytest

from attention_attn_fwd_11_b200 import fa


def sizes(B, Hq, Hkv, Sq, Sk, dk=128, dv=128):
    """(causal or not, not causal, causal)"""
    p = fa.BwdParams(B=B, Hq=Hq, Hkv=Hkv, Sq=Sq, Sk=Sk, dk=dk, dv=dv, scale=1.0)
    n = ctypes.c_size_t(0)
    got = []
    for f, causal in (("size", 0), ("need", 0), ("need", 1)):
        p.causal = causal
        assert getattr(fa.load(), "fa_bwd_workspace_" + f)(ctypes.byref(p), ctypes.byref(n)) == fa.FA_OK
        got.append(n.value)
    assert got[0] == max(got)
    return got


def rows(B, Hq, Sq):  # LSE, D and their bf16 pieces, and the counter
    return 6 * ((4 * B * Hq * ((Sq + 383) // 384 * 384) + 255) // 256 * 256) + 256


MB = 1 << 20


@pytest.mark.parametrize("Hq,Hkv,Sq,Sk,causal_mb", [(32, 8, 65536, 512, 48), (32, 8, 8192, 512, 48), (8, 1, 131072, 64, 32)])
def test_many_queries_that_see_nothing(Hq, Hkv, Sq, Sk, causal_mb):
    """Under the causal rule only the last Sk queries see a key: the others get no parts."""
    _, full, causal = sizes(1, Hq, Hkv, Sq, Sk)
    assert causal - rows(1, Hq, Sq) <= causal_mb * MB and full - rows(1, Hq, Sq) <= 16 * MB


def test_parts_stay_below_the_gradients():
    rng = random.Random(3)
    cases = [(4, 128, 1, 131072, 4096), (2, 512, 16, 4016, 382), (3, 256, 8, 2615, 459), (1, 512, 16, 3612, 803)]
    for _ in range(3000):
        log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
        Hkv = 1 << rng.randrange(6)
        Sq = log(1, 200000)
        cases.append((rng.randrange(1, 5), Hkv << rng.randrange(6), Hkv, Sq, Sq if rng.random() < 0.5 else log(1, 200000)))
    for B, Hq, Hkv, Sq, Sk in cases:
        for dk, dv in ((64, 64), (128, 128), (192, 128)):
            gradients = 4 * B * (Hq * Sq * dk + Hkv * Sk * (dk + dv))
            if B * Hq * Sq < 1 << 28:
                assert sizes(B, Hq, Hkv, Sq, Sk, dk, dv)[0] <= rows(B, Hq, Sq) + max(256_000_000, gradients), (B, Hq, Hkv, Sq, Sk, dk)


def test_a_smaller_shape_can_need_more_and_a_short_workspace_is_refused():
    small, large = sizes(2, 8, 8, 16, 4096), sizes(4, 8, 8, 16, 4096)
    assert small[1] > large[1]
    p = fa.BwdParams(B=2, Hq=8, Hkv=8, Sq=16, Sk=4096, dk=128, dv=128, scale=0.1, workspace=1 << 40, workspace_bytes=large[0])
    for i, (n, h, s) in enumerate((("q", 8, 16), ("k", 8, 4096), ("v", 8, 4096), ("o", 8, 16), ("do", 8, 16), ("gq", 8, 16), ("gk", 8, 4096), ("gv", 8, 4096))):
        setattr(p, "dout" if n == "do" else n, (i + 1) << 30)
        for e, v in (("_sb", h * s * 128), ("_sh", s * 128), ("_ss", 128)):
            setattr(p, n + e, v)
    p.lse = 1 << 36
    assert fa.load().fa_bwd(ctypes.byref(p), None) == fa.FA_ERR_WORKSPACE


def test_null():
    p = fa.BwdParams(B=1, Hq=1, Hkv=1, Sq=1, Sk=1, dk=64, dv=64, scale=1.0)
    assert fa.load().fa_bwd_workspace_need(ctypes.byref(p), None) == fa.FA_ERR_INVALID_ARG
    assert fa.load().fa_bwd_workspace_need(None, ctypes.byref(ctypes.c_size_t(0))) == fa.FA_ERR_INVALID_ARG
