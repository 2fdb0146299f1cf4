"""Rotary positions and the cache append: the host side, which needs no GPU --
the frequencies, and the arguments that are refused before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

from attention_attn_fwd_11_b200 import fa


def test_frequencies_plain_and_linear():
    inv, m = fa.rope_frequencies(64, base=500.0)
    assert m == 1.0 and inv.dtype == torch.float64
    np.testing.assert_allclose(inv.numpy(), [500.0 ** (-2 * i / 64) for i in range(32)], rtol=1e-15)
    lin, m = fa.rope_frequencies(64, base=500.0, scaling="linear", factor=4.0)
    assert m == 1.0
    np.testing.assert_allclose(lin.numpy() * 4, inv.numpy(), rtol=1e-15)


def test_frequencies_ntk_slows_the_slowest_pair_by_the_factor():
    inv, _ = fa.rope_frequencies(128)
    ntk, m = fa.rope_frequencies(128, scaling="ntk", factor=8.0)
    assert m == 1.0 and ntk[0] == inv[0]
    assert math.isclose(float(inv[-1] / ntk[-1]), 8.0, rel_tol=1e-12)


def test_frequencies_yarn_by_parts():
    inv, _ = fa.rope_frequencies(128)
    y, m = fa.rope_frequencies(128, scaling="yarn", factor=16.0, original_len=4096)
    assert math.isclose(m, 0.1 * math.log(16.0) + 1.0, rel_tol=1e-15)
    turns = 4096 * inv / (2 * math.pi)
    assert torch.equal(y[turns > 40], inv[turns > 40])  # fast pairs are kept
    torch.testing.assert_close(y[turns < 0.8], inv[turns < 0.8] / 16, rtol=1e-14, atol=0)  # slow ones stretched
    assert bool(((y <= inv * (1 + 1e-14)) & (y >= inv / 16 * (1 - 1e-14))).all())


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=64, scaling="other"),
                                dict(rot_dim=64, base=1.0), dict(rot_dim=64, scaling="linear", factor=0.5),
                                dict(rot_dim=64, scaling="yarn", factor=2.0),
                                dict(rot_dim=2, scaling="ntk", factor=2.0)])
def test_frequencies_refused(kw):
    with pytest.raises(ValueError):
        fa.rope_frequencies(**kw)


INV = (ctypes.c_double * 128)(*([0.5] * 128))
NAN = (ctypes.c_double * 128)(*([0.5] * 7 + [math.nan] + [0.5] * 120))


def call(kind, name, **kw):
    p = kind()
    for k, v in kw.items():
        setattr(p, k, ctypes.addressof(v) if isinstance(v, ctypes.Array) else v)
    return getattr(fa.load(), name)(ctypes.byref(p), None)


ROPE = dict(q=16, q_out=32, q_sb=2048, q_sh=1024, q_ss=128, qo_sb=2048, qo_sh=1024, qo_ss=128, B=2, Hq=2, Hk=0, S=8,
            d=128, dtype=fa.FA_BF16, inv_freq=INV, rot_dim=128, mscale=1.0)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), fa.FA_ERR_INVALID_ARG), (dict(Hq=0), fa.FA_ERR_INVALID_ARG), (dict(d=0), fa.FA_ERR_INVALID_ARG),
    (dict(d=120), fa.FA_ERR_UNSUPPORTED), (dict(d=1040, rot_dim=64), fa.FA_ERR_UNSUPPORTED),
    (dict(rot_dim=0), fa.FA_ERR_UNSUPPORTED), (dict(rot_dim=40), fa.FA_ERR_UNSUPPORTED),
    (dict(rot_dim=144), fa.FA_ERR_UNSUPPORTED), (dict(rot_dim=64, rot_offset=80), fa.FA_ERR_UNSUPPORTED),
    (dict(rot_dim=64, rot_offset=8), fa.FA_ERR_UNSUPPORTED), (dict(rot_dim=64, rot_offset=-16), fa.FA_ERR_UNSUPPORTED),
    (dict(inv_freq=0), fa.FA_ERR_INVALID_ARG), (dict(inv_freq=NAN), fa.FA_ERR_INVALID_ARG),
    (dict(mscale=math.inf), fa.FA_ERR_INVALID_ARG), (dict(dtype=5), fa.FA_ERR_INVALID_ARG),
    (dict(q=0), fa.FA_ERR_INVALID_ARG), (dict(q_out=0), fa.FA_ERR_INVALID_ARG), (dict(q=24), fa.FA_ERR_INVALID_ARG),
    (dict(q_ss=132), fa.FA_ERR_INVALID_ARG), (dict(qo_ss=0), fa.FA_ERR_INVALID_ARG),
    (dict(qo_sh=0), fa.FA_ERR_INVALID_ARG), (dict(q_out=16, qo_ss=256), fa.FA_ERR_INVALID_ARG),
    (dict(pos=2), fa.FA_ERR_INVALID_ARG), (dict(k=16), fa.FA_ERR_INVALID_ARG), (dict(Hk=2), fa.FA_ERR_INVALID_ARG),
    (dict(pos0=(1 << 31) - 8), fa.FA_ERR_INVALID_ARG),
    (dict(B=1 << 16, S=1 << 15), fa.FA_ERR_INVALID_ARG), (dict(Hq=65536), fa.FA_ERR_INVALID_ARG),
    (dict(B=0, q=0, q_out=0), fa.FA_OK), (dict(S=0), fa.FA_OK)])
def test_rope_refused(kw, status):
    assert call(fa.RopeParams, "fa_rope", **{**ROPE, **kw}) == status


APPEND = dict(k=16, v=32, k_sb=2048, k_sh=1024, k_ss=128, v_sb=2048, v_sh=1024, v_ss=128, k_cache=48, v_cache=64,
              block_table=16, seq_lens=16, max_blocks_per_seq=4, B=2, Hkv=2, Sq=8, dk=128, dv=128, block_size=64,
              num_blocks=8, kv_type=0, inv_freq=INV, rot_dim=128, mscale=1.0)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), fa.FA_ERR_INVALID_ARG), (dict(Hkv=0), fa.FA_ERR_INVALID_ARG),
    (dict(num_blocks=0), fa.FA_ERR_INVALID_ARG), (dict(block_size=32), fa.FA_ERR_UNSUPPORTED),
    (dict(kv_type=7), fa.FA_ERR_UNSUPPORTED), (dict(dk=136), fa.FA_ERR_UNSUPPORTED),
    (dict(dk=64, rot_dim=64, kv_type=fa.FA_KV_Q8_0), fa.FA_ERR_UNSUPPORTED),
    (dict(kv_type=fa.FA_KV_FP8_E4M3), fa.FA_ERR_INVALID_ARG),
    (dict(kv_type=fa.FA_KV_FP8_E4M3, k_scale=1.0, v_scale=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(kv_type=fa.FA_KV_FP8_E4M3, k_scale=1e-40, v_scale=1.0), fa.FA_ERR_INVALID_ARG),
    (dict(kv_type=fa.FA_KV_Q8_0, rot_dim=96), fa.FA_ERR_UNSUPPORTED),
    (dict(kv_type=fa.FA_KV_Q4_0, rot_dim=48, interleaved=1), fa.FA_ERR_UNSUPPORTED),
    (dict(kv_type=fa.FA_KV_Q8_0, rot_dim=64, rot_offset=16), fa.FA_ERR_UNSUPPORTED),
    (dict(k=0), fa.FA_ERR_INVALID_ARG), (dict(v=40), fa.FA_ERR_INVALID_ARG), (dict(k_sh=1020), fa.FA_ERR_INVALID_ARG),
    (dict(k_cache=0), fa.FA_ERR_INVALID_ARG), (dict(v_cache=72), fa.FA_ERR_INVALID_ARG),
    (dict(block_table=0), fa.FA_ERR_INVALID_ARG), (dict(seq_lens=18), fa.FA_ERR_INVALID_ARG),
    (dict(q=16, q_out=32, Hq=4, inv_freq=0), fa.FA_ERR_INVALID_ARG), (dict(q=16, q_out=32, Hq=0), fa.FA_ERR_INVALID_ARG),
    (dict(q=16, Hq=4, q_ss=128, q_sh=1024, q_sb=4096), fa.FA_ERR_INVALID_ARG),
    (dict(B=1 << 20, Sq=1 << 11), fa.FA_ERR_INVALID_ARG), (dict(inv_freq=NAN), fa.FA_ERR_INVALID_ARG),
    (dict(B=0, k=0), fa.FA_OK), (dict(Sq=0), fa.FA_OK)])
def test_append_refused(kw, status):
    assert call(fa.KvAppendParams, "fa_kv_append", **{**APPEND, **kw}) == status


def test_cpu_tensors_are_refused():
    inv, _ = fa.rope_frequencies(64)
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.rope(x, inv)
    with pytest.raises(ValueError):
        fa.kv_append(x, x, x, x, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("cls,pack,n", [(fa.BwdParams, fa._pack_bwd, 45), (fa.RopeParams, fa._pack_rope, 31),
                                        (fa.KvAppendParams, fa._pack_append, 22)])
def test_packed_arguments(cls, pack, n):
    """Every field gets its value, the rest 0; what a field cannot hold is refused."""
    p = pack(*range(1, n + 1))
    for i, (name, _) in enumerate(cls._fields_):
        assert (getattr(p, name) or 0) == (i + 1 if i < n else 0), name
    ints = [i for i, (_, t) in enumerate(cls._fields_[:n]) if t is ctypes.c_int]
    for bad in (1 << 31, -(1 << 31) - 1):
        with pytest.raises(ValueError):
            pack(*[bad if i == ints[0] else 1 for i in range(n)])
    for i, (name, t) in enumerate(cls._fields_[:n]):
        if t is ctypes.c_float:  # as in C; the library refuses it
            assert getattr(pack(*[1e300 if j == i else 1 for j in range(n)]), name) == math.inf
