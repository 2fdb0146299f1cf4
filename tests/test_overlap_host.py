"""Whether strided rows share memory (csrc/overlap.h) against brute force, and the calls that are refused for it."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from attention_attn_fwd_11_b200 import fa

HEADER = os.path.join(os.path.dirname(os.path.abspath(fa.__file__)), "csrc", "overlap.h")


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("overlap")
    (d / "o.cpp").write_text('''#include "%s"
static fa::Rows rows(const long *x) {
    return fa::Rows{(const void *)x[0], x[1], {x[2], x[3], x[4]}, {x[5], x[6], x[7]}};
}
extern "C" int meet(const long *a, const long *b) { return fa::rows_meet(rows(a), rows(b)); }
extern "C" int self(const long *a) { return fa::rows_meet_themselves(rows(a)); }
''' % HEADER)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-o", str(d / "o.so"), str(d / "o.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "o.so"))
    arr = lambda x: (ctypes.c_long * 8)(*x)  # noqa: E731
    return (lambda a, b: bool(lib.meet(arr(a), arr(b)))), (lambda a: bool(lib.self(arr(a))))


def starts(x):
    p, _, n0, n1, n2, s0, s1, s2 = x
    return np.array([p + i * s0 + j * s1 + k * s2 for i in range(n0) for j in range(n1) for k in range(n2)])


def test_against_brute_force(overlap):
    meet, self_ = overlap
    rng = np.random.default_rng(1)
    seen = [0, 0, 0, 0]
    for _ in range(4000):
        make = lambda: [1 << 20] + [int(rng.integers(1, 5))] + [int(rng.integers(1, 5)) for _ in range(3)] + [  # noqa: E731
            int(rng.choice([0, 1, 2, 3, 4, 5, 7, 8, 12, 16, 20, 40, 60, -4, -6, -16, -33])) for _ in range(3)]
        a, b = make(), make()
        b[0] += int(rng.integers(-120, 120))
        if rng.random() < 0.5:
            b[5:] = a[5:]
        x, y = starts(a), starts(b)
        d = y[None] - x[:, None]
        want = bool(((d < a[1]) & (d > -b[1])).any())
        assert meet(a, b) == want and meet(b, a) == want, (a, b)
        e = np.abs(x[None] - x[:, None])[~np.eye(len(x), dtype=bool)]
        own = bool((e < a[1]).any())
        assert self_(a) == own, a
        seen[want] += 1
        seen[2 + own] += 1
    assert min(seen) > 300


def test_large_layouts(overlap):
    """Projections side by side in one buffer are apart; one row or one head too many and they are not."""
    meet, self_ = overlap
    S, d = 1 << 20, 256
    for pitch in (d * 48, d * 48 + 32):
        q = [1 << 30, d, 7, 32, S, pitch * S, d, pitch]
        k = [(1 << 30) + 32 * d, d, 7, 8, S, pitch * S, d, pitch]
        assert not meet(q, k) and not meet(k, q) and not self_(q)
        assert meet([q[0], d, 7, 33, S, pitch * S, d, pitch], k)
        assert meet(q, [k[0] - 16, *k[1:]])
        assert not meet(q, [k[0] + 7 * pitch * S, *k[1:]])  # behind q
        assert self_([q[0], d + 32, *q[2:]]) and self_([q[0], d, 7, 50, S, pitch * S, d, pitch])
    assert self_([0, 256, 2, 4, 100, 0, 25600, 256]) and not self_([0, 256, 1, 4, 100, 0, 25600, 256])
    assert not self_([0, 256, 2, 4, 100, -102400, 25600, 256])


INV = (ctypes.c_double * 64)(*([0.5] * 64))
MB = 1 << 20


def rope(**kw):
    base = dict(q=MB, q_out=2 * MB, k=3 * MB, k_out=4 * MB, B=2, Hq=4, Hk=2, S=8, d=128, dtype=fa.FA_BF16,
                inv_freq=ctypes.addressof(INV), rot_dim=128, mscale=1.0)
    for t, h in (("q", 4), ("qo", 4), ("k", 2), ("ko", 2)):
        base.update({t + "_sb": h * 1024, t + "_sh": 1024, t + "_ss": 128})
    p = fa.RopeParams()
    for n, v in {**base, **kw}.items():
        setattr(p, n, v)
    return fa.load().fa_rope(ctypes.byref(p), None), fa.load().fa_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(k_out=2 * MB), dict(q_out=3 * MB), dict(k_out=MB), dict(k_out=2 * MB + 2048), dict(k_out=2 * MB - 256),
    dict(q_out=MB + 256), dict(q_out=MB - 16), dict(k_out=3 * MB + 4096), dict(qo_sh=64), dict(qo_sh=-64), dict(ko_sh=120),
    dict(qo_sb=128), dict(ko_ss=1024, ko_sh=1024), dict(qo_sb=1024), dict(dtype=fa.FA_F32, qo_sh=64),
    dict(dtype=fa.FA_F32, k_out=2 * MB + 16384 - 256)])
def test_rotary_outputs_that_share_memory_are_refused(kw):
    status, message = rope(**kw)
    assert status == fa.FA_ERR_INVALID_ARG and ("overlap" in message or "apart" in message), message


def append(**kw):
    base = dict(k=MB, v=2 * MB, k_cache=16 * MB, v_cache=32 * MB, block_table=64, seq_lens=64, max_blocks_per_seq=4, B=2,
                Hkv=2, Sq=8, dk=128, dv=128, block_size=64, num_blocks=8, inv_freq=ctypes.addressof(INV), rot_dim=128,
                mscale=1.0, q=3 * MB, q_out=4 * MB, Hq=4)
    for t, h in (("q", 4), ("qo", 4), ("k", 2), ("v", 2)):
        base.update({t + "_sb": h * 1024, t + "_sh": 1024, t + "_ss": 128})
    p = fa.KvAppendParams()
    for n, v in {**base, **kw}.items():
        setattr(p, n, v)
    return fa.load().fa_kv_append(ctypes.byref(p), None), fa.load().fa_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(q_out=MB), dict(q_out=2 * MB), dict(q_out=MB + 4096), dict(q_out=2 * MB - 512), dict(q_out=3 * MB + 256),
    dict(qo_sh=64), dict(q_out=16 * MB + 1024), dict(q_out=32 * MB - 256), dict(v_cache=16 * MB),
    dict(v_cache=16 * MB + 8 * 2 * 64 * 256 - 256),
    dict(kv_type=fa.FA_KV_Q4_0, v_cache=16 * MB - 8 * 2 * 64 * 72 + 16)])
def test_appended_outputs_that_share_memory_are_refused(kw):
    status, message = append(**kw)
    assert status == fa.FA_ERR_INVALID_ARG and ("overlap" in message or "apart" in message), message
