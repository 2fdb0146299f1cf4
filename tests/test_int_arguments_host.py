"""Integers that a C int cannot hold are refused, not cut to their lowest 32 bits."""
import types

import pytest
import torch

from attention_attn_fwd_11_b200 import fa


@pytest.fixture
def launched(monkeypatch):
    """The parameters of the calls that reach the library, which is not there."""
    got = []
    call = lambda p, *a: got.append(p._obj) or fa.FA_OK  # noqa: E731
    monkeypatch.setattr(fa, "load", lambda: types.SimpleNamespace(fa_kv_append=call, fa_bwd_workspace_size=call))
    monkeypatch.setattr(fa, "_need_current_device", lambda *a: None)
    monkeypatch.setattr(fa, "_stream", lambda *a: None)
    return got


def append(**kw):
    x, cache = torch.zeros(1, 2, 3, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 64, 128, dtype=torch.bfloat16)
    args = dict(k=x, v=x, k_cache=cache, v_cache=cache, block_table=torch.zeros(1, 2, dtype=torch.int32),
                seq_lens=torch.zeros(1, dtype=torch.int32), inv_freq=fa.rope_frequencies(64)[0])
    fa.kv_append(**{**args, **kw})


@pytest.mark.parametrize("offset", [1 << 32, (1 << 32) + 32, -(1 << 32), 1 << 31, -(1 << 31) - 1])
def test_offset(launched, offset):
    with pytest.raises(ValueError):
        append(offset=offset)
    assert not launched


def test_what_fits(launched):
    append(offset=32, interleaved=1 << 32)
    assert launched[0].rot_offset == 32 and launched[0].interleaved == 1 and launched[0].rot_dim == 64


def test_heads_and_lengths(launched):
    big = (1 << 32) + 2
    with pytest.raises(ValueError):
        append(q=torch.zeros(128, dtype=torch.bfloat16).as_strided((1, big, 3, 128), (0, 0, 0, 1)),
               q_out=torch.zeros(128, dtype=torch.bfloat16).as_strided((1, big, 3, 128), (0, 0, 0, 1)))
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.bwd_workspace_bytes(x, x, x.expand(1, 1, big, 64))
    assert not launched
