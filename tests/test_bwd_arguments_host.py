"""fa.bwd: arguments that are refused before the library is asked."""
import pytest
import torch

from attention_attn_fwd_11_b200 import fa


def test_without_log_sum_exp(monkeypatch):
    monkeypatch.setattr(fa, "_need_current_device", lambda *a: None)
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="log-sum-exp"):
        fa.bwd(x, x, x, x, None, x)
