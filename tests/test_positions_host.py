"""Shapes of position tensors that are refused."""
import pytest
import torch

from attention_attn_fwd_11_b200 import fa


@pytest.mark.parametrize("pos", [torch.tensor(3, dtype=torch.int32), torch.zeros(4), torch.zeros(3, dtype=torch.int32),
                                 torch.zeros((3, 4), dtype=torch.int32), torch.zeros((2, 8), dtype=torch.int32)[:, ::2],
                                 torch.zeros((1, 1, 4), dtype=torch.int32)])
def test_refused(pos):
    with pytest.raises(ValueError, match="pos must be"):
        fa._check_pos(pos, 2, 4)


def test_pitch():
    x = torch.zeros((2, 9), dtype=torch.int32)
    assert fa._check_pos(x[:, :4], 2, 4) == 9 and fa._check_pos(x[:1, :4], 2, 4) == 0 and fa._check_pos(x[0, :4], 2, 4) == 0
    assert fa._check_pos(x[:1, :4].expand(2, 4), 2, 4) == 0 and fa._check_pos(x[:, :1], 2, 1) == 9
