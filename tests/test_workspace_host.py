"""A workspace tensor whose elements do not fill the bytes from its address on is refused (an expanded one has hardly any
memory behind its size)."""
import pytest
import torch

from attention_attn_fwd_11_b200 import fa

BF, I32 = torch.bfloat16, torch.int32
BAD = [torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(1 << 20, dtype=torch.uint8)[::2],
       torch.empty((64, 64), dtype=torch.float32).t()]


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("ws", BAD)
def test_refused(ws, monkeypatch):
    q, cache, table, lens = z(1, 2, 128), z(2, 2, 64, 128), z(1, 2, dtype=I32), z(1, dtype=I32)
    with pytest.raises(ValueError, match="contiguous"):
        fa.paged_params(q, cache, cache, table, lens, q, None, 1.0, 0, ws)
    with pytest.raises(ValueError, match="contiguous"):
        fa.gather_params(z(2, 128, 576), z(4, 576), z(2, 4, dtype=I32), None, None, None, None, 1.0, 0, ws)
    with pytest.raises(ValueError, match="contiguous"):
        fa.mla_tail_params(z(2, 4, 8), z(4, 6, 8), z(10, 24), z(2, 10), 0, ws)
    x = z(1, 1, 2, 64)
    monkeypatch.setattr(fa, "_need_current_device", lambda *a: None)
    with pytest.raises(ValueError, match="contiguous"):
        fa.bwd(x, x, x, x, z(1, 1, 2, dtype=torch.float32), x, workspace=ws)


def test_taken():
    ws = torch.empty((4, 128), dtype=torch.float32)[1:]
    assert fa._workspace(ws) == (ws.data_ptr(), 3 * 512) and fa._workspace(None) == (None, 0)


def test_a_workspace_or_output_on_the_cpu_is_refused():
    q, cache, table, lens = z(1, 2, 128), z(2, 2, 64, 128), z(1, 2, dtype=I32), z(1, dtype=I32)
    for kw in (dict(workspace=torch.empty(512, dtype=torch.uint8)), dict(out=q)):
        with pytest.raises(ValueError):
            fa.decode_paged(q, cache, cache, table, lens, **kw)
