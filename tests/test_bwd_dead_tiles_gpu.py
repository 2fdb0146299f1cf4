"""Many queries that see no key, beside shared walks: zeros for them, and nothing written past the workspace."""
import math

import pytest
import torch

from attention_attn_fwd_11_b200 import fa
from test_bwd_gpu import check, inputs, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("Hq,Hkv,Sq,Sk", [(8, 2, 3000, 200), (4, 4, 1700, 900), (2, 1, 1285, 1), (6, 2, 700, 643), (16, 4, 2000, 512)])
def test_dead_query_tiles(dk, dv, Hq, Hkv, Sq, Sk):
    q, k, v, do = inputs(1, Hq, Hkv, Sq, Sk, dk, dv, Sq + dk)
    kw = dict(scale=1 / math.sqrt(dk), causal=True, mask=None, max_bias=0.0, softcap=0.0)
    o, lse = fa.fwd(q, k, v, **kw)
    n = fa.bwd_workspace_bytes(q, k, v, causal=True)
    room = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.full_like(t, math.nan) for t in (q, k, v)]
    got = fa.bwd(q, k, v, o, lse, do, dq=outs[0], dk=outs[1], dv=outs[2], workspace=room[:n], **kw)
    torch.cuda.synchronize()
    assert fa.device_error() == 0 and bool((room[n:] == 255).all())
    check(got, reference(q, k, v, o, lse, do, **kw))
    assert bool((got[0][:, :, :Sq - Sk] == 0).all())
    with pytest.raises(fa.FAError):
        fa.bwd(q, k, v, o, lse, do, workspace=room[:n - 256], **kw)


def test_memory_of_a_call():
    """65536 queries on 512 keys: 50 MB of rows and some parts, not gigabytes."""
    q, k, v, do = inputs(1, 32, 8, 65536, 512, 64, 64, 5)
    o, lse = fa.fwd(q, k, v, causal=True)
    for causal in (True, False):
        fa.bwd(q, k, v, o, lse, do, causal=causal)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        outs = fa.bwd(q, k, v, o, lse, do, causal=causal)
        gradients = sum(t.numel() * 2 for t in outs)
        assert torch.cuda.max_memory_allocated() - before <= gradients + 6 * 4 * 32 * 65664 + (64 << 20)
        del outs
