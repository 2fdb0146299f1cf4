"""fa.bwd with views of one buffer, beside one another or not."""
import pytest
import torch

from attention_attn_fwd_11_b200 import fa

pytestmark = pytest.mark.gpu


def test_gradients_beside_their_inputs_in_one_buffer():
    B, S, Hq, Hkv, d = 2, 150, 4, 2, 128
    H = Hq + 2 * Hkv
    g = torch.Generator(device="cuda").manual_seed(1)
    buf = torch.full((B, S, 2 * H + 1, d), 7.0, device="cuda", dtype=torch.bfloat16)
    buf[:, :, :H] = torch.randn((B, S, H, d), generator=g, device="cuda")
    q, k, v, dq, dk, dv, rest = (t.transpose(1, 2) for t in buf.split((Hq, Hkv, Hkv, Hq, Hkv, Hkv, 1), 2))
    do = torch.randn((B, Hq, S, d), generator=g, device="cuda").bfloat16()
    o, lse = fa.fwd(q, k, v, causal=True)
    before = buf[:, :, :H].clone()
    want = fa.bwd(q, k, v, o, lse, do, causal=True)
    got = fa.bwd(q, k, v, o, lse, do, causal=True, dq=dq, dk=dk, dv=dv)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(buf[:, :, :H], before) and bool((rest == 7.0).all())
    for kw in (dict(dq=buf[:, :, 1:1 + Hq].transpose(1, 2)), dict(dk=dv, dv=dv), dict(dk=buf[:, :, H + 1:H + 3].transpose(1, 2), dq=dq),
               dict(workspace=buf.view(-1).view(torch.uint8)), dict(dv=o.view(torch.bfloat16)[..., :d][:, :Hkv])):
        with pytest.raises(fa.FAError):
            fa.bwd(q, k, v, o, lse, do, causal=True, **kw)
    torch.cuda.synchronize()
    assert torch.equal(buf[:, :, :H], before) and fa.device_error() == 0
