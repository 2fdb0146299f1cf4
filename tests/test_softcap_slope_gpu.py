"""The softcap's derivative where it is nearly flat: softcap (1 - tanh^2 z) down to 1e-6 of the softcap, as accurate as
elsewhere.  q = 1 / (e^2z + 1) is off by 8 roundings, 5e-7 of itself, and by its argument's error: |z| below 7.5 with 2^-22
of it (the scores' fp32 sums and two products), 4e-6 in 2z; so 4 (q - q^2) by 1e-5 of itself, wherever it is above 1e-6.
Otherwise the bounds of test_bwd_gpu."""
import math

import pytest
import torch

from attention_attn_fwd_11_b200 import fa
from test_bwd_gpu import forward, inputs, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
def test_saturated(dk, dv):
    softcap = 2.0
    q, k, v, do = inputs(1, 2, 2, 150, 180, dk, dv, 3)
    z = q.double() @ k.double().transpose(-1, -2)
    kw = dict(scale=7.0 / float(z.abs().max()), causal=False, mask=None, max_bias=0.0, softcap=softcap)
    o, lse = forward(q.double(), k.double(), v.double(), **kw)
    o, lse = o.float(), lse.float()
    ref = reference(q, k, v, o, lse, do, **kw)
    s = torch.tanh(z * kw["scale"])
    assert float((1 - s * s).min()) < 1e-5
    got = fa.bwd(q, k, v, o, lse, do, grad_dtype=torch.float32, **kw)
    # the same sums with the bound of a relative error alone
    p = torch.exp(softcap * s - lse.double()[..., None])
    t = do.double() @ v.double().transpose(-1, -2) - (do.double() * o.double()).sum(-1, keepdim=True)
    ds = (p * t * softcap * (1 - s * s)).abs()
    M = do.double().abs() @ v.double().abs().transpose(-1, -2) + (do.double().abs() * o.double().abs()).sum(-1, keepdim=True)
    E = (2.0 ** -8 + 2e-4 + 1e-5) * ds + 8e-6 * p * M * softcap * (1 - s * s)
    for g, name, bound in ((got[0], "dq", kw["scale"] * E @ k.double().abs()), (got[1], "dk", kw["scale"] * E.transpose(-1, -2) @ q.double().abs())):
        r = ref[name][0]
        assert float(((g.double() - r).abs() - bound - 2.0 ** -24 * (r.abs() + bound)).max()) <= 0, name


def test_one_saturated_pair():
    """A single query on a few keys, one far into saturation: the others' gradients cannot cover its own."""
    d, softcap = 64, 2.0
    q = torch.zeros((1, 1, 1, d), device="cuda", dtype=torch.bfloat16)
    k, v, do = (torch.zeros((1, 1, n, d), device="cuda", dtype=torch.bfloat16) for n in (3, 3, 1))
    q[..., 0] = 1.0
    k[0, 0, :, 0] = torch.tensor([6.5, -6.5, 0.5], device="cuda")
    k[0, 0, :, 1] = 1.0
    v[0, 0, :, 0] = torch.tensor([1.0, -2.0, 3.0], device="cuda")
    do[..., 0] = 1.0
    kw = dict(scale=1.0, causal=False, mask=None, max_bias=0.0, softcap=softcap)
    o, lse = forward(q.double(), k.double(), v.double(), **kw)
    o, lse = o.float(), lse.float()
    r = reference(q, k, v, o, lse, do, **kw)["dk"][0][0, 0, :, 0]
    g = fa.bwd(q, k, v, o, lse, do, grad_dtype=torch.float32, **kw)[1][0, 0, :, 0]
    # dS rounds once to bf16; t is of order one here, so 8e-6 M / |t| is below 1e-4
    assert bool(((g.double() - r).abs() <= (2.0 ** -8 + 5e-4) * r.abs()).all()), (g, r)
