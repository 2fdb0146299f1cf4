"""Rows that see a NaN score: O and LSE are NaN, not those of a row that sees nothing, and so are the gradients."""
import math

import pytest
import torch

from attention_attn_fwd_11_b200 import fa

pytestmark = pytest.mark.gpu

S, KEY = 200, 100


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128), (192, 192), (256, 256), (320, 256)])
@pytest.mark.parametrize("mods", [{}, dict(softcap=20.0), "mask", "sinks"])
def test_rows(dk, dv, mods):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn((1, 2, S, d), generator=g, device="cuda").bfloat16() for d in (dk, dk, dv, dv))
    kw = dict(causal=True)
    if mods == "mask":
        kw["mask"] = torch.zeros((1, 1, S, S), device="cuda", dtype=torch.float16)
    elif mods == "sinks":
        kw["sinks"] = torch.zeros(2, device="cuda")
    else:
        kw.update(mods)
    k[:, :, KEY, 3] = math.nan
    o, lse = fa.fwd(q, k, v, **kw)
    for t in (o, lse):
        assert bool(torch.isnan(t[:, :, KEY:]).all()) and bool(torch.isfinite(t[:, :, :KEY]).all())
    q2 = q.clone()
    q2[:, :, 7] = math.nan  # every score of the row
    o2, lse2 = fa.fwd(q2, k, v, **kw)
    assert bool(torch.isnan(o2[:, :, 7]).all()) and bool(torch.isnan(lse2[:, :, 7]).all())
    if (dk, dv) in ((64, 64), (128, 128), (192, 128)):
        dq, gk, gv = fa.bwd(q, k, v, o, lse, do, **kw)[:3]
        assert bool(torch.isnan(dq[:, :, KEY:]).all()) and bool(torch.isnan(gk).all()) and bool(torch.isnan(gv).all())
