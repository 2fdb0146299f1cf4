"""A score that is NaN stays NaN under a softcap, in the forward and in the backward pass, and does not spread to scores of
other keys; infinite scores are capped.  One value of key 102 is NaN, so under the causal rule
queries from 102 on see it."""
import math

import pytest
import torch

from attention_attn_fwd_11_b200 import fa
from test_bwd_gpu import reference

pytestmark = pytest.mark.gpu

S, KEY = 200, 102
# Keys 100 to 103 may share one reciprocal, whose rounding (7 steps of 2^-24 of 2 / d in each of two results: below 20 *
# 2 * 14 * 2^-24 = 3.4e-5 in a score) then depends on key 102, hidden or not.  Queries 100 and 101 see two of them, so
# their LSE may move by that, and their weights, rounded to bf16 for the product with V, by a step: 2^-8 of sum P |V|,
# with |V| below 5.  The queries before have equal bits.
EXACT, D_LSE, D_O = 100, 3.4e-5, 2.0 ** -8 * 5 + 7e-5 * 5


def inputs(dk, dv, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((1, 2, S, d), generator=g, device="cuda").bfloat16() for d in (dk, dk, dv, dv)]


def keywords(dk, masked):
    mask = None
    if masked:
        mask = torch.randn((1, 1, S, S), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").half()
        mask[..., 99] = -math.inf
    return dict(causal=True, softcap=20.0, scale=1 / (20 * math.sqrt(dk)), mask=mask)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128), (192, 192), (256, 256), (320, 256)])
@pytest.mark.parametrize("masked", [False, True])
def test_forward(dk, dv, masked):
    q, k, v, _ = inputs(dk, dv)
    kw = keywords(dk, masked)
    want, lse = fa.fwd(q, k, v, **kw)
    assert bool(torch.isfinite(want).all())
    k[:, :, KEY, 3] = math.nan
    o, l = fa.fwd(q, k, v, **kw)
    assert bool(torch.isnan(o[:, :, KEY:]).all())
    assert torch.equal(o[:, :, :EXACT], want[:, :, :EXACT]) and torch.equal(l[:, :, :EXACT], lse[:, :, :EXACT])
    assert float((o - want)[:, :, EXACT:KEY].abs().max()) <= D_O and float((l - lse)[:, :, EXACT:KEY].abs().max()) <= D_LSE
    q, k, v, _ = inputs(dk, dv)
    q[:, :, KEY, 3] = math.nan
    o, _ = fa.fwd(q, k, v, **kw)
    rest = [i for i in range(S) if i != KEY]
    assert bool(torch.isnan(o[:, :, KEY]).all()) and torch.equal(o[:, :, rest], want[:, :, rest])


@pytest.mark.parametrize("masked", [False, True])
def test_paged_forward(masked):
    q, k, v, _ = inputs(128, 128)
    kw = keywords(128, masked)
    if masked:
        kw["mask"] = torch.nn.functional.pad(kw["mask"], (0, 56))
    table = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([S], dtype=torch.int32, device="cuda")

    def run(k):
        kc, vc = (torch.zeros((4, 2, 64, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        fa.kv_append(k, v, kc, vc, table, lens)
        return fa.prefill_paged(q, kc, vc, table, lens, **kw)[0]

    want = run(k)
    k[:, :, KEY, 3] = math.nan
    o = run(k)
    assert bool(torch.isnan(o[:, :, KEY:]).all()) and torch.equal(o[:, :, :EXACT], want[:, :, :EXACT])
    assert float((o - want)[:, :, EXACT:KEY].abs().max()) <= D_O


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("masked", [False, True])
def test_backward(dk, dv, masked):
    """With O and LSE of finite keys, so that what is NaN comes from the scores of the backward itself.  (Column 3 of dq
    is a sum that the NaN value enters with the factor 0.)"""
    q, k, v, do = inputs(dk, dv)
    kw = keywords(dk, masked)
    o, lse = fa.fwd(q, k, v, **kw)
    want = fa.bwd(q, k, v, o, lse, do, **kw)
    ref, lim = reference(q, k, v, o, lse, do, max_bias=0.0, **kw)["dq"]
    assert all(bool(torch.isfinite(t).all()) for t in want)
    k[:, :, KEY, 3] = math.nan
    gq, gk, gv = fa.bwd(q, k, v, o, lse, do, **kw)
    rest, cols = [i for i in range(S) if i != KEY], [i for i in range(dk) if i != 3]
    assert bool(torch.isnan(gq[:, :, KEY:]).all()) and torch.equal(gq[:, :, :EXACT][..., cols], want[0][:, :, :EXACT][..., cols])
    over = (gq.double() - ref).abs() - (lim + 2.0 ** -8 * (ref.abs() + lim))
    assert float(over[:, :, EXACT:KEY][..., cols].max()) <= 0
    for got, ref in ((gk, want[1]), (gv, want[2])):
        assert bool(torch.isnan(got[:, :, KEY]).all()) and torch.equal(got[:, :, rest], ref[:, :, rest])
    # and as a chain: O is NaN where the forward says so
    o, lse = fa.fwd(q, k, v, **kw)
    gq, gk, gv = fa.bwd(q, k, v, o, lse, do, **kw)
    assert bool(torch.isnan(gq[:, :, KEY:]).all()) and bool(torch.isnan(gk).all()) and bool(torch.isnan(gv[:, :, KEY]).all())


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
def test_infinite_scores_are_capped(dk, dv):
    q, k, v, _ = inputs(dk, dv)
    kw = keywords(dk, False)
    sign = torch.sign(q[:, :, :1].float()).bfloat16()
    q = (q.float().abs() + 0.1).bfloat16() * sign  # one sign pattern for all queries: the score of a key like it overflows
    large = []
    for x in (1e4, 3e38, -1e4, -3e38):  # saturated, infinite
        k[:, :, KEY] = (x * sign[:, :, 0].float()).bfloat16()
        large.append(fa.fwd(q, k, v, **kw)[0])
    assert all(bool(torch.isfinite(t).all()) for t in large)
    assert torch.equal(large[0], large[1]) and torch.equal(large[2], large[3])
