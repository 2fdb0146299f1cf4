"""The attention backward pass against the formulas in 64 bits.

Bounds, element by element.  With u = 2^-8 (half a step of bf16, relative):
  P    is off by e_p = 1e-4 of itself in fp32: the score by d 2^-24 sum |q k|
       (below 6e-5 in base 2 for these inputs), the LSE, the subtraction and
       the exponential by a few 2^-23 each; then it rounds to bf16.
  dS = P (dP - D): dP and D are fp32 sums of up to 128 products, off by at
       most 128 * 2^-24 < 8e-6 of M = |dO||V| + |dO||O|; then it rounds.
  so  |dV error| <= (u + e_p) sum P |dO|
      |dS error| <= E = (u + 2 e_p) |dS| + 8e-6 P M (+ 1e-5 softcap P |dP - D| under a softcap)
      |dQ error| <= scale sum E |K|,  |dK error| <= scale sum E |Q|
plus half a step of the output's own type."""
import math

import pytest
import torch

from attention_attn_fwd_11_b200 import fa

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def slopes(Hq, max_bias):
    if not max_bias:
        return torch.ones(Hq)
    n = 1 << (Hq.bit_length() - 1)
    m0, m1 = 2.0 ** (-max_bias / n), 2.0 ** (-max_bias / 2 / n)
    return torch.tensor([m0 ** (h + 1) if h < n else m1 ** (2 * (h - n) + 1) for h in range(Hq)])


def scores(q, k, scale, causal, mask, max_bias, softcap):
    """64-bit scores after the modifiers, and ds / dz."""
    G, Sq, Sk = q.shape[1] // k.shape[1], q.shape[2], k.shape[2]
    s = q @ k.repeat_interleave(G, 1).transpose(-1, -2) * scale
    f = torch.ones_like(s)
    if softcap:
        t = torch.tanh(s)
        s, f = softcap * t, softcap * (1 - t * t)
    if mask is not None:
        s = s + slopes(q.shape[1], max_bias).double().to(s.device).view(1, -1, 1, 1) * mask.double()
    if causal:
        hide = torch.arange(Sk, device=s.device)[None] > torch.arange(Sq, device=s.device)[:, None] + Sk - Sq
        s = s.masked_fill(hide, -math.inf)
    return s, f


def forward(q, k, v, sinks=None, **kw):
    s, _ = scores(q, k, **kw)
    B, Hq, Sq, _ = s.shape
    all_s = s if sinks is None else torch.cat([s, sinks.double().view(1, Hq, 1, 1).expand(B, Hq, Sq, 1)], -1)
    lse = torch.logsumexp(all_s, -1) if all_s.shape[-1] else torch.full((B, Hq, Sq), -math.inf, device=s.device).double()
    p = torch.where(s > -math.inf, torch.exp(s - lse[..., None]), 0.0)
    return p @ v.repeat_interleave(Hq // k.shape[1], 1), lse


def reference(q, k, v, o, lse, do, dlse=None, sinks=None, **kw):
    """{name: (gradient, bound before the output's rounding)}"""
    q, k, v, o, lse, do = (t.double() for t in (q, k, v, o, lse, do))
    B, Hq, Sq, _ = q.shape
    Hkv, G = k.shape[1], Hq // k.shape[1]
    s, f = scores(q, k, **kw)
    L = torch.where(lse == -math.inf, math.inf, lse)[..., None]
    p = torch.exp(s - L)
    D = (do * o).sum(-1, keepdim=True)
    if dlse is not None:
        D = D - torch.where(lse == -math.inf, 0.0, dlse.double())[..., None]
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    t = do @ vv.transpose(-1, -2) - D
    ds = p * t * f
    M = do.abs() @ vv.abs().transpose(-1, -2) + (do.abs() * o.abs()).sum(-1, keepdim=True)
    u, ep, scale = 2.0 ** -8, 1e-4, kw["scale"]
    E = (u + 2 * ep) * ds.abs() + 8e-6 * p * f.abs() * M
    if kw["softcap"]:
        E = E + 1e-5 * kw["softcap"] * p * t.abs()
    fold = lambda x: x.view(B, Hkv, G, *x.shape[2:]).sum(2)  # noqa: E731
    r = {"dq": (scale * ds @ kk, scale * E @ kk.abs()),
         "dk": (fold(scale * ds.transpose(-1, -2) @ q), fold(scale * E.transpose(-1, -2) @ q.abs())),
         "dv": (fold(p.transpose(-1, -2) @ do), fold((u + ep) * p.transpose(-1, -2) @ do.abs()))}
    if sinks is not None:
        ps = torch.exp(sinks.double().view(1, Hq, 1, 1) - L)
        r["dsinks"] = (-(ps * D).sum((0, 2, 3)), (1e-5 * ps * ((do * o).abs().sum(-1, keepdim=True) + D.abs())).sum((0, 2, 3)))
    return r


def check(got, ref, what=""):
    for (name, (g, lim)), x in zip(ref.items(), got):
        assert x.shape == g.shape and bool(torch.isfinite(x).all()), what + name
        over = (x.double() - g).abs() - (lim + HALF[x.dtype] * (g.abs() + lim) + 1e-20)
        assert x.numel() == 0 or float(over.max()) <= 0, "%s %s: %g over the bound" % (what, name, float(over.max()))


def rand(g, shape, layout="bhsd", scale=1.0):
    B, H, S, d = shape
    if layout == "bshd":
        return (torch.randn((B, S, H, d), generator=g, device="cuda") * scale).bfloat16().transpose(1, 2)
    if layout == "wide":  # rows inside a wider projection
        return (torch.randn((B, S, H, d + 24), generator=g, device="cuda") * scale).bfloat16()[..., 8:8 + d].transpose(1, 2)
    return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()


def inputs(B, Hq, Hkv, Sq, Sk, dk, dv, seed, layout="bhsd", scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [rand(g, s, layout, scale) for s in ((B, Hq, Sq, dk), (B, Hkv, Sk, dk), (B, Hkv, Sk, dv), (B, Hq, Sq, dv))]


def run(B, Hq, Hkv, Sq, Sk, dk, dv, causal, seed, layout="bhsd", o_dtype=torch.float32, grad_dtype=torch.bfloat16,
        mask=None, max_bias=0.0, softcap=0.0, sinks=None, scale=None, magnitude=1.0):
    """Forward and backward through the library, checked."""
    q, k, v, do = inputs(B, Hq, Hkv, Sq, Sk, dk, dv, seed, layout, magnitude)
    kw = dict(scale=scale or 1.0 / math.sqrt(dk), causal=causal, mask=mask, max_bias=max_bias, softcap=softcap)
    o, lse = fa.fwd(q, k, v, out_dtype=o_dtype, sinks=sinks, **kw)
    got = fa.bwd(q, k, v, o, lse, do, sinks=sinks, grad_dtype=grad_dtype, **kw)
    torch.cuda.synchronize()
    assert fa.device_error() == 0
    check(got, reference(q, k, v, o, lse, do, sinks=sinks, **kw),
          "B%d Hq%d Hkv%d Sq%d Sk%d d%d/%d causal%d: " % (B, Hq, Hkv, Sq, Sk, dk, dv, causal))
    return got


PAIRS = [(64, 64), (128, 128), (192, 128)]


@pytest.mark.parametrize("dk,dv", PAIRS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("sq,sk", [(1, 1), (128, 128), (64, 300), (300, 64), (129, 257), (257, 129), (1, 500), (500, 1),
                                   (191, 193), (640, 640)])
def test_lengths(dk, dv, causal, sq, sk):
    run(1, 2, 2, sq, sk, dk, dv, causal, seed=sq + 3 * sk + dk)


@pytest.mark.parametrize("dk,dv", PAIRS)
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (6, 2), (8, 8)])
@pytest.mark.parametrize("layout", ["bhsd", "bshd", "wide"])
def test_heads_and_layouts(dk, dv, Hq, Hkv, layout):
    run(2, Hq, Hkv, 200, 333, dk, dv, True, seed=Hq + dk, layout=layout)


@pytest.mark.parametrize("dk,dv", PAIRS)
@pytest.mark.parametrize("o_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
def test_types(dk, dv, o_dtype, grad_dtype):
    run(2, 2, 1, 150, 222, dk, dv, False, seed=5 + dk, o_dtype=o_dtype, grad_dtype=grad_dtype)


@pytest.mark.parametrize("magnitude", [0.01, 3.0])
def test_magnitudes(magnitude):
    """Nearly equal weights, and weights that gather on one key (scores up to about 100; 9 times the sums |q k| of
    unit inputs, so the score's own error grows to 9 * 6e-5 and e_p no longer covers it: scale it back)."""
    run(1, 2, 2, 260, 260, 128, 128, True, seed=9, magnitude=magnitude, scale=1.0 / math.sqrt(128) / max(1.0, magnitude))


@pytest.mark.parametrize("sq,sk", [(1025, 1999), (2048, 2048)])
def test_long(sq, sk):
    run(1, 4, 2, sq, sk, 128, 128, True, seed=sq)


@pytest.mark.parametrize("dk,dv", PAIRS)
@pytest.mark.parametrize("causal", [False, True])
def test_modifiers(dk, dv, causal):
    B, Hq, Sq, Sk = 2, 6, 203, 261
    g = torch.Generator(device="cuda").manual_seed(77)
    wide = torch.randn((B, 1, Sq, 264), generator=g, device="cuda")
    wide[0, :, :, 200:] = -math.inf  # padded keys
    wide[1, :, 3::41] = -math.inf    # rows that see nothing
    wide[1, :, 5, 1:] = -65504.0     # the type's lowest value
    mask = wide.half()[..., :Sk]
    sinks = torch.randn(Hq, generator=g, device="cuda")
    kw = dict(layout="bshd", o_dtype=torch.float32)
    run(B, Hq, 3, Sq, Sk, dk, dv, causal, seed=1, mask=mask, **kw)
    run(B, Hq, 3, Sq, Sk, dk, dv, causal, seed=2, mask=mask, max_bias=8.0, **kw)
    run(B, Hq, 3, Sq, Sk, dk, dv, causal, seed=3, softcap=15.0, scale=1 / (15 * math.sqrt(dk)), **kw)
    run(B, Hq, 3, Sq, Sk, dk, dv, causal, seed=4, sinks=sinks, **kw)
    run(B, Hq, 3, Sq, Sk, dk, dv, causal, seed=5, mask=mask, max_bias=4.0, softcap=15.0, sinks=sinks,
        scale=1 / (15 * math.sqrt(dk)), **kw)
    per_head = torch.randn((1, Hq, Sq, 264), generator=g, device="cuda").half()[..., :Sk]
    run(B, Hq, 3, Sq, Sk, dk, dv, causal, seed=6, mask=per_head, **kw)


@pytest.mark.parametrize("dk,dv", PAIRS)
@pytest.mark.parametrize("lowest", [-65504.0, -30000.0])
def test_rows_whose_mask_is_the_lowest_value_everywhere(dk, dv, lowest):
    """Such rows are not empty: their weights follow from the scores, although scores and LSE sit at the mask's value."""
    mask = torch.zeros((2, 1, 150, 264), device="cuda")
    mask[:, :, 7::13] = lowest
    mask[1, :, 100:] = lowest
    run(2, 4, 2, 150, 261, dk, dv, False, seed=6, mask=mask.half()[..., :261], grad_dtype=torch.float32)


@pytest.mark.parametrize("dk,dv", PAIRS)
@pytest.mark.parametrize("S", [128, 256, 300])
@pytest.mark.parametrize("causal", [False, True])
def test_many_short_walks(dk, dv, S, causal):
    """More tiles than SMs, each with one to three tiles to walk: an SM goes through several of dK / dV and on to dQ
    with hardly any work in between."""
    for seed in range(3):
        run(8, 32, 32, S, S, dk, dv, causal, seed=seed, o_dtype=torch.bfloat16)


@pytest.mark.parametrize("dk,dv", PAIRS)
def test_many_walks_again_and_again(dk, dv):
    q, k, v, do = inputs(2, 16, 16, 2048, 2048, dk, dv, 77)
    o, lse = fa.fwd(q, k, v, causal=True)
    first = fa.bwd(q, k, v, o, lse, do, causal=True)
    check(first, reference(q, k, v, o, lse, do, scale=1 / math.sqrt(dk), causal=True, mask=None, max_bias=0.0, softcap=0.0))
    for _ in range(20):
        for a, b in zip(first, fa.bwd(q, k, v, o, lse, do, causal=True)):
            assert torch.equal(a, b)


# Walks long beside the whole work, which several SMs share: few keys or KV
# heads with many queries, few queries with many keys, parts that a causal mask
# leaves empty, parts that end inside a head's queries.
@pytest.mark.parametrize("Hq,Hkv,sq,sk,causal", [
    (7, 1, 1500, 40, False), (7, 1, 1500, 40, True), (4, 1, 342, 342, True), (8, 1, 700, 130, True), (3, 3, 1, 1700, True),
    (2, 2, 16, 2000, False), (1, 1, 1300, 1300, True), (10, 2, 777, 333, False), (9, 1, 129, 1, True), (2, 1, 1000, 1601, True)])
@pytest.mark.parametrize("dk,dv", PAIRS)
def test_shared_walks(Hq, Hkv, sq, sk, causal, dk, dv):
    seed = Hq + sq + sk + dk
    x = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((2, Hq, sq, dk), (2, Hkv, sk, dk), (2, Hkv, sk, dv))]
    rows = 6 * 4 * 2 * Hq * ((sq + 383) // 384 * 384)
    assert fa.bwd_workspace_bytes(*x) > rows + 512  # holds parts
    f32 = run(2, Hq, Hkv, sq, sk, dk, dv, causal, seed=seed, layout="wide", grad_dtype=torch.float32)
    again = run(2, Hq, Hkv, sq, sk, dk, dv, causal, seed=seed, layout="wide", grad_dtype=torch.float32)
    assert all(torch.equal(a, b) for a, b in zip(f32, again))
    bf16 = run(2, Hq, Hkv, sq, sk, dk, dv, causal, seed=seed, layout="bshd", o_dtype=torch.bfloat16)
    assert all(t.dtype == torch.bfloat16 for t in bf16)


@pytest.mark.parametrize("dk,dv", PAIRS)
@pytest.mark.parametrize("causal", [False, True])
def test_shared_walks_with_modifiers(dk, dv, causal):
    g = torch.Generator(device="cuda").manual_seed(dk)
    mask = torch.randn((1, 1, 900, 208), generator=g, device="cuda").half()[..., :203]
    mask[:, :, 40:60] = -math.inf  # rows that see nothing
    sinks = torch.randn(6, generator=g, device="cuda")
    run(1, 6, 1, 900, 203, dk, dv, causal, seed=dk, mask=mask, max_bias=8.0, softcap=5.0, sinks=sinks,
        scale=1 / (5 * math.sqrt(dk)))


def test_shared_walks_write_their_workspace_alone():
    q, k, v, do = inputs(1, 5, 1, 1100, 70, 128, 128, seed=12)
    o, lse = fa.fwd(q, k, v)
    n = fa.bwd_workspace_bytes(q, k, v)
    room = torch.full((n + 4096,), 90, dtype=torch.uint8, device="cuda")
    want = fa.bwd(q, k, v, o, lse, do)
    got = fa.bwd(q, k, v, o, lse, do, workspace=room[:n])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((room[n:] == 90).all())
    with pytest.raises(fa.FAError):
        fa.bwd(q, k, v, o, lse, do, workspace=room[:n - 256])


def test_rows_that_see_nothing_give_zeros():
    q, k, v, do = inputs(1, 2, 2, 300, 130, 128, 128, 3)
    o, lse = fa.fwd(q, k, v, causal=True)
    dq, dk, dv = fa.bwd(q, k, v, o, lse, do, causal=True)
    assert bool((lse[:, :, :170] == -math.inf).all()) and bool((dq[:, :, :170] == 0).all())
    for what in (q, do):  # those rows add nothing to dk and dv, whatever finite values they hold
        what[:, :, :170] = 1e4
    again = fa.bwd(q, k, v, o, lse, do, causal=True)
    assert torch.equal(dk, again[1]) and torch.equal(dv, again[2])
    mask = torch.full((1, 1, 300, 136), -math.inf, device="cuda", dtype=torch.float16)[..., :130]
    sinks = torch.tensor([0.5, -1.0], device="cuda")
    o, lse = fa.fwd(q, k, v, mask=mask, sinks=sinks)
    for g in fa.bwd(q, k, v, o, lse, do, mask=mask, sinks=sinks):
        assert bool((g == 0).all())


def test_empty_lengths():
    q, k, v, do = inputs(2, 2, 1, 70, 90, 64, 64, 4)
    none = lambda t: t[:, :, :0]  # noqa: E731
    dq, dk, dv = fa.bwd(none(q), k, v, none(q).float(), torch.empty(2, 2, 0, device="cuda"), none(do))
    assert dq.shape == (2, 2, 0, 64) and bool((dk == 0).all()) and bool((dv == 0).all())
    lse = torch.full((2, 2, 70), -math.inf, device="cuda")
    dq, dk, dv = fa.bwd(q, none(k), none(v), torch.zeros_like(q), lse, do)
    assert bool((dq == 0).all()) and dk.shape == (2, 1, 0, 64)
    e = fa.bwd(q[:0], k[:0], v[:0], q[:0], lse[:0], do[:0], sinks=torch.zeros(2, device="cuda"))
    assert e[0].shape[0] == 0 and e[3].tolist() == [0.0, 0.0]


@pytest.mark.parametrize("dk,dv", PAIRS)
def test_log_sum_exp_gradient(dk, dv):
    q, k, v, do = inputs(2, 4, 2, 133, 180, dk, dv, 8)
    kw = dict(scale=1 / math.sqrt(dk), causal=True, mask=None, max_bias=0.0, softcap=0.0)
    sinks = torch.tensor([0.3, -0.2, 1.0, 0.0], device="cuda")
    dlse = torch.randn(2, 4, 133, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    o, lse = fa.fwd(q, k, v, sinks=sinks, **kw)
    check(fa.bwd(q, k, v, o, lse, do, dlse=dlse, sinks=sinks, **kw),
          reference(q, k, v, o, lse, do, dlse=dlse, sinks=sinks, **kw))


@pytest.mark.parametrize("softcap", [0.0, 6.0])
def test_against_differences(softcap):
    """Directional differences of the forward map in 64 bits, whose own error at step h is O(h^2) = 1e-7 of the
    third derivative; the gradients' bounds carry over along the direction."""
    B, Hq, Hkv, Sq, Sk, d = 1, 2, 1, 37, 53, 64
    q, k, v, do = inputs(B, Hq, Hkv, Sq, Sk, d, d, 21)
    sinks = torch.tensor([0.4, -0.7], device="cuda")
    kw = dict(scale=1 / math.sqrt(d) / (softcap or 1.0), causal=True, mask=None, max_bias=0.0, softcap=softcap)
    dlse = torch.randn(B, Hq, Sq, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    x = [t.double() for t in (q, k, v, sinks)]

    def loss(q, k, v, s):
        o, lse = forward(q, k, v, sinks=s, **kw)
        return (o * do.double()).sum() + (lse * dlse.double()).sum()

    o, lse = forward(*x[:3], sinks=x[3], **kw)
    got = fa.bwd(q, k, v, o.float(), lse.float(), do, dlse=dlse, sinks=sinks, grad_dtype=torch.float32, **kw)
    ref = reference(q, k, v, o, lse, do, dlse=dlse, sinks=sinks, **kw)
    g = torch.Generator(device="cuda").manual_seed(3)
    for i, name in enumerate(("dq", "dk", "dv", "dsinks")):
        for _ in range(3):
            e = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
            up, dn = list(x), list(x)
            up[i], dn[i] = x[i] + 1e-4 * e, x[i] - 1e-4 * e
            diff = float(loss(*up) - loss(*dn)) / 2e-4
            lim = float(((ref[name][1] + 2.0 ** -24 * ref[name][0].abs()) * e.abs()).sum())
            assert abs(float((got[i].double() * e).sum()) - diff) <= lim + 1e-5 * (1 + abs(diff)), name


def test_equal_calls_give_equal_bits():
    q, k, v, do = inputs(2, 8, 2, 515, 700, 128, 128, 31)
    o, lse = fa.fwd(q, k, v, causal=True)
    first = fa.bwd(q, k, v, o, lse, do, causal=True)
    for _ in range(3):
        for a, b in zip(first, fa.bwd(q, k, v, o, lse, do, causal=True)):
            assert torch.equal(a, b)


def test_given_outputs_and_what_lies_around_them():
    q, k, v, do = inputs(2, 4, 2, 130, 70, 128, 128, 33)
    o, lse = fa.fwd(q, k, v)
    want = fa.bwd(q, k, v, o, lse, do)
    bufs, outs = [], []
    for t in (q, k, v):
        B, H, S, d = t.shape
        buf = torch.full((B, S + 2, H, d + 16), 7.0, device="cuda", dtype=torch.bfloat16)
        bufs.append(buf)
        outs.append(buf[:, 1:S + 1, :, 8:d + 8].transpose(1, 2))
    ws = torch.full((fa.bwd_workspace_bytes(q, k, v),), 255, device="cuda", dtype=torch.uint8)
    got = fa.bwd(q, k, v, o, lse, do, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    for w, g, out, buf in zip(want, got, outs, bufs):
        assert g.data_ptr() == out.data_ptr() and torch.equal(g, w)
        out.fill_(7.0)
        assert bool((buf == 7.0).all()), "something outside the gradient was written"


def test_training_step_with_rotary_positions():
    """q and k turned, attention, and the gradients turned back: against the same chain in 64 bits."""
    B, Hq, Hkv, S, d = 2, 4, 2, 150, 128
    q, k, v, do = inputs(B, Hq, Hkv, S, S, d, d, 41)
    inv, _ = fa.rope_frequencies(d)
    qr, kr = fa.rope(q, inv, k=k)
    o, lse = fa.fwd(qr, kr, v, causal=True)
    dq, dk, dv = fa.bwd(qr, kr, v, o, lse, do, causal=True, grad_dtype=torch.float32)
    dq, dk = fa.rope(dq, inv, k=dk, inverse=True)
    a = torch.arange(S, device="cuda").double()[:, None] * inv.cuda()
    rot = torch.polar(torch.ones_like(a), a)

    def turn(x, w):
        y = torch.view_as_complex(x.double().unflatten(-1, (2, d // 2)).transpose(-1, -2).contiguous()) * w
        return torch.view_as_real(y).transpose(-1, -2).flatten(-2)

    kw = dict(scale=1 / math.sqrt(d), causal=True, mask=None, max_bias=0.0, softcap=0.0)
    ref = reference(qr, kr, v, o, lse, do, **kw)
    for got, name in ((dq, "dq"), (dk, "dk")):
        g, lim = ref[name]
        back = turn(g, rot.conj())
        pair = (lim + 1e-6 * g.abs()).unflatten(-1, (2, d // 2)).sum(-2, keepdim=True).expand(*lim.shape[:-1], 2, d // 2)
        assert bool(((got.double() - back).abs() <= pair.flatten(-2)).all()), name
    check([dv], {"dv": ref["dv"]})


def test_captured_and_replayed_on_another_stream():
    q, k, v, do = inputs(1, 4, 2, 200, 300, 128, 128, 51)
    o, lse = fa.fwd(q, k, v, causal=True)
    ws = torch.empty(fa.bwd_workspace_bytes(q, k, v), device="cuda", dtype=torch.uint8)
    outs = [torch.empty_like(t) for t in (q, k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw = dict(causal=True, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    with torch.cuda.stream(side):
        fa.bwd(q, k, v, o, lse, do, **kw)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            fa.bwd(q, k, v, o, lse, do, **kw)
    do.copy_(torch.randn(do.shape, device="cuda"))
    for t in outs:
        t.zero_()
    ws.fill_(255)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, fa.bwd(q, k, v, o, lse, do, causal=True)):
        assert torch.equal(a, b)


def test_on_a_given_stream_that_is_still_busy():
    """The workspace made inside outlives the call until its kernels are done."""
    q, k, v, do = inputs(1, 5, 1, 1100, 70, 128, 128, seed=3)
    o, lse = fa.fwd(q, k, v)
    want = fa.bwd(q, k, v, o, lse, do)
    n = fa.bwd_workspace_bytes(q, k, v)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms
    got = fa.bwd(q, k, v, o, lse, do, stream=side)
    others = [torch.full((n,), 90, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(bool((t == 90).all()) for t in others)


def test_two_calls_at_once():
    cases = [inputs(1, 7, 1, 1500, 40, 128, 128, seed=1), inputs(2, 8, 8, 700, 700, 64, 64, seed=2)]
    fwd = [fa.fwd(*c[:3], causal=True) for c in cases]
    want = [fa.bwd(*c[:3], o, lse, c[3], causal=True) for c, (o, lse) in zip(cases, fwd)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (c, (o, lse)) in enumerate(zip(cases, fwd)):
            with torch.cuda.stream(streams[i]):
                got[i].append(fa.bwd(*c[:3], o, lse, c[3], causal=True))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))


def test_refusals():
    q, k, v, do = inputs(1, 4, 2, 20, 30, 64, 64, 61)
    o, lse = fa.fwd(q, k, v)
    ok = dict(q=q, k=k, v=v, o=o, lse=lse, do=do)
    for bad in (dict(q=q.float()), dict(do=do.float()), dict(k=k[:, :, :5]), dict(v=v[:, :1]), dict(o=o[:, :, :3]),
                dict(lse=lse.double()), dict(lse=lse[:, :2]), dict(lse=lse.transpose(1, 2)), dict(dq=k), dict(dk=q),
                dict(dv=v.float()), dict(mask=torch.zeros(1, 1, 20, 30, device="cuda")),
                dict(mask=torch.zeros(1, 3, 20, 30, device="cuda", dtype=torch.float16)),
                dict(mask=torch.zeros(1, 1, 20, 32, device="cuda", dtype=torch.float16)),
                dict(sinks=torch.zeros(3, device="cuda")), dict(dlse=lse.half()), dict(grad_dtype=torch.float16),
                dict(do=do.transpose(2, 3))):
        with pytest.raises(ValueError):
            fa.bwd(**{**ok, **bad})
    with pytest.raises(fa.FAError):  # a broadcast gradient has no rows to read
        fa.bwd(**{**ok, "do": do[:, :, :1].expand(1, 4, 20, 64)})
    with pytest.raises(fa.FAError):
        fa.bwd(**{**ok, "scale": -1.0})
    with pytest.raises(fa.FAError):
        fa.bwd(**ok, workspace=torch.empty(16, device="cuda", dtype=torch.uint8))
