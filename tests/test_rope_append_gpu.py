"""Rotary positions and the paged cache append against 64-bit arithmetic.

Tolerance of a turned value.  The angle is off by at most 1.5e-9 radians (the
32-bit fraction of a turn) plus half a step of the fp32 fraction, pi 2^-24;
sine and cosine by 2 units of the last place (of values below 1: 2^-23);
the factor mscale, the product and the difference round three times.  Together
|error| <= (1.9e-7 + 1.2e-7 + 3 * 6e-8) mscale (|x0| + |x1|) < 5e-7 mscale
(|x0| + |x1|) before the output's own rounding, which is half a step: 2^-8
of the value for bf16, 2^-24 for fp32."""
import numpy as np
import pytest
import torch

from attention_attn_fwd_11_b200 import fa

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def turned(x, pos, inv, mscale=1.0, interleaved=False, offset=0, inverse=False):
    """x [B, H, S, d], pos [B, S] -> (y, |x0| + |x1| of each value's pair) in 64 bits."""
    x = x.double().cpu().clone()
    y, mag = x.clone(), torch.zeros_like(x)
    m = inv.numel()
    a = pos.double().cpu()[:, None, :, None] * inv * (-1.0 if inverse else 1.0)
    c, s = torch.cos(a) * mscale, torch.sin(a) * mscale
    for i in range(m):
        p, q = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + m + i)
        u, w, ci, si = x[..., p], x[..., q], c[..., i], s[..., i]
        y[..., p], y[..., q] = u * ci - w * si, w * ci + u * si
        mag[..., p] = mag[..., q] = (u.abs() + w.abs()) * abs(mscale)
    return y, mag


def check(got, ref, mag, what=""):
    half = HALF[got.dtype]
    err = (got.double().cpu() - ref).abs() - (half * (ref.abs() + 5e-7 * mag) + 5e-7 * mag)
    assert float(err.max()) <= 0, "%s: %g over" % (what, float(err.max()))


def strided(shape, dtype, layout, seed):
    B, H, S, d = shape
    if layout == "bhsd":
        return torch.randn(shape, generator=gen(seed)).to(dtype).cuda()
    if layout == "bshd":
        return torch.randn((B, S, H, d), generator=gen(seed)).to(dtype).cuda().transpose(1, 2)
    # one row of a wider projection, with columns in front and behind
    wide = torch.randn((B, S, H, d + 48), generator=gen(seed)).to(dtype).cuda()
    return wide[..., 16:16 + d].transpose(1, 2)


CASES = [  # B, Hq, Hk, S, d, rot, offset, interleaved, inverse, dtype, layout
    (1, 1, 0, 1, 16, 16, 0, False, False, torch.bfloat16, "bhsd"),
    (2, 3, 1, 77, 64, 64, 0, False, False, torch.bfloat16, "bshd"),
    (2, 3, 1, 77, 64, 64, 0, True, True, torch.bfloat16, "wide"),
    (1, 32, 8, 130, 128, 128, 0, False, True, torch.bfloat16, "bshd"),
    (3, 5, 5, 9, 128, 32, 96, True, False, torch.float32, "bhsd"),
    (1, 2, 1, 33, 192, 64, 128, False, False, torch.float32, "wide"),
    (2, 2, 2, 17, 96, 96, 0, False, False, torch.float32, "bshd"),
    (1, 128, 1, 5, 576, 64, 0, True, False, torch.bfloat16, "bhsd"),
    (1, 2, 2, 11, 256, 256, 0, False, False, torch.bfloat16, "wide"),
    (1, 3, 0, 21, 1024, 48, 496, True, True, torch.bfloat16, "bhsd"),
]


@pytest.mark.parametrize("B,Hq,Hk,S,d,rot,offset,inter,inverse,dtype,layout", CASES)
@pytest.mark.parametrize("far", [False, True])
def test_rope(B, Hq, Hk, S, d, rot, offset, inter, inverse, dtype, layout, far):
    inv, m = fa.rope_frequencies(rot, scaling="yarn", factor=8.0, original_len=4096) if far else (
        fa.rope_frequencies(rot))
    q = strided((B, Hq, S, d), dtype, layout, 1)
    k = strided((B, Hk, S, d), dtype, layout, 2) if Hk else None
    pos = torch.randint(0, 2 ** 31 - 1 if far else 5000, (B, S), generator=gen(3)).to(torch.int32)
    q0, k0 = q.clone(), None if k is None else k.clone()
    qo, ko = fa.rope(q, inv, k=k, pos=pos.cuda(), interleaved=inter, offset=offset, inverse=inverse, mscale=m)
    assert (ko is None) == (k is None) and torch.equal(q, q0)
    kw = dict(mscale=m, interleaved=inter, offset=offset, inverse=inverse)
    check(qo, *turned(q, pos, inv, **kw), "q")
    if k is not None:
        check(ko, *turned(k, pos, inv, **kw), "k")
        fa.rope(q, inv, k=k, pos=pos.cuda(), out=q, k_out=k, **kw)  # in place: the same bits
        assert torch.equal(q, qo) and torch.equal(k, ko)


def test_rope_leaves_what_lies_around_the_rows():
    wide = torch.randn((2, 7, 3, 128), generator=gen(5)).to(torch.bfloat16).cuda()
    before = wide.clone()
    x = wide[..., 32:96].transpose(1, 2)
    inv, _ = fa.rope_frequencies(64)
    fa.rope(x, inv, pos0=3, out=x)
    assert torch.equal(wide[..., :32], before[..., :32]) and torch.equal(wide[..., 96:], before[..., 96:])
    pos = torch.arange(3, 10)[None].expand(2, 7)
    check(x, *turned(before[..., 32:96].transpose(1, 2), pos, inv))


def test_rope_positions_broadcast_default_and_negative():
    x = torch.randn((3, 2, 10, 64), generator=gen(6)).cuda()
    inv, _ = fa.rope_frequencies(64)
    p = torch.arange(-4, 6, dtype=torch.int32)
    ref = turned(x, p[None].expand(3, 10), inv)
    for got in (fa.rope(x, inv, pos0=-4)[0], fa.rope(x, inv, pos=p.cuda())[0], fa.rope(x, inv, pos=p[None].cuda())[0],
                fa.rope(x, inv, pos=p[None].cuda().expand(3, 10))[0]):
        check(got, *ref)


def test_rope_broadcast_input_and_empty():
    inv, _ = fa.rope_frequencies(32)
    x = torch.randn((1, 1, 6, 32), generator=gen(7)).cuda().expand(2, 4, 6, 32)
    check(fa.rope(x, inv)[0], *turned(x, torch.arange(6)[None].expand(2, 6), inv))
    assert fa.rope(torch.empty(0, 2, 3, 32, device="cuda"), inv)[0].shape == (0, 2, 3, 32)
    assert fa.rope(torch.empty(2, 2, 0, 32, device="cuda"), inv)[0].shape == (2, 2, 0, 32)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient_is_the_transpose(inter):
    """<dy, R x> = <R^T dy, x>, and against differences of the map itself (it is linear: they are exact up to rounding)."""
    inv, m = fa.rope_frequencies(48, scaling="yarn", factor=4.0, original_len=64)
    x, dy = (torch.randn((2, 2, 19, 64), generator=gen(s)).cuda() for s in (8, 9))
    kw = dict(pos0=1000, interleaved=inter, offset=16, mscale=m)
    y, dx = fa.rope(x, inv, **kw)[0], fa.rope(dy, inv, inverse=True, **kw)[0]
    a, b = float((dy.double() * y.double()).sum()), float((dx.double() * x.double()).sum())
    # every term of either sum is off by at most 5e-7 mscale (|x0| + |x1|) |dy| and 2^-24 |y| |dy|
    assert abs(a - b) <= 2e-6 * m * float((dy.double().abs() * x.double().abs().amax()).sum())
    e = torch.zeros_like(x)
    e[1, 0, 5, 20] = 1.0
    diff = (fa.rope(x + e, inv, **kw)[0].double() - fa.rope(x - e, inv, **kw)[0].double()) / 2
    assert abs(float((diff * dy.double()).sum()) - float(dx[1, 0, 5, 20])) <= 1e-5 * (1 + float(dy.abs().max()))


def test_rope_refusals():
    inv, _ = fa.rope_frequencies(64)
    x = torch.zeros((1, 2, 3, 64), device="cuda", dtype=torch.bfloat16)
    for bad in (dict(q=x.half()), dict(q=x[0]), dict(k=x.float()), dict(k=x[:, :, :2]), dict(k_out=x),
                dict(inv_freq=inv.float()), dict(inv_freq=inv.cuda()), dict(pos=torch.zeros(3, device="cuda")),
                dict(pos=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(out=x.float()),
                dict(q=x.transpose(2, 3))):
        with pytest.raises(ValueError):
            fa.rope(**{**dict(q=x, inv_freq=inv), **bad})
    with pytest.raises(fa.FAError):
        fa.rope(x, fa.rope_frequencies(40)[0])
    with pytest.raises(fa.FAError):
        fa.rope(x, inv, offset=16)


# ------------------------------------------------------------------ append --

def blocks_of(x, kv):
    """(d [.., n], codes [.., n, 32]) of 64-bit rows x, by the formulas of fa_kv_append."""
    b = x.unflatten(-1, (-1, 32))
    if kv == "q8_0":
        d = (b.abs().amax(-1) / 127)
    else:
        first = (b.abs() == b.abs().amax(-1, keepdim=True)).to(torch.int8).argmax(-1, keepdim=True)
        d = b.gather(-1, first)[..., 0] / -8
    d = d.to(torch.float16).double()
    lo, hi = (-127, 127) if kv == "q8_0" else (-8, 7)
    c = torch.where(d[..., None] == 0, 0.0, (b / d[..., None]).round().clamp(lo, hi))
    return d, c


def decode(cache, kv):
    """Stored rows -> (d, codes), the layouts of fa_kv_dequant."""
    size = 34 if kv == "q8_0" else 18
    b = cache.cpu().unflatten(-1, (-1, size))
    d = b[..., :2].contiguous().view(torch.float16)[..., 0].double()
    if kv == "q8_0":
        return d, b[..., 2:].contiguous().view(torch.int8).double()
    return d, torch.cat([b[..., 2:] & 15, b[..., 2:] >> 4], -1).double() - 8


def e4m3_near(x):
    return x.clamp(-448, 448)


def make(B, Hq, Hkv, Sq, dk, dv, kv, lens, qlens, seed, extra_blocks=2):
    width = max(1, -(-max(lens) // 64))
    nb = B * width + extra_blocks
    table = torch.randperm(nb, generator=gen(seed))[:B * width].view(B, width).to(torch.int32)
    row = {None: (dk, dv), "fp8_e4m3": (dk, dv), "q8_0": (dk // 32 * 34, dv // 32 * 34),
           "q4_0": (dk // 32 * 18, dv // 32 * 18)}[kv]
    if kv is None:
        kc, vc = (torch.randn((nb, Hkv, 64, r), generator=gen(seed + 1 + j)).bfloat16() for j, r in enumerate(row))
    else:
        kc, vc = (torch.randint(0, 120, (nb, Hkv, 64, r), generator=gen(seed + 1 + j)).to(torch.uint8)
                  for j, r in enumerate(row))
    k, v, q = (torch.randn((B, Sq, h, d), generator=gen(seed + 3 + j)).bfloat16().transpose(1, 2)
               for j, (h, d) in enumerate(((Hkv, dk), (Hkv, dv), (Hq, dk))))
    return dict(table=table, kc=kc, vc=vc, k=k, v=v, q=q, lens=torch.tensor(lens, dtype=torch.int32),
                qlens=None if qlens is None else torch.tensor(qlens, dtype=torch.int32))


def dev(t):
    return None if t is None else torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)


def check_cache(s, cache, got, rows, mag, kv, scale, n):
    """The slots of the new rows hold them; every other byte is as it was."""
    B, Sq = rows.shape[0], rows.shape[2]
    got = got.cpu()
    expect_same = torch.ones(cache.shape[0], cache.shape[2], dtype=torch.bool)
    for b in range(B):
        for i in range(n[b]):
            at = int(s["lens"][b]) - n[b] + i
            if at < 0:
                continue
            blk, slot = int(s["table"][b, at // 64]), at % 64
            expect_same[blk, slot] = False
            new, x, m = got[blk, :, slot], rows[b, :, i], mag[b, :, i]
            if kv is None:
                check(new, x, m, "row %d %d" % (b, i))
            elif kv == "fp8_e4m3":
                val = new.view(torch.float8_e4m3fn).double()
                q, near = x / scale, 5e-7 * m / scale
                # half a step of e4m3 is 2^-4 of the value, 2^-10 below its smallest normal; the quotient rounds once more
                err = (val - e4m3_near(q)).abs() - (2.0 ** -4 * (q.abs() + near) + 2.0 ** -10 + near + 2.0 ** -24 * q.abs())
                assert float(err.max()) <= 0
            else:
                # A value is off by half its block's step, or by the step a rounded scale leaves at the ends
                # (|x| <= 127.5 d holds to 2^-11 of it), plus the turn's own error.
                d, c = decode(new, kv)
                d2, _ = blocks_of(x, kv)
                bm = 5e-7 * m.unflatten(-1, (-1, 32)).amax(-1)
                tie = kv == "q4_0"  # equal magnitudes of either sign after an inexact turn
                dd, rr = (d.abs(), d2.abs()) if tie else (d, d2)
                assert bool(((dd - rr).abs() <= 2.0 ** -10 * rr + bm + 2.0 ** -24).all())
                val = (d[..., None] * c).flatten(-2)
                step = d.abs().repeat_interleave(32, -1)
                lim = 0.5 * step * (1 + 1e-6) + 127 * step * 2.0 ** -11 + 5e-7 * m + 2.0 ** -24
                if kv == "q4_0":  # the value opposite the largest one may lie a whole step outside [-8, 7]
                    lim = torch.where(x / torch.where(step == 0, 1.0, d.repeat_interleave(32, -1)) > 7.5 - 1e-3,
                                      1.01 * step + lim, lim)
                assert bool(((val - x).abs() <= lim).all())
    same = got.view(torch.int16 if kv is None else torch.uint8) == cache.view(torch.int16 if kv is None else torch.uint8)
    assert bool(same.all(-1).all(1)[expect_same].all()), "a slot outside the new rows changed"


KV = [None, "fp8_e4m3", "q8_0", "q4_0"]


def run(s, kv, n, inv=None, m=1.0, inter=False, offset=0, pos=None, with_q=True, ks=0.02, vs=0.03, in_place=False):
    kc, vc, q = dev(s["kc"]), dev(s["vc"]), dev(s["q"]) if with_q and inv is not None else None
    qo = fa.kv_append(dev(s["k"]), dev(s["v"]), kc, vc, dev(s["table"]), dev(s["lens"]), q_lens=dev(s["qlens"]),
                      inv_freq=inv, mscale=m, interleaved=inter, offset=offset, pos=dev(pos), q=q,
                      q_out=q if in_place else None, kv_type=kv, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert fa.device_error() == 0
    B, Sq = s["k"].shape[0], s["k"].shape[2]
    place = s["lens"].long()[:, None] - torch.tensor(n)[:, None] + torch.arange(Sq)[None]
    p = place if pos is None else pos.long().expand(B, Sq)
    zero = lambda t: (t.double(), torch.zeros(t.shape, dtype=torch.float64))  # noqa: E731
    kr = zero(s["k"]) if inv is None else turned(s["k"], p, inv, m, inter, offset)
    check_cache(s, s["kc"], kc, *kr, kv, ks, n)
    check_cache(s, s["vc"], vc, *zero(s["v"]), kv, vs, n)
    if q is not None:
        ref, mag = turned(s["q"], p, inv, m, inter, offset)
        live = torch.arange(Sq)[None, :] < torch.tensor(n)[:, None]
        check(qo, ref * live[:, None, :, None], mag, "q")
        assert bool((qo.cpu()[~live[:, None].expand(B, s["q"].shape[1], Sq)] == 0).all())
    else:
        assert qo is None
    return kc, vc, qo


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("inter,rot", [(False, 128), (True, 128), (False, 64), (True, 32), (None, 0)])
def test_append_types_and_pairs(kv, inter, rot):
    s = make(3, 4, 2, 9, 128, 128, kv, [9, 70, 200], [9, 4, 0], seed=11)
    inv, m = fa.rope_frequencies(rot, scaling="yarn", factor=4.0, original_len=64) if rot else (None, 1.0)
    run(s, kv, [9, 4, 0], inv, m, bool(inter), offset=32 if rot == 64 else 0)


@pytest.mark.parametrize("kv", KV)
def test_append_one_token_at_block_borders(kv):
    lens = [1, 2, 63, 64, 65, 128, 129, 191]
    s = make(8, 8, 2, 1, 128, 128, kv, lens, None, seed=21)
    run(s, kv, [1] * 8, fa.rope_frequencies(128)[0])


@pytest.mark.parametrize("dk,dv,rot,offset", [(64, 64, 64, 0), (192, 128, 64, 128), (256, 256, 256, 0), (320, 256, 96, 16),
                                              (576, 512, 64, 0), (16, 48, 16, 0)])
def test_append_head_sizes(dk, dv, rot, offset):
    s = make(2, 3, 3, 70, dk, dv, None, [75, 133], [70, 64], seed=31)
    run(s, None, [70, 64], fa.rope_frequencies(rot)[0], offset=offset, in_place=True)


def test_append_given_positions_and_rows_before_the_start():
    s = make(2, 2, 1, 6, 128, 128, None, [4, 100], None, seed=41)  # sequence 0 has four places for six rows
    pos = torch.tensor([[5, 900000, 3, 2, 1, 0], [7, 7, 7, 8, 8, 8]], dtype=torch.int32)
    run(s, None, [6, 6], fa.rope_frequencies(128)[0], pos=pos)
    run(s, None, [6, 6], fa.rope_frequencies(128)[0], pos=pos[1:])


@pytest.mark.parametrize("kv", ["q8_0", "q4_0"])
def test_append_blocks_of_zeros_ties_and_extremes(kv):
    """Without a turn the stored bytes follow from the formulas exactly."""
    s = make(1, 1, 1, 6, 128, 128, kv, [6], None, seed=51)
    s["k"][0, 0, 0] = 0
    s["k"][0, 0, 1, :64] = torch.tensor([2.0, -2.0] * 32)  # equal magnitudes: the first decides
    s["k"][0, 0, 1, 64:] = torch.tensor([-2.0, 2.0] * 32)
    s["k"][0, 0, 2] = 1e-9  # below f16: the scale is 0
    s["k"][0, 0, 3] = 3e38  # above it: the scale is the largest f16
    s["k"][0, 0, 4, 5] = 0.5 ** 24 * 127 * 1.5  # a subnormal scale
    s["k"][0, 0, 4, :5] = s["k"][0, 0, 4, 6:] = 0
    kc, _, _ = fa.kv_append(dev(s["k"]), dev(s["v"]), c := dev(s["kc"]), dev(s["vc"]), dev(s["table"]), dev(s["lens"]),
                            kv_type=kv), 0, 0
    b = s["k"][0, 0].double().unflatten(-1, (-1, 32))
    blk = int(s["table"][0, 0])
    d, codes = decode(c[blk, 0, :6], kv)
    if kv == "q8_0":
        want = (b.abs().amax(-1).float() / 127).double()
        lo, hi = -127, 127
    else:
        first = (b.abs() == b.abs().amax(-1, keepdim=True)).to(torch.int8).argmax(-1, keepdim=True)
        want = b.gather(-1, first)[..., 0] / -8
        lo, hi = -8, 7
    want = want.clamp(-65504, 65504).to(torch.float16).double()
    assert torch.equal(d, want)
    w = want[..., None]
    ref = torch.where(w == 0, 0.0, (b.float() / w.float()).double().round().clamp(lo, hi))
    assert torch.equal(codes, ref)


@pytest.mark.parametrize("kv", ["q8_0", "q4_0"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_append_block_with_a_value_that_is_no_number(kv, bad):
    s = make(1, 1, 1, 2, 128, 128, kv, [2], None, seed=61)
    s["k"][0, 0, 1, 40] = bad
    c = dev(s["kc"])
    fa.kv_append(dev(s["k"]), dev(s["v"]), c, dev(s["vc"]), dev(s["table"]), dev(s["lens"]), kv_type=kv)
    d, _ = decode(c[int(s["table"][0, 0]), 0, :2], kv)
    assert bool(torch.isnan(d[1, 1])) and int(torch.isnan(d).sum()) == 1


def test_append_fp8_limits_and_nan():
    s = make(1, 1, 1, 1, 128, 128, "fp8_e4m3", [1], None, seed=71)
    s["k"][0, 0, 0, :6] = torch.tensor([1e30, -1e30, float("inf"), float("-inf"), float("nan"), 0.0])
    c = dev(s["kc"])
    fa.kv_append(dev(s["k"]), dev(s["v"]), c, dev(s["vc"]), dev(s["table"]), dev(s["lens"]), kv_type="fp8_e4m3")
    x = c[int(s["table"][0, 0]), 0, 0, :6].view(torch.float8_e4m3fn).float().cpu()
    assert x[:4].tolist() == [448.0, -448.0, 448.0, -448.0] and bool(torch.isnan(x[4])) and x[5] == 0


def test_append_bad_blocks_are_latched_and_skipped():
    s = make(4, 1, 2, 3, 128, 128, None, [10, 64, 65, 30], None, seed=81)
    table = s["table"].clone()
    table[0, 0], table[1, 0] = -1, s["kc"].shape[0]
    lens = s["lens"].clone()
    lens[2] = table.shape[1] * 64 + 1  # the last new row lies past the table's end
    kc, vc = dev(s["kc"]), dev(s["vc"])
    fa.device_error()
    fa.kv_append(dev(s["k"]), dev(s["v"]), kc, vc, dev(table), dev(lens))
    assert fa.device_error() == 2 and fa.device_error() == 0
    s["lens"], n = lens, [0, 0, 3, 3]
    s["k"], s["v"] = s["k"][:, :, :3], s["v"][:, :, :3]
    # sequence 2 keeps its first two rows, sequence 3 all three
    want = s["kc"].clone()
    for b, i in ((2, 0), (2, 1), (3, 0), (3, 1), (3, 2)):
        at = int(lens[b]) - 3 + i
        want[int(table[b, at // 64]), :, at % 64] = s["k"][b, :, i]
    assert torch.equal(kc.cpu().view(torch.int16), want.view(torch.int16))


def test_append_refusals():
    s = make(2, 2, 1, 3, 128, 128, None, [5, 6], None, seed=91)
    inv, _ = fa.rope_frequencies(128)
    ok = dict(k=dev(s["k"]), v=dev(s["v"]), k_cache=dev(s["kc"]), v_cache=dev(s["vc"]), block_table=dev(s["table"]),
              seq_lens=dev(s["lens"]), inv_freq=inv, q=dev(s["q"]))
    u8 = torch.zeros((4, 1, 64, 136), dtype=torch.uint8, device="cuda")
    for bad in (dict(k=ok["k"].float()), dict(v=ok["v"][:, :, :2]), dict(v=ok["v"][:1]), dict(q=ok["q"][:, :, :2]),
                dict(k_cache=ok["k_cache"][..., :64].contiguous()), dict(k_cache=u8), dict(kv_type="q8_0"),
                dict(k_cache=u8, v_cache=u8, kv_type="q4_0"), dict(block_table=ok["block_table"].long()),
                dict(seq_lens=ok["seq_lens"][:1]), dict(q_lens=ok["seq_lens"].long()), dict(inv_freq=None),
                dict(q=None, q_out=ok["q"]), dict(q_out=ok["q"].float()), dict(k_cache=ok["k_cache"].transpose(0, 1))):
        with pytest.raises(ValueError):
            fa.kv_append(**{**ok, **bad})
    with pytest.raises(fa.FAError):
        fa.kv_append(**{**ok, "k_cache": ok["k_cache"].view(-1, 1, 32, 128), "v_cache": ok["v_cache"].view(-1, 1, 32, 128)})


def test_append_then_decode_reads_the_rows():
    """The serving step: a prompt and then single tokens appended with their turn, and read by the paged kernels."""
    B, Hq, Hkv, n0 = 2, 4, 2, 70
    inv, _ = fa.rope_frequencies(128)
    s = make(B, Hq, Hkv, n0 + 3, 128, 128, None, [n0 + 3] * B, None, seed=101)
    kc, vc, table = torch.zeros_like(dev(s["kc"])), torch.zeros_like(dev(s["vc"])), dev(s["table"])
    k, v, q = (dev(s[n]) for n in ("k", "v", "q"))
    pos = torch.arange(n0 + 3)
    kt, qt = (turned(t, pos[None].expand(B, n0 + 3), inv)[0] for t in (s["k"], s["q"]))
    outs = []
    lens = torch.full((B,), n0, dtype=torch.int32, device="cuda")
    qp = fa.kv_append(k[:, :, :n0], v[:, :, :n0], kc, vc, table, lens, inv_freq=inv, q=q[:, :, :n0])
    outs.append(fa.prefill_paged(qp, kc, vc, table, lens)[0])
    for t in range(3):
        lens = lens + 1
        qp = fa.kv_append(k[:, :, n0 + t:n0 + t + 1], v[:, :, n0 + t:n0 + t + 1], kc, vc, table, lens, inv_freq=inv,
                          q=q[:, :, n0 + t:n0 + t + 1])
        outs.append(fa.decode_paged(qp[:, :, 0].contiguous(), kc, vc, table, lens)[0][:, :, None])
    got = torch.cat(outs, 2).double().cpu()
    z = qt @ kt.repeat_interleave(Hq // Hkv, 1).transpose(-1, -2) / 128 ** 0.5
    z = z.masked_fill(torch.ones(n0 + 3, n0 + 3).triu(1).bool(), -np.inf)
    ref = torch.softmax(z, -1) @ s["v"].double().repeat_interleave(Hq // Hkv, 1)
    # q and k round once to bf16 (2^-8): the score moves by at most 2 * 2^-8 |q| |k| / sqrt(d), in the mean over
    # 128 products about 2^-8; the forward's own bar is 1e-2 on values of order one
    assert float((got - ref).abs().max()) <= 2e-2


def test_append_captured_and_replayed():
    s = make(2, 2, 1, 4, 128, 128, None, [20, 90], None, seed=111)
    inv, _ = fa.rope_frequencies(128)
    kc, vc, q = dev(s["kc"]), dev(s["vc"]), dev(s["q"])
    k, v, table, lens, out = dev(s["k"]), dev(s["v"]), dev(s["table"]), dev(s["lens"]), torch.empty_like(q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fa.kv_append(k, v, kc, vc, table, lens, inv_freq=inv, q=q, q_out=out)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            fa.kv_append(k, v, kc, vc, table, lens, inv_freq=inv, q=q, q_out=out)
            turned_k, _ = fa.rope(k, inv, pos0=5)
    k.copy_(torch.randn(k.shape, device="cuda"))
    lens.add_(7)  # what a replay reads is what the tensors hold then
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want_k, want_v, want_q = dev(s["kc"]), dev(s["vc"]), torch.empty_like(q)
    fa.kv_append(k, v, want_k, want_v, table, dev(s["lens"]), inv_freq=inv, q=q, q_out=want_q)  # the first call's rows
    fa.kv_append(k, v, want_k, want_v, table, lens, inv_freq=inv, q=q, q_out=want_q)
    new = [int(lens[b]) - 4 + i for b in range(2) for i in range(4)]
    for j, at in enumerate(new):
        blk = int(table[j // 4, at // 64])
        assert torch.equal(kc[blk, :, at % 64], want_k[blk, :, at % 64])
    assert torch.equal(out, want_q)
    assert torch.equal(turned_k, fa.rope(k, inv, pos0=5)[0])
