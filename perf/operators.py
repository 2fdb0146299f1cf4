"""What is measured of the training and serving operators beside the
attention forward: its backward pass (`fa.bwd`), rotary positions and their
gradient (`fa.rope`), and the write of new rows into a paged cache with the
rotation fused in (`fa.kv_append`).

`own` chooses between the operators' plain form (elementary torch operations,
32 bits, rounded once at the end) and the framework's calls.
"""
import math
import random

import torch

own = False

BLOCK = 64  # slots of a cache block
DEV = "cuda"


# -------------------------------------------------------------------- cases --

def listed():
    bwd = dict(op="bwd", mods=False, o_bf16=True, seq_major=False)
    app = dict(op="append", interleaved=False, rot=128, rope=True, with_q=True, min_len=1)
    return [
        # the smallest training call: two heads of a short full attention, where latency counts
        dict(bwd, name="bwd_tiny_full", B=1, Hq=2, Hkv=2, Sq=256, Sk=256, dk=64, dv=64, causal=False, o_bf16=False),
        # the framework's headline shape, as a training step runs it
        dict(bwd, name="bwd_causal_mha", B=2, Hq=16, Hkv=16, Sq=2048, Sk=2048, dk=128, dv=128, causal=True),
        # one long sequence with four query heads to a key head: the gradients of shared heads
        dict(bwd, name="bwd_causal_gqa", B=1, Hq=32, Hkv=8, Sq=4096, Sk=4096, dk=128, dv=128, causal=True),
        # ragged lengths, more keys than queries (a continued sequence), sequence-major storage
        dict(bwd, name="bwd_ragged", B=3, Hq=6, Hkv=2, Sq=517, Sk=1291, dk=64, dv=64, causal=True, seq_major=True),
        # a mask with padded keys and empty rows, ALiBi, a softcap and sinks
        dict(bwd, name="bwd_modifiers", B=2, Hq=8, Hkv=8, Sq=1024, Sk=1024, dk=128, dv=128, causal=False, mods=True),
        # heads with a rotary part beside the plain one: wider keys than values
        dict(bwd, name="bwd_dk192_dv128", B=2, Hq=16, Hkv=16, Sq=2048, Sk=2048, dk=192, dv=128, causal=True),
        # queries and keys of a prefill, scaled for contexts 8 times as long
        dict(op="rope", name="rope_prefill", B=2, Hq=32, Hkv=8, S=4096, d=128, rot=128, offset=0, interleaved=False,
             inverse=False, f32=False, factor=8.0, max_pos=131072),
        # the gradient: the last 64 of 192 columns, interleaved pairs, 32-bit gradients
        dict(op="rope", name="rope_gradient_f32", B=1, Hq=16, Hkv=0, S=2048, d=192, rot=64, offset=128,
             interleaved=True, inverse=True, f32=True, factor=1.0, max_pos=16384),
        # one new token for each of 64 sequences, as before a decode step
        dict(app, name="append_decode_bf16", B=64, Hq=32, Hkv=8, Sq=1, d=128, kv="bf16", max_len=512, ragged=False),
        # chunks of 512 new rows behind long sequences, as before a chunked prefill
        dict(app, name="append_chunk_bf16", B=16, Hq=32, Hkv=8, Sq=512, d=128, kv="bf16", max_len=4096, ragged=False),
        # chunks of unequal length into an 8-bit cache
        dict(app, name="append_ragged_fp8", B=8, Hq=16, Hkv=4, Sq=333, d=128, kv="fp8_e4m3", max_len=2048,
             ragged=True),
        # a prefill into a cache of 32-value blocks, read back as the values it holds
        dict(app, name="append_q8_0", B=4, Hq=16, Hkv=8, Sq=1024, d=128, kv="q8_0", max_len=1100, ragged=False,
             with_q=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["bwd", "bwd", "rope", "append"])
    if op == "bwd":
        dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
        Hkv, G, B = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 4, 7]), rng.randint(1, 3)
        Sq = _log_int(rng, 16, 4096)
        Sk = Sq if rng.random() < 0.5 else _log_int(rng, 16, 4096)
        while B > 1 and B * Hkv * G * Sq * Sk > 2 ** 27:
            B -= 1
        while B * Hkv * G * Sq * Sk > 2 ** 27:
            Sq, Sk = max(1, Sq * 3 // 4), max(1, Sk * 3 // 4)
        return dict(op="bwd", B=B, Hq=Hkv * G, Hkv=Hkv, Sq=Sq, Sk=Sk, dk=dk, dv=dv, causal=rng.random() < 0.6,
                    mods=dk == dv and rng.random() < 0.25, o_bf16=rng.random() < 0.5, seq_major=rng.random() < 0.5)
    if op == "rope":
        d = rng.choice([64, 96, 128, 192, 256])
        rot = rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= d])
        return dict(op="rope", B=rng.randint(1, 4), Hq=rng.choice([1, 8, 12, 32]), Hkv=rng.choice([0, 1, 8]),
                    S=_log_int(rng, 1, 1024), d=d, rot=rot, offset=rng.choice([0, d - rot]),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, f32=rng.random() < 0.3,
                    factor=rng.choice([1.0, 4.0, 32.0]), max_pos=rng.choice([4096, 131072, 1048576]))
    kv = rng.choice(["bf16", "bf16", "fp8_e4m3", "q8_0", "q4_0"])
    d = rng.choice([64, 128, 256]) if kv == "bf16" else 128
    Hkv, rope = rng.choice([1, 2, 4, 8]), kv != "q4_0" and rng.random() < 0.8
    B, Sq = _log_int(rng, 1, 32), _log_int(rng, 1, 512)
    while B * Sq > 4096:
        B = max(1, B // 2)
    return dict(op="append", B=B, Hq=Hkv * rng.choice([1, 4, 5]), Hkv=Hkv, Sq=Sq, d=d, kv=kv,
                max_len=Sq + _log_int(rng, 1, 1024), min_len=1, ragged=rng.random() < 0.5, rope=rope,
                with_q=rope and rng.random() < 0.7, rot=d if rng.random() < 0.7 else 64,
                interleaved=rng.random() < 0.3)


# ------------------------------------------------------------------- inputs --

def _frequencies(rot, factor):
    """Angular frequencies of rot / 2 pairs in 64 bits, and the factor on cos
    and sin: base 10000, for factor > 1 interpolated by parts (slow pairs by
    the whole factor, fast ones not at all, a ramp between)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    inv = 10000.0 ** (-2.0 * i / rot)
    if factor == 1.0:
        return inv, 1.0
    turn = lambda n: rot * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    low, high = max(0, math.floor(turn(32))), min(rot - 1, math.ceil(turn(1)))
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return inv / factor * ramp + inv * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _randn(g, shape, dtype, seq_major=False, scale=1.0):
    if seq_major:  # [B, S, H, d] storage seen as [B, H, S, d]
        b, h, s, d = shape
        return (torch.randn((b, s, h, d), generator=g, device=DEV) * scale).to(dtype).transpose(1, 2)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _slopes(Hq, max_bias):
    n = 1 << (Hq.bit_length() - 1)
    m0, m1 = 2.0 ** (-max_bias / n), 2.0 ** (-max_bias / 2 / n)
    return [m0 ** (h + 1) if h < n else m1 ** (2 * (h - n) + 1) for h in range(Hq)]


def _visible(c, dev):
    i = torch.arange(c["Sq"], device=dev)[:, None]
    j = torch.arange(c["Sk"], device=dev)[None, :]
    return j <= i + c["Sk"] - c["Sq"]


def _prepare_bwd(c, g):
    B, Hq, Hkv, Sq, Sk = c["B"], c["Hq"], c["Hkv"], c["Sq"], c["Sk"]
    sm = c["seq_major"]
    s = dict(case=c, scale=1.0 / math.sqrt(c["dk"]), mask=None, max_bias=0.0, softcap=0.0, sinks=None)
    s["q"] = _randn(g, (B, Hq, Sq, c["dk"]), torch.bfloat16, sm)
    s["k"] = _randn(g, (B, Hkv, Sk, c["dk"]), torch.bfloat16, sm)
    s["v"] = _randn(g, (B, Hkv, Sk, c["dv"]), torch.bfloat16, sm)
    s["do"] = _randn(g, (B, Hq, Sq, c["dv"]), torch.bfloat16, sm)
    if c["mods"]:
        # distances for ALiBi, the last keys of each batch entry padded away, a few rows that see nothing
        pad = (Sk + 7) // 8 * 8
        i = torch.arange(Sq, device=DEV)[:, None]
        j = torch.arange(pad, device=DEV)[None, :]
        m = (-(i + Sk - Sq - j).abs().float()).expand(B, 1, Sq, pad).clone()
        keep = torch.randint(max(1, Sk // 2), Sk + 1, (B,), generator=g, device=DEV)
        m.masked_fill_((j >= keep[:, None, None])[:, None], -math.inf)
        m[:, :, 3::97] = -math.inf
        s["mask"] = m.to(torch.float16)[..., :Sk]
        s["max_bias"], s["softcap"] = 8.0, 20.0
        s["scale"] /= s["softcap"]  # softcap * tanh(q.k / (sqrt(d) * softcap))
        s["sinks"] = torch.randn(Hq, generator=g, device=DEV)
    # the forward pass whose gradient is asked for: its output and log-sum-exp
    z, p = _scores(s, s["q"].float(), s["k"].float())
    lse = torch.logsumexp(p, -1) if s["sinks"] is None else torch.logsumexp(
        torch.cat([p, s["sinks"].view(1, Hq, 1, 1).expand(B, Hq, Sq, 1)], -1), -1)
    w = torch.where(p > -math.inf, torch.exp(p - lse[..., None]), 0.0)
    o = w @ s["v"].float().repeat_interleave(Hq // Hkv, 1)
    s["o"] = o.to(torch.bfloat16 if c["o_bf16"] else torch.float32)
    if sm:
        s["o"] = s["o"].transpose(1, 2).contiguous().transpose(1, 2)
    s["lse"] = lse.contiguous()
    return s


def _prepare_rope(c, g):
    B, S, d, t = c["B"], c["S"], c["d"], torch.float32 if c["f32"] else torch.bfloat16
    inv, m = _frequencies(c["rot"], c["factor"])
    start = torch.randint(0, max(1, c["max_pos"] - S), (B, 1), generator=g, device=DEV)
    return dict(case=c, q=_randn(g, (B, c["Hq"], S, d), t), k=_randn(g, (B, c["Hkv"], S, d), t) if c["Hkv"] else None,
                pos=(start + torch.arange(S, device=DEV)).to(torch.int32), inv=inv, inv_dev=inv.to(DEV), mscale=m)


def _prepare_append(c, g):
    B, Hq, Hkv, Sq, d, kv = c["B"], c["Hq"], c["Hkv"], c["Sq"], c["d"], c["kv"]
    n = torch.randint(0, Sq + 1, (B,), generator=g, device=DEV) if c["ragged"] else torch.full((B,), Sq, device=DEV)
    old = torch.randint(c["min_len"] - 1, max(c["min_len"], c["max_len"] - Sq + 1), (B,), generator=g, device=DEV)
    width = -(-c["max_len"] // BLOCK)
    nb = B * width
    table = torch.randperm(nb, generator=g, device=DEV).to(torch.int32).view(B, width).contiguous()
    s = dict(case=c, table=table, lens=(old + n).to(torch.int32), n=n.to(torch.int32) if c["ragged"] else None,
             k=_randn(g, (B, Hkv, Sq, d), torch.bfloat16, True), v=_randn(g, (B, Hkv, Sq, d), torch.bfloat16, True),
             q=_randn(g, (B, Hq, Sq, d), torch.bfloat16, True) if c["with_q"] else None, ks=1.0, vs=1.0)
    s["inv"], s["mscale"] = _frequencies(c["rot"], 4.0) if c["rope"] else (None, 1.0)
    s["inv_dev"] = s["inv"].to(DEV) if c["rope"] else None
    if kv == "fp8_e4m3":
        s["ks"], s["vs"] = 0.0175, 0.0125
    for name in ("kc", "vc"):
        rows = torch.randn((nb, Hkv, BLOCK, d), generator=g, device=DEV)
        s[name] = _encode(rows, kv, s["ks" if name == "kc" else "vs"])
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"bwd": _prepare_bwd, "rope": _prepare_rope, "append": _prepare_append}[case["op"]](case, g)


# -------------------------------------------------------------- plain forms --

def _scores(s, q, k):
    """(q k^T * scale, those scores after the modifiers), hidden keys at -inf."""
    c = s["case"]
    z = q @ k.repeat_interleave(c["Hq"] // c["Hkv"], 1).transpose(-1, -2) * s["scale"]
    p = z
    if s["softcap"]:
        p = s["softcap"] * torch.tanh(p)
    if s["mask"] is not None:
        slope = torch.tensor(_slopes(c["Hq"], s["max_bias"]) if s["max_bias"] else [1.0] * c["Hq"], device=DEV)
        p = p + slope.to(p.dtype).view(1, -1, 1, 1) * s["mask"].to(p.dtype)
    if c["causal"]:
        p = p.masked_fill(~_visible(c, q.device), -math.inf)
    return z, p


def _plain_bwd(s):
    c = s["case"]
    B, Hq, Hkv, Sq, Sk = c["B"], c["Hq"], c["Hkv"], c["Sq"], c["Sk"]
    q, k, v, do = (s[n].float() for n in ("q", "k", "v", "do"))
    z, p = _scores(s, q, k)
    lse = s["lse"][..., None]
    w = torch.where((p > -math.inf) & (lse > -math.inf), torch.exp(p - lse), 0.0)
    delta = (do * s["o"].float()).sum(-1, keepdim=True)
    dp = do @ v.repeat_interleave(Hq // Hkv, 1).transpose(-1, -2)
    ds = w * (dp - delta)
    if s["softcap"]:
        ds = ds * (s["softcap"] * (1 - torch.tanh(z) ** 2))
    ds = ds * s["scale"]
    dq = ds @ k.repeat_interleave(Hq // Hkv, 1)
    dk = (ds.transpose(-1, -2) @ q).view(B, Hkv, Hq // Hkv, Sk, -1).sum(2)
    dv = (w.transpose(-1, -2) @ do).view(B, Hkv, Hq // Hkv, Sk, -1).sum(2)
    out = [t.to(torch.bfloat16) for t in (dq, dk, dv)]
    if s["sinks"] is not None:
        ps = torch.where(lse > -math.inf, torch.exp(s["sinks"].view(1, Hq, 1, 1) - lse), 0.0)
        out.append(-(ps.double() * delta.double()).sum((0, 2, 3)).float())
    return out


def _rotate(x, pos, inv, mscale, interleaved, offset, inverse):
    """Pairs of x [B, H, S, d] turned by pos [B, S] * inv; 32 bits, angles in 64."""
    rot = 2 * inv.numel()
    a = pos.double()[..., None] * inv
    cos, sin = (torch.cos(a) * mscale).float()[:, None], (torch.sin(a) * mscale).float()[:, None]
    if inverse:
        sin = -sin
    x = x.float()
    y = x.clone()
    part = x[..., offset:offset + rot]
    if interleaved:
        u, w = part[..., 0::2], part[..., 1::2]
        y[..., offset:offset + rot:2] = u * cos - w * sin
        y[..., offset + 1:offset + rot:2] = w * cos + u * sin
    else:
        u, w = part[..., :rot // 2], part[..., rot // 2:]
        y[..., offset:offset + rot // 2] = u * cos - w * sin
        y[..., offset + rot // 2:offset + rot] = w * cos + u * sin
    return y


def _plain_rope(s):
    c = s["case"]
    out = [_rotate(x, s["pos"], s["inv_dev"], s["mscale"], c["interleaved"], c["offset"], c["inverse"]).to(x.dtype)
           for x in (s["q"], s["k"]) if x is not None]
    return out


def _encode(x, kv, scale):
    """Rows of a cache of type `kv` from 32-bit values [..., d]."""
    if kv == "bf16":
        return x.to(torch.bfloat16)
    if kv == "fp8_e4m3":
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    b = x.unflatten(-1, (-1, 32))
    if kv == "q8_0":  # scale = the largest magnitude / 127 in 16 bits; codes to the nearest, ties to even
        d = (b.abs().amax(-1, keepdim=True) / 127).to(torch.float16)
        q = torch.where(d == 0, 0.0, (b / d.float()).round().clamp(-127, 127)).to(torch.int8).view(torch.uint8)
    else:  # q4_0: scale = the first value of largest magnitude / -8; value j and j + 16 share a byte
        d = (b.gather(-1, b.abs().argmax(-1, keepdim=True)) / -8).to(torch.float16)
        n = torch.where(d == 0, 0.0, (b / d.float()).round().clamp(-8, 7)).to(torch.int32) + 8
        q = (n[..., :16] + 16 * n[..., 16:]).to(torch.uint8)
    return torch.cat([d.view(torch.uint8), q], -1).flatten(-2)


def _values(cache, kv):
    """What a cache holds, as floating values (bf16 for the blocks of 32)."""
    if kv == "bf16":
        return cache
    if kv == "fp8_e4m3":
        return cache.view(torch.float8_e4m3fn)
    b = cache.unflatten(-1, (-1, 34 if kv == "q8_0" else 18))
    d = b[..., :2].contiguous().view(torch.float16).float()
    if kv == "q8_0":
        q = b[..., 2:].contiguous().view(torch.int8).float()
    else:
        q = torch.cat([b[..., 2:] & 15, b[..., 2:] >> 4], -1).float() - 8
    return (d * q).flatten(-2).to(torch.bfloat16)


def _new_rows(s):
    """For the rows that are there: (batch entry, row, block, slot), and the position of every row."""
    c = s["case"]
    n = s["n"] if s["n"] is not None else torch.full_like(s["lens"], c["Sq"])
    i = torch.arange(c["Sq"], device=DEV)[None, :]
    pos = s["lens"][:, None] - n[:, None] + i
    live = i < n[:, None]
    b, r = live.nonzero(as_tuple=True)
    at = pos[b, r].long()
    return b, r, s["table"][b, at // BLOCK].long(), at % BLOCK, pos, live


def _plain_append(s):
    c = s["case"]
    b, r, block, slot, pos, live = _new_rows(s)
    turn = lambda x: _rotate(x, pos, s["inv_dev"], s["mscale"], c["interleaved"], 0, False)  # noqa: E731
    k = turn(s["k"]) if c["rope"] else s["k"].float()
    s["kc"][block, :, slot] = _encode(k[b, :, r], c["kv"], s["ks"])
    s["vc"][block, :, slot] = _encode(s["v"].float()[b, :, r], c["kv"], s["vs"])
    out = [_values(s["kc"], c["kv"]), _values(s["vc"], c["kv"])]
    if s["q"] is not None:
        out.append((turn(s["q"]) * live[:, None, :, None]).to(torch.bfloat16))
    return out


# ---------------------------------------------------------- framework's form --

def _own_bwd(s):
    from attention_attn_fwd_11_b200 import fa
    c = s["case"]
    return list(fa.bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], scale=s["scale"], causal=c["causal"],
                       mask=s["mask"], max_bias=s["max_bias"], softcap=s["softcap"], sinks=s["sinks"]))


def _own_rope(s):
    from attention_attn_fwd_11_b200 import fa
    c = s["case"]
    q, k = fa.rope(s["q"], s["inv"], k=s["k"], pos=s["pos"], interleaved=c["interleaved"], offset=c["offset"],
                   inverse=c["inverse"], mscale=s["mscale"])
    return [q] if k is None else [q, k]


def _own_append(s):
    from attention_attn_fwd_11_b200 import fa
    c = s["case"]
    kv = c["kv"]
    q = fa.kv_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], q_lens=s["n"], inv_freq=s["inv"],
                     mscale=s["mscale"], interleaved=c["interleaved"], q=s["q"],
                     kv_type=None if kv == "bf16" else kv, k_scale=s["ks"], v_scale=s["vs"])
    if kv in ("q8_0", "q4_0"):
        out = fa.kv_dequant_many([(s["kc"], kv, c["d"], None), (s["vc"], kv, c["d"], None)])
    else:
        out = [_values(s["kc"], kv), _values(s["vc"], kv)]
    return out + [q] if q is not None else out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"bwd": _own_bwd, "rope": _own_rope, "append": _own_append}[op](state)
    return {"bwd": _plain_bwd, "rope": _plain_rope, "append": _plain_append}[op](state)


# --------------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] == "bwd":
        B, Hq, Hkv, Sq, Sk, dk, dv = (c[n] for n in ("B", "Hq", "Hkv", "Sq", "Sk", "dk", "dv"))
        pairs = Sq * Sk
        if c["causal"]:
            pairs = sum(min(Sk, max(0, i + Sk - Sq + 1)) for i in range(Sq))
        rows = B * Hq * Sq * ((2 * dk + dv) * 2 + dv * (2 if c["o_bf16"] else 4) + 4)
        keys = B * Hkv * Sk * (dk + dv) * 4
        return {"bytes": rows + keys + (B * Sq * Sk * 2 if c["mods"] else 0),
                "flops": 2 * B * Hq * pairs * (3 * dk + 2 * dv)}
    if c["op"] == "rope":
        e = c["B"] * (c["Hq"] + c["Hkv"]) * c["S"] * c["d"]
        return {"bytes": e * (8 if c["f32"] else 4) + 4 * c["B"] * c["S"], "flops": 3 * e}
    per = {"bf16": 2.0, "fp8_e4m3": 1.0, "q8_0": 34 / 32, "q4_0": 18 / 32}[c["kv"]]
    rows = c["B"] * c["Sq"] * (0.5 if c["ragged"] else 1.0)
    e = rows * c["Hkv"] * c["d"]
    got = 2 * e * (2 + per) + (rows * c["Hq"] * c["d"] * 4 if c["with_q"] else 0)
    if c["kv"] in ("q8_0", "q4_0"):  # read back as the values it holds
        got += 2 * c["B"] * -(-c["max_len"] // BLOCK) * BLOCK * c["Hkv"] * c["d"] * (per + 2)
    return {"bytes": got, "flops": 6 * e}


# -------------------------------------------------------------------- exact --

def _exact_bwd(s):
    """dS_ij = P_ij (dO_i . V_j - dO_i . O_i) dz_ij, one head at a time."""
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    dq = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    dk = torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV)
    dv = torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
    dsink = torch.zeros(c["Hq"], dtype=torch.float64, device=DEV)
    slopes = _slopes(c["Hq"], s["max_bias"]) if s["max_bias"] else [1.0] * c["Hq"]
    hidden = ~_visible(c, DEV) if c["causal"] else None
    for b in range(c["B"]):
        for h in range(c["Hq"]):
            q, do, o = s["q"][b, h].double(), s["do"][b, h].double(), s["o"][b, h].double()
            k, v, lse = s["k"][b, h // G].double(), s["v"][b, h // G].double(), s["lse"][b, h].double()
            x = torch.mm(q, k.T).mul_(s["scale"])
            slope_of_cap = None
            if s["softcap"]:
                t = torch.tanh(x)
                slope_of_cap = s["softcap"] * (1 - t * t)
                x = s["softcap"] * t
            if s["mask"] is not None:
                x = x + s["mask"][b, 0].double() * slopes[h]
            if hidden is not None:
                x[hidden] = -math.inf
            lse = torch.where(lse == -math.inf, math.inf, lse)
            p = torch.exp(x - lse[:, None])
            dv[b, h // G] += torch.mm(p.T, do)
            row = (do * o).sum(1)
            d = torch.mm(do, v.T).sub_(row[:, None]).mul_(p)
            if slope_of_cap is not None:
                d *= slope_of_cap
            d *= s["scale"]
            dq[b, h] = torch.mm(d, k)
            dk[b, h // G] += torch.mm(d.T, q)
            if s["sinks"] is not None:
                dsink[h] -= (torch.exp(s["sinks"][h].double() - lse) * row).sum()
    return [dq, dk, dv] + ([dsink] if s["sinks"] is not None else [])


def _exact_turn(x, pos, inv, mscale, interleaved, offset, inverse):
    """Complex multiplication of each pair by mscale * exp(+-i pos inv)."""
    x = x.double().clone()
    m = inv.numel()
    unit = torch.polar(torch.full((), mscale, dtype=torch.float64, device=DEV).expand(*pos.shape, m).contiguous(),
                       (-1.0 if inverse else 1.0) * pos.double()[..., None] * inv)[:, None]
    part = x[..., offset:offset + 2 * m]
    pairs = part.unflatten(-1, (m, 2)) if interleaved else part.unflatten(-1, (2, m)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
    x[..., offset:offset + 2 * m] = (turned if interleaved else turned.transpose(-1, -2)).flatten(-2)
    return x


def _exact_append(s):
    c = s["case"]
    n = s["n"].tolist() if s["n"] is not None else [c["Sq"]] * c["B"]
    lens, table = s["lens"].tolist(), s["table"].long()
    first = torch.tensor([a - b for a, b in zip(lens, n)], device=DEV)
    pos = first[:, None] + torch.arange(c["Sq"], device=DEV)
    turn = lambda x: _exact_turn(x, pos, s["inv_dev"], s["mscale"], c["interleaved"], 0, False)  # noqa: E731
    out = []
    for rows, cache, scale in ((turn(s["k"]) if c["rope"] else s["k"].double(), s["kc"], s["ks"]),
                               (s["v"].double(), s["vc"], s["vs"])):
        got = _values(cache, c["kv"]).double()
        if c["kv"] == "fp8_e4m3":
            new = (rows / scale).clamp(-448, 448)
        elif c["kv"] in ("q8_0", "q4_0"):
            b = rows.unflatten(-1, (-1, 32))
            if c["kv"] == "q8_0":
                step, lo, hi = b.abs().amax(-1, keepdim=True) / 127, -127, 127
            else:
                step, lo, hi = b.gather(-1, b.abs().argmax(-1, keepdim=True)) / -8, -8, 7
            step = step.half().double()
            new = torch.where(step == 0, 0.0, (b / step).round().clamp(lo, hi) * step).flatten(-2)
        else:
            new = rows
        for e in range(c["B"]):
            p = first[e] + torch.arange(n[e], device=DEV)
            got[table[e, p // BLOCK], :, p % BLOCK] = new[e, :, :n[e]].transpose(0, 1)
        out.append(got)
    if s["q"] is not None:
        live = torch.arange(c["Sq"], device=DEV)[None, :] < torch.tensor(n, device=DEV)[:, None]
        out.append(turn(s["q"]) * live[:, None, :, None])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "bwd":
        return _exact_bwd(s)
    if case["op"] == "rope":
        return [_exact_turn(x, s["pos"], s["inv_dev"], s["mscale"], case["interleaved"], case["offset"],
                            case["inverse"]) for x in (s["q"], s["k"]) if x is not None]
    return _exact_append(s)
