"""Calls on a given stream: what they make comes from that stream's memory, and what they use is kept for it.  Without a
GPU: stand-ins for the library, for torch's streams and for the tensors' device."""
import contextlib
import inspect
import types

import pytest
import torch

from attention_attn_fwd_11_b200 import fa

BF, I32 = torch.bfloat16, torch.int32


class Library:
    """Accepts every call, says which stream was current at the launch, and asks for a workspace of 512 bytes."""

    def __init__(self, now):
        self.now, self.launches = now, []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace_size") or name.endswith("_workspace_need"):
                args[1]._obj.value = 512
            else:
                self.launches.append((name, args[-1].value, self.now[0]))
            return fa.FA_OK
        return call


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def world(monkeypatch):
    outer, given = Stream(1), Stream(2)
    now = [outer]
    made, kept = [], []
    lib = Library(now)

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream
        try:
            yield
        finally:
            now[0] = before

    for name in ("empty", "empty_like", "arange"):
        def make(*a, _f=getattr(torch, name), **kw):
            kw.pop("device", None)
            t = _f(*a, **kw)
            made.append((t, now[0]))
            return t
        monkeypatch.setattr(torch, name, make)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[0])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: now[0].cuda_stream, raising=False)
    monkeypatch.setattr(fa, "load", lambda: lib)
    monkeypatch.setattr(fa, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(fa, "_need_current_device", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(fa, "_check_inv_freq", lambda t: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t, s)))
    return types.SimpleNamespace(outer=outer, given=given, made=made, kept=kept, lib=lib)


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def calls():
    q, k, q3 = z(1, 2, 3, 128), z(1, 2, 5, 128), z(1, 2, 128)
    o, lse = z(1, 2, 3, 128), z(1, 2, 3, dtype=torch.float32)
    cache, table, lens = z(2, 2, 64, 128), z(1, 2, dtype=I32), z(1, dtype=I32)
    inv, _ = fa.rope_frequencies(128)
    rows, lat = z(4, 576), z(2, 128, 576)
    q8 = z(1, 2, 5, 136, dtype=torch.uint8)
    return {
        "fwd": (q, k, k), "bwd": (q, k, k, o, lse, q), "decode_paged": (q3, cache, cache, table, lens),
        "prefill_paged": (q, cache, cache, table, lens), "decode_gather": (lat, rows, z(2, 4, dtype=I32)),
        "prefill_latent": (lat, rows), "kv_dequant": (q8, "q8_0", 128),
        "kv_dequant_many": ([(q8, "q8_0", 128, None), (q8, "q8_0", 128, None)],),
        "fwd_quant": (q, q8, q8, "q8_0", 128, 128), "mla_tail": (z(2, 4, 8), z(4, 6, 8), z(10, 24)),
        "rope": (q, inv, k[:, :, :3]), "kv_append": (q, q, cache, cache, table, lens, None, inv),
    }


def tensors(x):
    if isinstance(x, torch.Tensor):
        return [x]
    return [t for y in x for t in tensors(y)] if isinstance(x, (tuple, list)) else []


def test_every_call_with_a_stream_is_here():
    named = {n for n, f in vars(fa).items() if inspect.isfunction(f) and not n.startswith("_") and
             "stream" in inspect.signature(f).parameters}
    assert named == set(calls())


@pytest.mark.parametrize("name", sorted(calls()))
def test_on_a_given_stream(world, name):
    args = calls()[name]
    del world.made[:]
    got = getattr(fa, name)(*args, stream=world.given)
    assert world.lib.launches and all(h == 2 for _, h, _ in world.lib.launches)
    # A block of the outer stream's memory might still be in use by work queued there.
    assert all(s is world.given for _, s in world.made), "made on another stream than the kernels run on"
    kept = {(id(t), s) for t, s in world.kept}
    for t in tensors(got):
        if any(t is m for m, _ in world.made):
            assert (id(t), world.outer) in kept, "the caller's stream may go on with the results"
    for t in tensors(args):
        assert (id(t), world.given) in kept, "an input may be let go while the kernels still read it"


@pytest.mark.parametrize("name", sorted(calls()))
def test_on_the_current_stream(world, name):
    args = calls()[name]
    getattr(fa, name)(*args)
    assert world.lib.launches and all(h == 1 for _, h, _ in world.lib.launches) and not world.kept


def test_q_turned_for_a_given_stream(world):
    q, k, _, _, _, _ = calls()["bwd"]
    _, _, cache, _, table, lens, _, inv = calls()["kv_append"]
    del world.made[:]
    out = fa.kv_append(q, q, cache, cache, table, lens, inv_freq=inv, q=q, stream=world.given)
    assert [s for t, s in world.made if t is out] == [world.given]
    assert any(t is out and s is world.outer for t, s in world.kept)


def test_the_outer_stream_is_current_again_after_a_refusal(world):
    with pytest.raises(ValueError):
        fa.rope(z(2, 3), None, stream=world.given)
    assert torch.cuda.current_stream() is world.outer


@pytest.mark.parametrize("name", sorted(calls()))
def test_every_argument_reaches_the_call_on_the_stream(monkeypatch, name):
    seen = []
    monkeypatch.setattr(fa, "_on", lambda stream, call, *args, **kwargs: seen.append((stream, call, args, kwargs)))
    f = getattr(fa, name)
    names = [n for n, p in inspect.signature(f).parameters.items() if p.kind is not p.VAR_KEYWORD]
    given = {n: object() for n in names}
    if name == "fwd_quant":
        given["softcap"] = object()
    f(**given)
    (stream, call, args, kwargs), = seen
    got = inspect.signature(call).bind(*args, **kwargs).arguments
    got.update(got.pop("mods", {}))
    assert stream is given.pop("stream") and call is f and got.pop("stream", None) is None
    assert got == given
