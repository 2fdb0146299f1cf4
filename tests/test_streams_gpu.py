"""Calls on a given stream beside work that is still queued on the current one."""
import pytest
import torch

from attention_attn_fwd_11_b200 import fa

pytestmark = pytest.mark.gpu

LONG = 40_000_000  # clock cycles: some 20 ms


def rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def calls():  # (inputs are made here, before anything is queued: the given stream does not wait for them)
    q, k, v, do = rand(1, 5, 300, 128), rand(1, 1, 70, 128, seed=1), rand(1, 1, 70, 128, seed=2), rand(1, 5, 300, 128, seed=3)
    o, lse = fa.fwd(q, k, v)
    inv, _ = fa.rope_frequencies(128)
    cache, other = rand(8, 2, 64, 128, seed=4), rand(8, 2, 64, 128, seed=5)
    table = torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
    lens = torch.tensor([200, 130], device="cuda", dtype=torch.int32)
    q3, q4 = rand(2, 4, 128, seed=6), rand(2, 4, 9, 128, seed=7)
    new = rand(2, 2, 9, 128, seed=8)
    blocks = torch.randint(0, 100, (1, 2, 200, 136), device="cuda", dtype=torch.uint8)
    blocks.unflatten(-1, (4, 34))[..., 1] = 0x2c  # scales of 0.06 or so
    lat, rows = rand(3, 128, 576, seed=9), rand(128, 576, seed=10)
    w = rand(4, 128, 512, seed=11), rand(256, 512, seed=12)
    q5, latent, k2 = rand(1, 4, 77, 128, seed=13), rand(5, 4, 512, seed=14), rand(1, 1, 300, 128, seed=15)
    return {
        "fwd": lambda **kw: fa.fwd(q, k, v, **kw), "bwd": lambda **kw: fa.bwd(q, k, v, o, lse, do, **kw),
        "decode_paged": lambda **kw: fa.decode_paged(q3, cache, other, table, lens, num_splits=4, **kw),
        "prefill_paged": lambda **kw: fa.prefill_paged(q4, cache, other, table, lens, **kw),
        "prefill_latent": lambda **kw: fa.prefill_latent(lat, rows, num_splits=2, **kw),
        "kv_dequant": lambda **kw: fa.kv_dequant(blocks, "q8_0", 128, **kw),
        "fwd_quant": lambda **kw: fa.fwd_quant(q5, blocks, blocks, "q8_0", 128, 128, **kw),
        "mla_tail": lambda **kw: fa.mla_tail(latent, *w, **kw),
        "rope": lambda **kw: fa.rope(q, inv, k=k2, **kw),
        "kv_append": lambda **kw: fa.kv_append(new, new, cache, other, table, lens, inv_freq=inv, q=q4, **kw),
    }


NAMES = ["fwd", "bwd", "decode_paged", "prefill_paged", "prefill_latent", "kv_dequant", "fwd_quant", "mla_tail", "rope",
         "kv_append"]


def flat(x):
    return [t for t in (x if isinstance(x, (tuple, list)) else (x,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_blocks_that_the_current_stream_still_writes(name):
    """Blocks of every size are written by queued work and freed: none of them may come back inside the call, whose
    kernels run long before that work does."""
    call = calls()[name]
    want = flat(call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sizes = sorted({t.numel() * t.element_size() for t in want} | {512, 4096, 1 << 16, 1 << 18, 1 << 20, 1 << 21, 1 << 23})
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda._sleep(LONG)
    for t in blocks:
        t.fill_(90)
    del blocks, t
    got = flat(call(stream=side))
    side.synchronize()
    torch.cuda.synchronize()
    assert fa.device_error() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_results_used_on_the_callers_stream_and_let_go(name):
    """A later call on the same stream may not get a block that queued work of the caller still reads."""
    call = calls()[name]
    want = flat(call())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = flat(call(stream=side))
    side.synchronize()
    torch.cuda._sleep(LONG)
    copies = [t.clone() for t in got]  # queued on the current stream
    with torch.cuda.stream(side):
        sizes = [t.numel() * t.element_size() for t in got]
        del got
        others = [torch.full((n,), 90, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)
    assert all(bool((t == 90).all()) for t in others)


def test_on_a_stream_that_a_capture_forks():
    q, k, v, do = rand(1, 4, 200, 128), rand(1, 2, 200, 128, seed=1), rand(1, 2, 200, 128, seed=2), rand(1, 4, 200, 128, seed=3)
    inv, _ = fa.rope_frequencies(128)
    fork = torch.cuda.Stream()

    def step(stream):
        qr, kr = fa.rope(q, inv, k=k, **stream)
        o, lse = fa.fwd(qr, kr, v, **stream)
        return [o, lse, *fa.bwd(qr, kr, v, o, lse, do, **stream)]

    want = step({})
    step(dict(stream=fork))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fork.wait_stream(torch.cuda.current_stream())
        got = step(dict(stream=fork))
        torch.cuda.current_stream().wait_stream(fork)
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
