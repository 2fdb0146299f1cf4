"""Views of one buffer that lie beside one another are taken; outputs that share memory are refused."""
import pytest
import torch

from attention_attn_fwd_11_b200 import fa

pytestmark = pytest.mark.gpu


def fused(B=2, S=37, Hq=4, Hkv=2, d=128, dtype=torch.bfloat16):
    """A projection [B, S, (Hq + 2 Hkv) d] and its q, k, v as [B, H, S, d] views."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((B, S, Hq + 2 * Hkv, d), generator=g, device="cuda").to(dtype)
    return x, [t.transpose(1, 2) for t in x.split((Hq, Hkv, Hkv), 2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_in_place_inside_one_projection(dtype):
    x, (q, k, v) = fused(dtype=dtype)
    inv, _ = fa.rope_frequencies(128)
    want = fa.rope(q.contiguous(), inv, k=k.contiguous(), pos0=9)
    vs = v.clone()
    fa.rope(q, inv, k=k, pos0=9, out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, vs)


def test_rope_between_projections_and_with_reversed_roles():
    x, (q, k, v) = fused()
    y, (qo, ko, vo) = fused()
    inv, _ = fa.rope_frequencies(128)
    want = fa.rope(q, inv, k=k)
    for out, k_out in ((qo, ko), (qo, vo), (v.new_empty(q.shape), v)):  # v: an output beside the inputs
        fa.rope(q, inv, k=k, out=out, k_out=k_out)
        assert torch.equal(out, want[0]) and torch.equal(k_out, want[1])


def test_append_with_q_turned_inside_the_projection():
    x, (q, k, v) = fused()
    inv, _ = fa.rope_frequencies(128)
    table, lens = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda"), torch.tensor([37, 50], dtype=torch.int32, device="cuda")
    both = torch.zeros((2, 2, 2, 64, 128), device="cuda", dtype=torch.bfloat16)  # the caches of K and V in one buffer
    apart = [torch.zeros((2, 2, 64, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    want = fa.kv_append(k, v, *apart, table, lens, inv_freq=inv, q=q)
    fa.kv_append(k, v, both[0], both[1], table, lens, inv_freq=inv, q=q, q_out=q)
    assert torch.equal(q, want) and torch.equal(both[0], apart[0]) and torch.equal(both[1], apart[1])
    assert fa.device_error() == 0


def test_outputs_that_share_memory_are_refused():
    x, (q, k, v) = fused()
    inv, _ = fa.rope_frequencies(128)
    one = torch.empty(q.shape, device="cuda", dtype=q.dtype)
    flat = torch.empty(1 << 20, device="cuda", dtype=q.dtype)
    inside = flat.as_strided((2, 4, 37, 128), (4 * 37 * 128, 64, 512, 1))  # heads half a row apart
    before = x.clone()
    for kw in (dict(out=one, k_out=one[:, :2]), dict(out=one, k_out=one[:, 1:3]), dict(k_out=q[:, :2]), dict(out=x[:, :, 2:6].transpose(1, 2)),
               dict(out=inside), dict(out=flat[:q.numel()].view(q.shape), k_out=flat[64:64 + k.numel()].view(k.shape))):
        with pytest.raises(fa.FAError) as e:
            fa.rope(q, inv, k=k, **kw)
        assert e.value.status == fa.FA_ERR_INVALID_ARG
    cache, other = (torch.zeros((2, 2, 64, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table, lens = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda"), torch.tensor([37, 50], dtype=torch.int32, device="cuda")
    for kw in (dict(q_out=x[:, :, 1:5].transpose(1, 2)), dict(q_out=x[:, :, 3:7].transpose(1, 2)), dict(q_out=x[:, :, 4:].transpose(1, 2)),
               dict(v_cache=cache)):
        with pytest.raises(fa.FAError):
            fa.kv_append(**{**dict(k=k, v=v, k_cache=cache, v_cache=other, block_table=table, seq_lens=lens, inv_freq=inv, q=q), **kw})
    torch.cuda.synchronize()
    assert torch.equal(x, before) and not bool(cache.any())
