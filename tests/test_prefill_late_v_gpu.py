"""K and Q in the caches, V not: its loads come long after the first scores, and O may not be read before they are used."""
import math

import pytest
import torch

from attention_attn_fwd_11_b200 import fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128), (192, 192), (256, 256), (320, 256), (576, 512), (512, 512)])
@pytest.mark.parametrize("sk", [100, 128, 200, 300])
def test_cold_values(dk, dv, sk):
    g = torch.Generator(device="cuda").manual_seed(sk)
    q, k, v = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((1, 2, 200, dk), (1, 2, sk, dk), (1, 2, sk, dv)))
    flush = torch.empty(1 << 29, dtype=torch.uint8, device="cuda")  # four times the L2 cache
    kinds = [dict(causal=False), dict(causal=True)]
    if dk < 512:
        kinds.append(dict(causal=False, softcap=20.0))
    for kw in kinds:
        kw["scale"] = 1 / math.sqrt(dk) / kw.get("softcap", 1.0)
        s = q.double() @ k.double().transpose(-1, -2) * kw["scale"]
        if "softcap" in kw:
            s = 20 * torch.tanh(s)
        if kw["causal"]:
            s = s.masked_fill(torch.arange(sk, device="cuda") > torch.arange(200, device="cuda")[:, None] + sk - 200, -math.inf)
        p = torch.softmax(s, -1)
        ref = torch.where(s.isinf().all(-1, keepdim=True), 0.0, p) @ v.double()
        want, _ = fa.fwd(q, k, v, **kw)
        # P rounds to bf16 (2^-8 of itself) and is summed with |V| below 5; the softmax's own error is far below that
        assert float((want.double() - ref).abs().max()) <= 2.0 ** -8 * 5
        for _ in range(10):
            flush.fill_(1)
            q.add_(0), k.add_(0)  # back in L2
            got, _ = fa.fwd(q, k, v, **kw)
            assert torch.equal(got, want)
