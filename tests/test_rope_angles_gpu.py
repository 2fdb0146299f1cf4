"""How near the angles are.  A pair (1, 0) turned with mscale 1 is (cos a, sin a) itself: the products with 1 and 0 are exact.
The angle is off by at most 2.8e-8 radians (2.3e-8: half a step of the fp32 fraction below an eighth of a turn; 1.5e-9: the
fraction's 32 bits; 2.2e-9: the 64-bit frequency times 2^31), the sine and cosine of the angle taken by one unit of the
last place, at most 2^-23 of the value."""
import random
from fractions import Fraction

import pytest
import torch

from attention_attn_fwd_11_b200 import fa

pytestmark = pytest.mark.gpu

PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


def angle(pos, f):
    """pos * f less whole turns, in 64 bits; the turns are taken off in rational numbers."""
    x = pos * Fraction(f) / (2 * PI)
    return float((x - round(x)) * 2 * PI)


@pytest.mark.parametrize("inter", [False, True])
def test_angles(inter):
    rng, S = random.Random(5), 4096
    freq = [1.0, 0.5, 2.0 ** -20, 3.0, 6.28] + [10000.0 ** (-2 * i / 64) for i in range(11)]
    inv = torch.tensor(freq, dtype=torch.float64)
    pos = [rng.choice([rng.randrange(-2 ** 31, 2 ** 31), rng.randrange(1 << 20), rng.randrange(4096)]) for _ in range(S)]
    # among them positions that end next to a half turn of some frequency, where the old fraction was rounded most
    for i in range(0, S, 4):
        k = rng.randrange(1, 1 << 24)
        pos[i] = int(min(2 ** 31 - 1, round((2 * k + 1) * float(PI) / rng.choice(freq[:2] + freq[3:8]))))
    x = torch.zeros((1, 1, S, 32), device="cuda")
    x[..., 0::2 if inter else 1] = 1.0
    if not inter:
        x[..., 16:] = 0.0
    y = fa.rope(x, inv, pos=torch.tensor(pos, dtype=torch.int32, device="cuda"), interleaved=inter)[0][0, 0].double().cpu()
    a = torch.tensor([[angle(p, f) for f in freq] for p in pos], dtype=torch.float64)
    got_c, got_s = (y[:, 0::2], y[:, 1::2]) if inter else (y[:, :16], y[:, 16:])
    for got, want in ((got_c, torch.cos(a)), (got_s, torch.sin(a))):
        over = (got - want).abs() - (2.8e-8 + 2.0 ** -23 * want.abs())
        assert float(over.max()) <= 0, float(over.max())
    assert int((torch.sin(a).abs() < 1e-3).sum()) > 100  # where nothing but the angle's error shows
