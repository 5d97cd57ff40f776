"""The rotation at positions far out, against angles taken from whole numbers of any length: the error is what the
documentation says, 3 * 2^-53 of the angle and 2^-26 of a turn."""
import math
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")
from layer_testlib import U32, assert_within, gen, randn  # noqa: E402

pytestmark = pytest.mark.gpu
R = 64
BITS = 200


def arctan_inverse(n):
    """floor(2^BITS arctan(1 / n)) by its series, to a few units"""
    term = total = (1 << BITS) // n
    k, sign = 1, 1
    while term:
        term //= n * n
        k, sign = k + 2, -sign
        total += sign * (term // k)
    return total


PI = Fraction(4 * (4 * arctan_inverse(5) - arctan_inverse(239)), 1 << BITS)  # Machin's formula


def turn_of(pos, f):
    """cos and sin of pos * f, f a fp32 value"""
    a = Fraction(pos) * Fraction(f)
    a -= 2 * PI * round(a / (2 * PI))
    return math.cos(float(a)), math.sin(float(a))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D", [64, 70])  # whole vectors, and the kernel for any size
def test_far_positions(D, inter):
    import kimi_delta_attention_21_b200 as K
    at = [0, 1, -1, 1000, 1 << 20, (1 << 25) - 1, (1 << 30) + 12345, (1 << 31) - 1, -(1 << 31) + 1, 2111111111, -1999999999]
    g = gen(D)
    x = randn(g, 1, len(at), 1, D)
    pos = torch.tensor([at], device="cuda")
    inv = torch.cat([torch.rand(8, generator=g, device="cuda") * 0.5 + 0.5,  # the fastest, with all their bits
                     10000.0 ** (-torch.arange(8, R // 2, device="cuda") / (R // 2))])
    y, _ = K.qk_norm(x, x, norm="rms", positions=pos, inv_freq=inv, interleaved=inter)
    freq = inv.tolist()
    cs = torch.tensor([[turn_of(p, f) for f in freq] for p in at], dtype=torch.float64, device="cuda")[None, :, None]
    c, s = cs[..., 0], cs[..., 1]
    n = x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    want = n.clone()
    want[..., a], want[..., b] = n[..., a] * c - n[..., b] * s, n[..., a] * s + n[..., b] * c
    size = torch.zeros_like(want)  # |(a, b)| of a rotated channel
    size[..., a] = size[..., b] = (n[..., a].square() + n[..., b].square()).sqrt()
    angle = torch.zeros_like(want)
    angle[..., a] = angle[..., b] = (pos.double()[..., None, None] * inv.double()).abs()
    # beside the angle: the sum of squares 5 half-steps (10 additions in a row, halved by the root), mean and eps 2, root 4, its
    # product 2, sine and cosine 4 each, two products and a sum 3
    tol = size * (3 * 2.0 ** -53 * angle + 2 * math.pi * 2.0 ** -26 + 20 * U32) + 16 * U32 * n.abs()
    assert_within(y, want, tol, "y")
