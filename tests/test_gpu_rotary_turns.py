"""Angles of tp_rotary at far positions and large frequencies, against turns taken modulo 1 in whole numbers.

The exact turn of position * freq / (2 pi) modulo 1 comes from 400 bits of 1 / (2 pi) as integers, so what is left is the
call's own: the turn's 64-bit fraction of the frequency, off by 2 * 2^-64 and times a position of at most 2^31 by 2^-32
of a turn; its upper 32 bits (2^-33) rounded to f32 (2^-25 of a half turn, 2^-26 of a turn); sine and cosine within 2^-23, and three
roundings of the products and the sum (2^-24 each)."""
import math

import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BITS = 400


def inverse_two_pi():
    """floor(2^BITS / (2 pi)), pi by Machin's formula with 64 bits to spare."""
    one = 1 << (BITS + 64)

    def arctan_of_inverse(x):
        term, total, n, sign = one // x, 0, 1, 1
        while term:
            total += sign * (term // n)
            term //= x * x
            n, sign = n + 2, -sign
        return total

    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    return (one << BITS) // (2 * pi)


def turns(pos, freq):
    """pos * freq / (2 pi) modulo 1 of an integer and a float, to 2^-200 and better."""
    num, den = float(freq).as_integer_ratio()
    return (pos * num * inverse_two_pi() // den) % (1 << BITS) / (1 << BITS)


POSITIONS = [0, 1, -1, 3, 1000, 131071, 1 << 20, -(1 << 24) - 1, 1000000007, (1 << 31) - 1, -(1 << 31)]


@pytest.mark.parametrize("scale", [1e-6, 1.0, 3.0, 100.0, 12345.678, 1e6, 2.0 ** 39, 2.0 ** 55, 1e-30])
def test_far_turns(scale):
    need_gpu()
    pairs = 32
    freq = (scale * torch.logspace(0, -3, pairs, dtype=torch.float64)).float()
    freq[5] *= -1
    want = torch.tensor([[2 * math.pi * turns(p, f) for f in freq.tolist()] for p in POSITIONS], dtype=torch.float64, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(len(POSITIONS), 64, generator=g, device="cuda")
    y, back = torch.empty_like(x), torch.empty_like(x)
    plan = tp.tp_plan_create(1, 64, 1, 1, 64, 1)
    pos = torch.tensor(POSITIONS, dtype=torch.int32, device="cuda")
    tp.tp_rotary(plan, pos, freq.cuda(), [x], None, [y], None)
    a, b = x[:, :pairs].double(), x[:, pairs:].double()
    c, s = want.cos(), want.sin()
    slack = 2 * math.pi * (2.0 ** -26 + 2.0 ** -32 + 2.0 ** -33) + 2.0 ** -23 + 3 * 2.0 ** -24
    tol = 1.01 * slack * (a.abs() + b.abs())
    got = y.double()
    assert ((got[:, :pairs] - (a * c - b * s)).abs() <= tol).all()
    assert ((got[:, pairs:] - (a * s + b * c)).abs() <= tol).all()
    tp.tp_rotary(plan, pos, freq.cuda(), [y], None, [back], None, inverse=True)  # the same turn, back
    assert ((back - x).abs() <= 1.01 * (2.0 ** -22 + 6 * 2.0 ** -24) * (a.abs() + b.abs()).repeat(1, 2).float() * 2).all()
