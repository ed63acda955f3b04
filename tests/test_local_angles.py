"""The rotation's angles at far positions, for frequencies of any size, against whole-number arithmetic."""
import math
from fractions import Fraction

import pytest
import torch

from block_sparse_attention_qp_gb300 import binding as msa

DEV = "cuda:0"
BITS = 260


def inverse_two_pi():
    """2^BITS / (2 pi), from Machin's formula pi = 16 atan(1/5) - 4 atan(1/239)."""
    one = 1 << (BITS + 64)

    def atan(k):
        term, total, n, sign = one // k, 0, 1, 1
        while term:
            total += sign * (term // n)
            term //= k * k
            n, sign = n + 2, -sign
        return total

    pi = 16 * atan(5) - 4 * atan(239)
    return (one << BITS) // (2 * pi)


def angle(pos, f, inv2pi):
    """pos * f modulo 2 pi, off by no more than an fp64 rounding."""
    f = Fraction(f)
    turns = (pos * f.numerator * inv2pi) % (f.denominator << BITS)
    return 2 * math.pi * float(Fraction(turns, f.denominator << BITS))


def test_angle_itself():
    inv2pi = inverse_two_pi()
    assert abs(inv2pi / 2 ** BITS * 2 * math.pi - 1) < 1e-15
    for pos, f in ((0, 1.0), (1, 1.0), (-3, 0.25), (100, 7.5)):
        assert abs(angle(pos, f, inv2pi) - math.remainder(pos * f, 2 * math.pi) % (2 * math.pi)) < 1e-12


@pytest.mark.gpu
@pytest.mark.parametrize("lo,hi", [(1.0, 20.0), (-1.0, 1.0), (-3e4, 3e4), (-2.0 ** 40, 2.0 ** 40)])
@pytest.mark.parametrize("inter", [False, True])
def test_far_angles(lo, hi, inter):
    """Rotation alone.  Relative to the two elements of a pair an output is off by half a bf16 step of itself and by the
    angle's and the rotation's fp32 roundings: 2^-25 turns (1.9e-7) from the angle, 2 ulps of sine and cosine
    (1.2e-7), two of the products' sum (1.2e-7); the 64-bit fraction adds 2^31 2^-64 turns.  1e-6 covers them."""
    g = torch.Generator().manual_seed(int(abs(hi)) % 1000)
    f = (lo + (hi - lo) * torch.rand(64, generator=g, dtype=torch.float64)).float()
    pos = torch.cat([torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1, -1]),
                     torch.randint(-2 ** 31, 2 ** 31, (59,), generator=g)]).to(torch.int32)
    x = torch.randn(1, 64, 64, 128, generator=g).to(torch.bfloat16)
    y, = msa.msa_norm_rope_forward([x.to(DEV)], None, f.to(DEV), positions=pos.view(1, -1).to(DEV), interleaved=inter)
    dy, = msa.msa_norm_rope_backward([x.to(DEV)], None, [x.to(DEV)], f.to(DEV), positions=pos.view(1, -1).to(DEV),
                                     interleaved=inter)[0]
    inv2pi = inverse_two_pi()
    a = torch.tensor([[angle(int(p), float(z), inv2pi) for z in f] for p in pos], dtype=torch.float64)
    c, s = a.cos().view(1, 64, 1, 64), a.sin().view(1, 64, 1, 64)
    at = (slice(0, None, 2), slice(1, None, 2)) if inter else (slice(0, 64), slice(64, None))
    u, v = (x.double()[..., i] for i in at)
    for got, s in ((y, s), (dy, -s)):
        for i, want in zip(at, (u * c - v * s, v * c + u * s)):
            err = (got.cpu().double()[..., i] - want).abs()
            bound = torch.finfo(torch.bfloat16).eps / 2 * want.abs() + 1e-6 * (u.abs() + v.abs())
            assert (err <= bound).all(), float((err / bound).max())
