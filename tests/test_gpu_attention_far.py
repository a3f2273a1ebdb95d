"""Rotary positions far out on the GPU, against angles reduced in whole numbers."""
import math
from fractions import Fraction

import pytest
import torch

from gated_deltanet_rule_amd import attention as A
from tests import attention_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def pi(bits=256):
    """pi to 2^-bits, by Machin's formula in whole numbers."""
    one = 1 << (bits + 20)

    def arctan_inverse(x):
        total, term, n, sign = 0, one // x, 1, 1
        while term:
            total += sign * (term // n)
            term //= x * x
            n, sign = n + 2, -sign
        return total

    return Fraction(4 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)


PI = pi()


def angles(positions, inv_freq):
    """cos and sin of p f, the angle's whole turns taken off exactly."""
    rows = []
    for p in positions.tolist():
        row = []
        for f in inv_freq.double().tolist():
            turns = Fraction(p) * Fraction(f) / (2 * PI)
            row.append(float((turns - round(turns)) * 2 * PI))
        rows.append(row)
    a = torch.tensor(rows, dtype=torch.float64, device=DEV)
    return torch.cos(a), torch.sin(a)


def test_pi():
    assert float(PI) == math.pi


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base,factor", [(10000.0, 1.0), (5e6, 1.3465), (10000.0, -2.75)])
def test_far_positions_are_as_exact_as_near_ones(base, factor, interleaved):
    d = 128
    positions = torch.tensor([0, 1, 2, 1000, 2 ** 20 + 1, 10 ** 7 + 3, 2 ** 28 + 9, 10 ** 9 + 7, 2 ** 31 - 129, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    freq, _ = A.rotary_frequencies(d, base, device=DEV)
    freq[1], freq[2] = 1.0 - 2.0 ** -24, 1.0 + 2.0 ** -23          # all 24 bits of a frequency
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(len(positions), 3, d, generator=g, device=DEV)
    y = torch.empty_like(x)
    A.gdn_rotary(x, None, positions, freq, q_out=y, interleaved=interleaved, attention_factor=factor)
    cos, sin = (t[:, None] for t in angles(positions, freq))
    # the factor as the fp32 number that the call takes
    f = float(torch.tensor(factor, dtype=F32))
    lay = (lambda t: (t[..., 0::2], t[..., 1::2])) if interleaved else (lambda t: (t[..., : d // 2], t[..., d // 2:]))
    (a, b), (u, v) = lay(x.double()), lay(y.double())
    # cosine and sine times the factor rounded to fp32 once (2^-24 of them), one product's rounding and that of the sum with the other
    bound = (a.abs() + b.abs()) * abs(f) * (2 * 2.0 ** -24)
    for got, want in ((u, f * (a * cos - b * sin)), (v, f * (b * cos + a * sin))):
        R.check("far", got, want, bound + 2.0 ** -24 * (want.abs() + bound) + 1e-30)
