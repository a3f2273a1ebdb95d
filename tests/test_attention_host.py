"""What the attention layers' module computes on the host, against the formulas written out."""
import math

import pytest
import torch

from gated_deltanet_rule_amd import attention as A


@pytest.mark.parametrize("r,base", [(64, 10000.0), (2, 10000.0), (128, 5e6), (24, 1e4)])
def test_frequencies(r, base):
    f, factor = A.rotary_frequencies(r, base)
    assert f.dtype == torch.float32 and f.shape == (r // 2,) and factor == 1.0
    want = torch.tensor([base ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64).to(torch.float32)
    assert torch.equal(f, want)


def test_scaled_frequencies():
    r, base, s, length = 64, 10000.0, 8.0, 4096
    plain = [base ** (-2.0 * i / r) for i in range(r // 2)]
    near = lambda got, want: torch.testing.assert_close(got.double(), torch.tensor(want, dtype=torch.float64), rtol=2.0 ** -22, atol=0)  # noqa: E731
    near(A.rotary_frequencies(r, base, scaling="linear", factor=s)[0], [f / s for f in plain])
    stretched = A.rotary_frequencies(r, base, scaling="base", factor=s)[0]
    near(stretched, [(base * s ** (r / (r - 2))) ** (-2.0 * i / r) for i in range(r // 2)])
    assert stretched[0] == 1.0
    near(stretched[-1:], [plain[-1] / s])
    wave, factor = A.rotary_frequencies(r, base, scaling="wavelength", factor=s, original_length=length, turns=(1.0, 4.0))
    assert factor == 1.0
    want = []
    for f in plain:
        turns = length * f / (2 * math.pi)
        keep = min(max((turns - 1.0) / 3.0, 0.0), 1.0)
        want.append(f * keep + f / s * (1 - keep))
    near(wave, want)
    ramp, factor = A.rotary_frequencies(r, base, scaling="ramp", factor=s, original_length=length)
    assert factor == pytest.approx(0.1 * math.log(s) + 1.0, abs=1e-15)
    number = lambda t: r * math.log(length / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(number(32.0)), 0), min(math.ceil(number(1.0)), r - 1)
    want = [f * (1 - min(max((i - low) / (high - low), 0.0), 1.0)) + f / s * min(max((i - low) / (high - low), 0.0), 1.0) for i, f in enumerate(plain)]
    near(ramp, want)
    assert ramp[0] == 1.0 and ramp[-1] == pytest.approx(plain[-1] / s, rel=1e-6)


def test_frequency_refusals():
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, base=math.inf),
                dict(rotary_dim=8, scaling="cubic"), dict(rotary_dim=8, scaling="ramp", factor=2.0),
                dict(rotary_dim=8, scaling="wavelength", factor=2.0, original_length=100, turns=(4.0, 1.0))):
        with pytest.raises(ValueError):
            A.rotary_frequencies(**bad)


def test_tree_masks():
    mask, depth = A.tree_masks([[-1, 0, 0, 1, -1], [-1, 0, 1, 2, 3]])
    assert mask.tolist() == [1, 3, 5, 11, 16, 1, 3, 7, 15, 31] and depth.tolist() == [0, 1, 1, 2, 0, 0, 1, 2, 3, 4]
    chain, depth = A.tree_masks([list(range(-1, 63))])
    assert chain[-1] == -1 and chain[62] == 2 ** 63 - 1 and depth[-1] == 63
    for bad in ([[0]], [[-1, 1]], [[-1, -2]], [[-1], [-1, 0]], [[]], [[-1] * 65]):
        with pytest.raises(ValueError):
            A.tree_masks(bad)
