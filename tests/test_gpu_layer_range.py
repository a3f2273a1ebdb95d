"""The ends of the range that the header states: sums of squares past fp32's range and below its
normal numbers, and infinities in the scan's x."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_amd import layer
from tests.test_gpu_layer_ssm import i32, inputs, prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sums_of_squares_past_the_range(dtype):
    w = torch.ones(128, device="cuda")
    x = torch.full((3, 1, 128), 1e25, dtype=dtype, device="cuda")
    x[1], x[2] = 0.0, 1e-25
    y = torch.full_like(x, 7.0)
    layer.gdn_gated_norm(x, None, w, y, eps=0.0)
    assert (y[:2] == 0).all()                                      # past the range, and no values at all
    small = x[2].double() / np.sqrt(2.0 ** -126)
    assert ((y[2].double() - small).abs() <= 2.0 ** -7 * small).all()
    out = torch.full((3, 128), 7.0, dtype=dtype, device="cuda")
    pool = torch.zeros(1, 1, 128, dtype=dtype, device="cuda")
    weight = torch.tensor([0.0, 1.0], device="cuda").repeat(128, 1)          # the token itself
    layer.gdn_causal_conv_prefill(x[:, 0], weight, None, [out], pool, i32([0, 3]), i32([-1]), i32([-1]), activation="none", l2_dims=(128,), l2_eps=0.0)
    assert (out[:2] == 0).all() and ((out[2].double() - small[0]).abs() <= 2.0 ** -7 * small[0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("many", [0, 600])
def test_infinite_x(dtype, many):
    """An infinity at token 70: its column NaN to the chunk's end, not finite after it; everything
    else as without it."""
    L = 300
    d = inputs(6, L + many, 1, 2, 64, 64, dtype, 2)
    args = ([L] + [1] * many, [-1] * (1 + many), [0] + [-1] * many)
    clean = torch.empty_like(d["y"])
    prefill(d, *args, y=clean)
    state = d["pool"][0].clone()
    e = dict(d, x=d["x"].clone())
    e["x"][70, 1, 9] = float("inf")
    prefill(e, *args)
    y, keep = d["y"], torch.ones(2, 64, dtype=torch.bool, device="cuda")
    keep[1, 9] = False
    assert torch.equal(y[:70], clean[:70]) and torch.equal(y[L:], clean[L:]) and torch.equal(y[:, keep], clean[:, keep])
    assert torch.isnan(y[70:128, 1, 9]).all() and not torch.isfinite(y[128:L, 1, 9]).any()
    assert not torch.isfinite(d["pool"][0, 1, :, 9]).any()
    assert torch.equal(d["pool"][0, 0], state[0]) and torch.equal(d["pool"][0, 1][:, keep[1]], state[1][:, keep[1]])
