"""The scan with one very large step among small ones (a token that resets the state): the
tokens after it are decayed by their own small steps alone, however large the sum of the
chunk's exponents is."""
import math

import numpy as np
import pytest
import torch

from gated_deltanet_rule_amd import layer
from tests import layer_reference as R
from tests.test_gpu_layer_ssm import f64, i32, inputs, within

pytestmark = pytest.mark.gpu
L, LARGE = 300, (5, 64, 100, 191, 250)            # inside chunks, at a chunk's start and at its end


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("step", [1e3, 1e4, 6e4, 1e6, 1e20, 3e38])
@pytest.mark.parametrize("many", [0, 600])
def test_one_large_step_among_small_ones(dtype, step, many):
    """The large steps' tokens have b = x = 0, so they only take the state away.  The reference has a
    step there whose decay is e^-100: what that leaves of the state is below every bound here, and
    the bounds, which grow with a chunk's sum of exponents, then count the small steps' sums and
    not the large step's.  many: single tokens beside it, enough to take the whole-heads launch."""
    heads, slots = 2, many + 4
    d = inputs(5, L + many, 1, heads, 64, 64, dtype, slots, bias=False)
    d["A"] = torch.tensor([-16.0, -7.0], device="cuda")
    g = torch.Generator().manual_seed(3)
    small = torch.exp(torch.rand(L + many, heads, generator=g) * math.log(100.0) + math.log(1e-3))
    raw = torch.log(torch.expm1(small))
    at = torch.tensor(LARGE)
    mild = raw.clone()
    raw[at], mild[at] = step, 100.0 / d["A"].abs().cpu()      # softplus(v) >= v
    d["dt"] = raw.cuda()
    for k in ("b", "x"):
        d[k][at.cuda()] = 0.0
    lengths = [L] + [1] * many
    n = len(lengths)
    before = f64(d["pool"][:1])
    ws = layer.alloc_ssm_workspace(d["c"], d["x"], n)
    assert (ws is None) == (many > 0)
    layer.gdn_ssm_chunk_prefill(d["c"], d["b"], d["x"], d["dt"], d["A"], d["y"], i32(np.cumsum([0] + lengths)), d["pool"],
                                i32([0] + [-1] * many), i32([n] + [-1] * many), D=d["D"], workspace=ws)
    for h in range(heads):
        y, yb, S, Sb = R.scan(f64(d["c"][:L, 0]), f64(d["b"][:L, 0]), f64(d["x"][:L, h]), f64(mild[:L, h]), float(d["A"][h]), None,
                              float(d["D"][h]), True, 1.0, before[0, h], dtype)
        within("head %d y" % h, d["y"][:L, h], y, yb)
        within("head %d state" % h, d["pool"][n, h], S[-1], Sb[-1] + 1e-30)
