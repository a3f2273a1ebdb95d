"""One workspace allocated for the largest step serves the smaller ones, with the bits that a
workspace of their own gives."""
import pytest
import torch

from gated_deltanet_rule_amd import layer
from tests.test_gpu_layer_ssm import i32, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_workspace_for_steps_of_all_sizes(dtype):
    seqs, tokens = 600, 1500
    d = inputs(2, tokens, 2, 4, 128, 128, dtype, 2 * seqs)
    assert layer.alloc_ssm_workspace(d["c"], d["x"], seqs) is None          # the largest step needs none itself
    ws = layer.alloc_ssm_workspace(d["c"], d["x"], seqs, smaller_calls=True)
    for lengths in ([901] + [1] * 599, [1500], [700, 800], [3, 640, 5, 1], [64], [1]):
        n, t = len(lengths), sum(lengths)
        cu = i32([sum(lengths[:k]) for k in range(n + 1)])
        got = []
        for own in (False, True):
            pool, y = d["pool"].clone(), torch.full_like(d["y"][:t], float("nan"))
            layer.gdn_ssm_chunk_prefill(d["c"][:t], d["b"][:t], d["x"][:t], d["dt"][:t], d["A"], y, cu, pool, i32(range(n)), i32(range(n, 2 * n)),
                                        dt_bias=d["bias"], D=d["D"],
                                        workspace=layer.alloc_ssm_workspace(d["c"][:t], d["x"][:t], n) if own else ws)
            got += [y, pool]
        assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3]) and torch.isfinite(got[0]).all()
