"""The step plan with more prompts than one workgroup's LDS holds offsets of: the requests are
summed in a launch of their own and the rows filled from memory in a second one."""
import numpy as np
import pytest
import torch

from tests.test_gpu_layer_plan import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,B", [(4096, 0), (4097, 0), (4200, 103), (4201, 100), (9000, 700), (20011, 11)])
def test_many_prompts(requests, B):
    """Around the 4096 prompts that fit and far past them: whole numbers, equal."""
    rng = np.random.default_rng(requests)
    block, kv_block = 64, 16
    m = make(rng, requests, B, 5, 200, block, kv_block)
    need = B + int(m["new"][B:].sum())
    n_exp = int(((m["computed"] + m["new"]) // block - m["computed"] // block)[B:].sum())
    check(m, B, block, kv_block, need + 100, n_exp + 7)
    check(m, B, block, kv_block, need - 3, max(0, n_exp - 2))


def test_both_launches_agree():
    """4097 prompts, the last of them empty, against the same step without it."""
    rng = np.random.default_rng(1)
    m = make(rng, 4100, 3, 40, 3000, 64, 16)
    m["new"][-1] = 0
    short = {k: v[:-1] for k, v in m.items()}
    tokens, exports = 100000, 3000
    a, b = run(m, 3, 64, 16, tokens, exports), run(short, 3, 64, 16, tokens, exports)
    for name in a:
        assert torch.equal(a[name][:b[name].shape[0]], b[name]), name
