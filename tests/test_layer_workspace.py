"""The scan's workspace sizes without a GPU: the bound of a step's size holds for every smaller
call, and is no larger than one of them needs."""
import os

import pytest

from gated_deltanet_rule_amd import binding as B
from gated_deltanet_rule_amd import layer as L

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libgdn.so not built")


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("H_k,H_v,d_v", [(16, 32, 128), (1, 1, 64), (2, 6, 128), (8, 64, 64), (1, 700, 64)])
@pytest.mark.parametrize("seqs,tokens", [(0, 5000), (1, 0), (1, 63), (1, 8192), (3, 500), (16, 131072), (300, 20000), (1000, 1000)])
def test_bound(dtype, H_k, H_v, d_v, seqs, tokens):
    shape = B.make_shape(H_k, H_v, 128, d_v, dtype, 1.0)
    size, bound = L.library().gdn_ssm_chunk_prefill_workspace_size, L.library().gdn_ssm_chunk_prefill_workspace_bound
    most = bound(shape, seqs, tokens)
    some = sorted({tokens * k // 37 for k in range(38)})
    needs = [size(shape, n, t) for n in range(seqs + 1) for t in some]
    assert most == max(needs)
    assert bound(shape, seqs + 1, tokens) >= most and bound(shape, seqs, tokens + 1) >= most


def test_bound_of_a_refused_shape():
    bound = L.library().gdn_ssm_chunk_prefill_workspace_bound
    assert bound(B.make_shape(3, 4, 128, 128, 1, 1.0), 1, 8192) == 0
    assert bound(B.make_shape(2, 4, 128, 128, 1, 1.0), -1, 8192) == 0 and bound(B.make_shape(2, 4, 128, 128, 1, 1.0), 1, -1) == 0


def test_no_sequences_need_nothing():
    assert L.library().gdn_ssm_chunk_prefill_workspace_size(B.make_shape(2, 4, 128, 128, 1, 1.0), 0, 8192) == 0
