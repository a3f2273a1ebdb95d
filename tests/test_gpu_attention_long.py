"""Decode rows of long contexts on the GPU: row lengths up to the most that a table can hold."""
import pytest
import torch

from gated_deltanet_rule_amd import attention as A
from tests import attention_cases as C
from tests import attention_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def decode(q, cache, table, kv_block, past, per, scale, max_keys=0):
    o = torch.full(q.shape, 5.0, dtype=q.dtype, device=DEV)
    ws = A.alloc_attention_workspace(q, cache["k_cache"], tokens_per_row=per, max_keys=max_keys or table.shape[1] * kv_block)
    if ws is not None:
        ws.fill_(0xff)
    A.gdn_attention_decode(q, o=o, computed=C.i32(past, DEV), kv_table=table, kv_block=kv_block, scale=scale, tokens_per_row=per, max_keys=max_keys,
                           workspace=ws, **cache)
    return o


@pytest.mark.parametrize("dtype,per", [(BF16, 1), (F32, 1), (BF16, 33)])
def test_rows_of_two_thousand_million_keys(dtype, per):
    """Nearly all pages of a row are absent, and its length is as much as a table can hold: the keys that are there count.
    2113929216 keys are the most whose number, rounded up to whole spans of 2^25, stays below 2^31."""
    d, hq, block, have = 64, 2, 1 << 30, 70
    cache = C.filled_cache(have, 1, d, dtype, None, torch.arange(have, device=DEV), DEV, 1)
    table = C.i32([[0, -1]], DEV)
    q = C.queries(per, hq, d, dtype, DEV, 2)
    # the keys at the new tokens' positions are absent: each token sees the 70 there are
    seen = torch.ones(per, have, dtype=torch.bool, device=DEV)
    k, v = cache["k_cache"][:, 0].double(), cache["v_cache"][:, 0].double()
    ref, bound = R.attend(q, k, v, seen, 0.1)
    for keys in (2113929216, 2113929217, (1 << 31) - 1025):
        R.check(str(keys), decode(q, cache, table, block, [keys - per], per, 0.1, max_keys=keys), ref, bound)
