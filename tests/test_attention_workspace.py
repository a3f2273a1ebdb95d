"""The decode workspace's size without a GPU: which calls need one, what a too small one is told, calls too large for any."""
import os

import pytest

from gated_deltanet_rule_amd import attention as A
from gated_deltanet_rule_amd import binding as B
from tests import test_attention_abi as T

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libgdn.so not built")


def size(cache, heads, rows, per, keys):
    return A.library().gdn_attention_decode_workspace_size(cache, heads, rows, per, keys)


def test_one_span_needs_none_and_more_need_one():
    # 3 tokens of a group of 2 heads are 6 rows of a head: spans of 512 keys
    assert size(T.cache(), 4, 2, 3, 64) == 0 and size(T.cache(), 4, 2, 3, 512) == 0
    # partial sums of 64 dims and two numbers for each of 2 x 3 tokens, 4 heads, 2 (64) spans
    assert size(T.cache(), 4, 2, 3, 513) == 24 * 2 * (64 + 2) * 4
    assert size(T.cache(), 4, 2, 3, 1 << 20) == 24 * 64 * (64 + 2) * 4


def test_a_workspace_that_is_too_small_or_not_there():
    wide = size(T.cache(), 4, 2, 3, 1 << 20)
    assert wide > 0
    for kw in (dict(ws_bytes=wide - 1), dict(ws_bytes=0)):
        T.refused("gdn_attention_decode", T.decode(T.cache(), width=1 << 16, **kw), "workspace_bytes")
    T.refused("gdn_attention_decode", T.decode(T.cache(), width=1 << 16, ws=None, ws_bytes=wide), "workspace is NULL")
    T.refused("gdn_attention_decode", T.decode(T.cache(), width=1 << 16, ws=T.FAKE + 16, ws_bytes=wide), "workspace")
    # enough of it: the next invalid argument is what is told
    T.refused("gdn_attention_decode", T.decode(T.cache(), width=1 << 16, ws_bytes=wide), "o is NULL")


def test_more_tokens_than_a_call_takes():
    """Sizes do not wrap around: a step of more than 2^31 - 129 tokens has none, the largest one has its own."""
    many = (1 << 31) - 1
    small = T.cache(heads=1, dim=64)
    assert size(small, 1 << 14, many, 64, 1 << 40) == 0
    assert size(small, 1 << 14, 1 << 25, 64, 1 << 40) == 0
    rows = (many - 128) // 64
    assert size(small, 1 << 14, rows, 64, 1 << 40) == rows * 64 * (1 << 14) * 64 * (64 + 2) * 4
