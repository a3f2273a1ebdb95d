"""Calls of more threads than a launch may have (2^32 - 1) are refused by name before anything
is enqueued.  Needs no GPU: the addresses are stand-ins that nothing reads."""
import os

import pytest

from gated_deltanet_rule_amd import binding as B
from gated_deltanet_rule_amd import layer as L
from tests import test_layer_abi as A

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libgdn.so not built")

F = A.FAKE
ONE = A.conv_shape(channels=(8, 0, 0), l2=(0, 0, 0))
HEAD = B.make_shape(1, 1, 64, 64, 1, 1.0)


@pytest.mark.parametrize("name,args,what", [
    ("gdn_gated_norm", A.gated(rows=1 << 24, groups=1, dim=4096, xs=4096, zs=4096, y=F), "gated norm"),         # 256 threads a row
    ("gdn_gated_norm", A.gated(rows=1 << 20, groups=64, dim=256, xs=1 << 14, zs=1 << 14, y=F), "gated norm"),   # 64 threads a norm
    ("gdn_gated_norm", A.gated(rows=1 << 22, groups=1, dim=16384, dtype=0, xs=16384, zs=16384, y=F), "gated norm"),   # 1024 threads a row
    ("gdn_residual_norm", A.residual(rows=1 << 24, dim=520, xs=520, gs=520, out=F), "residual norm"),
    ("gdn_causal_conv_decode", A.conv_decode(shape=ONE, rows=1 << 24, stride=8, y2=None, slot_out=F), "convolution"),
    ("gdn_causal_conv_prefill", A.conv_prefill(shape=ONE, tokens=1 << 29, stride=8), "convolution"),
    ("gdn_ssm_recurrent_decode", A.ssm_decode(shape=HEAD, rows=1 << 24, slot_out=F), "scan"),
    ("gdn_ssm_chunk_prefill", A.ssm_prefill(shape=HEAD, n=1 << 24, tokens=100, y=F), "scan"),
    ("gdn_ssm_chunk_prefill", A.ssm_prefill(shape=B.make_shape(64, 64, 64, 64, 1, 1.0), n=1, tokens=(1 << 31) - 200, y=F, ws=F, ws_bytes=1 << 60),
     "scan")])
def test_refused(name, args, what):
    status = getattr(L.library(), name)(*args)
    message = B.gdn_last_error()
    assert status == B.GDN_ERR_UNSUPPORTED and what in message and "launch grid" in message, (status, message)


@pytest.mark.parametrize("k_heads,d_k,d_v,needle", [(20000, 128, 128, "num_v_heads 40000 x d_v 128"), (40000, 128, 64, "num_k_heads 40000 x d_k 128")])
def test_rows_too_wide_name_their_heads(k_heads, d_k, d_v, needle):
    shape = B.make_shape(k_heads, 40000, d_k, d_v, 1, 1.0)
    assert L.library().gdn_ssm_chunk_prefill(*A.ssm_prefill(shape=shape, n=1, y=None)) == B.GDN_ERR_UNSUPPORTED
    assert needle in B.gdn_last_error(), B.gdn_last_error()


@pytest.mark.parametrize("count", [1 << 31, 1 << 40, (1 << 63) - 1])
def test_export_capacity_takes_no_launch(count):
    """However many exports the caller has room for, they cost no threads: the same call is refused
    for its tokens alone."""
    args = A.conv_prefill(shape=ONE, tokens=1 << 29, stride=8, grid=64, eslots=F, count=count)
    assert L.library().gdn_causal_conv_prefill(*args) == B.GDN_ERR_UNSUPPORTED
    assert "threads" in B.gdn_last_error(), B.gdn_last_error()
