"""Attention calls of more threads than a launch may have (2^32 - 1) are refused by name before anything is
enqueued.  Needs no GPU: the addresses are stand-ins that nothing reads."""
import os

import pytest

from gated_deltanet_rule_amd import attention as A
from gated_deltanet_rule_amd import binding as B
from tests import test_attention_abi as T

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libgdn.so not built")

F = T.FAKE
MANY = (1 << 31) - 200


@pytest.mark.parametrize("name,args,what", [
    ("gdn_rotary", T.rotary(shape=(64, 64, 512, 512, 1, 0, 1.0), tokens=1 << 24, qs=1 << 15, ks=1 << 15, qos=1 << 15, ko=F * 3, kos=1 << 15), "rotary"),
    ("gdn_kv_cache_write", T.write(T.cache(heads=2048, dim=512), tokens=1 << 24, ks=1 << 20, vs=1 << 20, slots=F), "cache"),
    ("gdn_kv_cache_read", T.read(T.cache(heads=2048, dim=512), tokens=1 << 24, vo=F), "cache"),
    ("gdn_attention_prefill", T.prefill(T.cache(form=0), tokens=MANY, hq=2048, qs=1 << 17, o=F), "attention"),
    ("gdn_attention_prefill", T.prefill(T.cache(form=0, dtype=0), tokens=MANY, hq=2048, qs=1 << 17, o=F), "attention"),
    ("gdn_attention_prefill", T.prefill(T.cache(heads=2048, dim=64), n=1 << 24, tokens=100, hq=2048, qs=1 << 17, o=F), "attention"),
    ("gdn_attention_decode", T.decode(T.cache(), rows=1 << 25, per=1, o=F, ws_bytes=1 << 62), "attention"),
    ("gdn_attention_decode", T.decode(T.cache(heads=1), rows=1 << 23, per=1, hq=16, qs=1024, width=1 << 16, keys=1024, o=F, ws_bytes=1 << 62), "attention"),
    ("gdn_attention_decode", T.decode(T.cache(), rows=1 << 25, per=40, o=F, ws_bytes=1 << 62), "attention")])
def test_refused(name, args, what):
    status = getattr(A.library(), name)(*args)
    message = B.gdn_last_error()
    assert status == B.GDN_ERR_UNSUPPORTED and what in message and "launch grid" in message, (status, message)
