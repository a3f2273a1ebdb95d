"""The attention layers' C ABI without a GPU: every symbol that include/gdn_attention.h declares is exported and
bound, and bad host arguments are refused with a message naming them before anything is enqueued.

No call can reach a launch: besides the argument under test each one carries a second invalid argument that is
checked last (a NULL output)."""
import ctypes
import os
import re

import pytest

from gated_deltanet_rule_amd import attention as A
from gated_deltanet_rule_amd import binding as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdn_attention.h")
pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libgdn.so not built")

FAKE = 0x100000           # a 16-byte aligned stand-in address that is never dereferenced
INVALID, UNSUPPORTED = B.GDN_ERR_INVALID_ARGUMENT, B.GDN_ERR_UNSUPPORTED


def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdn_[a-z_]+)\s*\(", text))
    assert names == set(A.SIGNATURES)
    lib = ctypes.CDLL(B.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def refused(name, args, needle, code=INVALID):
    st = getattr(A.library(), name)(*args)
    assert st == code and needle in B.gdn_last_error(), (name, st, B.gdn_last_error())


def rotary(shape=(4, 2, 64, 64, 1, 0, 1.0), tokens=5, positions=FAKE, freq=FAKE, q=FAKE, qs=256, k=FAKE, ks=128, qo=FAKE * 2, qos=256, ko=None, kos=128):
    return [A.GdnRotaryShape(*shape) if shape else None, tokens, positions, freq, q, qs, k, ks, qo, qos, ko, kos, None]


@pytest.mark.parametrize("kw,needle,code", [
    (dict(shape=None), "shape is NULL", INVALID), (dict(shape=(-1, 2, 64, 64, 1, 0, 1.0)), "num_q_heads -1", INVALID),
    (dict(shape=(4, 2, 0, 0, 1, 0, 1.0)), "head_dim 0", INVALID), (dict(shape=(4, 2, 520, 64, 1, 0, 1.0)), "head_dim 520", UNSUPPORTED),
    (dict(shape=(4, 2, 64, 63, 1, 0, 1.0)), "rotary_dim 63", INVALID), (dict(shape=(4, 2, 64, 66, 1, 0, 1.0)), "rotary_dim 66", INVALID),
    (dict(shape=(4, 2, 64, 0, 1, 0, 1.0)), "rotary_dim 0", INVALID), (dict(shape=(4, 2, 64, 64, 2, 0, 1.0)), "dtype 2", UNSUPPORTED),
    (dict(shape=(2 ** 31 - 1, 2 ** 31 - 1, 512, 64, 1, 0, 1.0)), "2^20", UNSUPPORTED),
    (dict(shape=(4, 2, 64, 64, 1, 0, float("nan"))), "factor", INVALID), (dict(tokens=-1), "num_tokens -1", INVALID),
    (dict(tokens=1 << 31), "2^31 - 129", UNSUPPORTED), (dict(positions=None), "positions is NULL", INVALID), (dict(freq=FAKE + 2), "inv_freq", INVALID),
    (dict(qs=255), "q_stride 255", INVALID), (dict(qos=100), "q_out_stride 100", INVALID), (dict(ks=127), "k_stride 127", INVALID),
    (dict(q=None), "q is NULL", INVALID), (dict(q=FAKE + 1), "q (", INVALID), (dict(qo=FAKE, qos=512), "in place", INVALID),
    (dict(), "k_out is NULL", INVALID)])
def test_rotary_refusals(kw, needle, code):
    refused("gdn_rotary", rotary(**kw), needle, code)


def cache(heads=2, dim=64, dtype=1, form=1, rows=100, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE):
    return A.GdnKvCache(heads, dim, dtype, form, rows, k, v, ks, vs)


CACHES = [(None, "cache is NULL", INVALID), (cache(heads=0), "num_heads 0", INVALID), (cache(dim=-8), "head_dim -8", INVALID),
          (cache(dim=60), "head_dim 60", UNSUPPORTED), (cache(dim=520), "head_dim 520", UNSUPPORTED), (cache(dtype=7), "dtype 7", UNSUPPORTED),
          (cache(form=3), "format 3", UNSUPPORTED), (cache(heads=1 << 15), "2^20", UNSUPPORTED), (cache(rows=-1), "num_rows -1", INVALID),
          (cache(rows=1 << 31), "num_rows 2147483648", UNSUPPORTED),
          (cache(k=None), "cache k is NULL", INVALID), (cache(v=FAKE + 8), "cache v", INVALID), (cache(ks=None), "k_scale is NULL", INVALID),
          (cache(vs=FAKE + 2), "v_scale", INVALID)]


def write(c, tokens=5, k=FAKE, ks=128, v=FAKE, vs=128, slots=None):
    return [c, tokens, k, ks, v, vs, slots, None]


def read(c, tokens=5, slots=FAKE, ko=FAKE, vo=None):
    return [c, tokens, slots, ko, vo, None]


def prefill(c, hq=4, scale=0.1, n=2, tokens=10, cu=FAKE, start=FAKE, q=FAKE, qs=256, table=FAKE, width=4, block=16, o=None):
    return [c, hq, scale, n, tokens, cu, start, q, qs, table, width, block, o, None]


def decode(c, hq=4, scale=0.1, rows=2, per=3, computed=FAKE, mask=FAKE, q=FAKE, qs=256, table=FAKE, width=4, block=16, keys=0, o=None, ws=FAKE,
           ws_bytes=1 << 40):
    return [c, hq, scale, rows, per, computed, mask, q, qs, table, width, block, keys, o, ws, ws_bytes, None]


@pytest.mark.parametrize("c,needle,code", CACHES)
def test_cache_refusals(c, needle, code):
    for name, args in (("gdn_kv_cache_write", write(c)), ("gdn_kv_cache_read", read(c)), ("gdn_attention_prefill", prefill(c)),
                       ("gdn_attention_decode", decode(c))):
        refused(name, args, needle, code)


@pytest.mark.parametrize("kw,needle,code", [
    (dict(tokens=-1), "num_tokens -1", INVALID), (dict(tokens=1 << 31), "num_tokens", UNSUPPORTED), (dict(ks=120), "k_stride 120", INVALID),
    (dict(vs=132), "v_stride 132", INVALID), (dict(k=FAKE + 8), "k (", INVALID), (dict(v=None), "v is NULL", INVALID), (dict(), "slots is NULL", INVALID)])
def test_write_refusals(kw, needle, code):
    refused("gdn_kv_cache_write", write(cache(), **kw), needle, code)


@pytest.mark.parametrize("kw,needle", [(dict(tokens=-2), "num_tokens -2"), (dict(slots=FAKE + 4), "slots"), (dict(ko=None), "k_out is NULL"),
                                       (dict(), "v_out is NULL")])
def test_read_refusals(kw, needle):
    refused("gdn_kv_cache_read", read(cache(), **kw), needle)


BOTH = [(dict(hq=0), "num_q_heads 0", INVALID), (dict(hq=3), "num_q_heads 3", INVALID), (dict(hq=1 << 16), "2^20", UNSUPPORTED),
        (dict(scale=float("inf")), "scale", INVALID), (dict(width=-1), "kv_table_width -1", INVALID), (dict(block=0), "kv_block 0", INVALID),
        (dict(qs=248), "q_stride 248", INVALID), (dict(qs=260), "q_stride 260", INVALID), (dict(q=FAKE + 4), "q (", INVALID), (dict(q=None), "q is NULL", INVALID),
        (dict(table=None), "kv_table is NULL", INVALID), (dict(), "o is NULL", INVALID)]


@pytest.mark.parametrize("kw,needle,code", BOTH + [
    (dict(n=-1), "num_seqs -1", INVALID), (dict(tokens=-1), "total_tokens -1", INVALID), (dict(tokens=1 << 31), "total_tokens", UNSUPPORTED),
    (dict(cu=None), "cu_seqlens is NULL", INVALID), (dict(start=FAKE + 1), "start_pos", INVALID)])
def test_prefill_refusals(kw, needle, code):
    refused("gdn_attention_prefill", prefill(cache(), **kw), needle, code)


@pytest.mark.parametrize("kw,needle,code", BOTH + [
    (dict(rows=-1), "num_rows -1", INVALID), (dict(per=0), "tokens_per_row 0", INVALID), (dict(per=65), "tokens_per_row 65", UNSUPPORTED),
    (dict(rows=1 << 30, per=64), "num_rows x tokens_per_row", UNSUPPORTED), (dict(keys=-1), "max_keys -1", INVALID), (dict(mask=FAKE + 4), "tree_mask", INVALID),
    (dict(computed=None), "computed is NULL", INVALID)])
def test_decode_refusals(kw, needle, code):
    refused("gdn_attention_decode", decode(cache(), **kw), needle, code)


def test_head_dims_of_the_attention():
    for dim in (8, 80, 512):
        refused("gdn_attention_prefill", prefill(cache(dim=dim)), "the attention takes 64, 128 or 256", UNSUPPORTED)
        refused("gdn_attention_decode", decode(cache(dim=dim)), "the attention takes 64, 128 or 256", UNSUPPORTED)


def test_empty_calls_need_no_pointers():
    lib = A.library()
    none = cache(k=None, v=None, ks=None, vs=None, rows=0)
    assert lib.gdn_rotary(*rotary(tokens=0, positions=None, freq=None)) == 0
    assert lib.gdn_rotary(*rotary(shape=(0, 0, 64, 64, 1, 0, 1.0), positions=None)) == 0
    assert lib.gdn_kv_cache_write(*write(none, tokens=0)) == 0 and lib.gdn_kv_cache_read(*read(none, tokens=0)) == 0
    assert lib.gdn_attention_prefill(*prefill(none, n=0)) == 0 and lib.gdn_attention_prefill(*prefill(none, tokens=0)) == 0
    assert lib.gdn_attention_decode(*decode(none, rows=0)) == 0


def test_workspace_size_covers_smaller_calls():
    lib = A.library()
    size = lambda hq, rows, per, keys, c=cache(): lib.gdn_attention_decode_workspace_size(c, hq, rows, per, keys)  # noqa: E731
    assert size(3, 2, 1, 100) == 0 and size(4, 2, 65, 100) == 0 and size(4, -1, 1, 100) == 0 and size(4, 2, 1, -5) == 0
    for hq in (2, 8, 64):
        for per in (1, 2, 7, 16, 33, 64):
            keys = [0, 1, 200, 256, 257, 600, 1000, 5000, 16384, 16385, 40000, 131072, 131073, 1 << 20, (1 << 31) - 200, 1 << 40]
            sizes = [size(hq, 5, per, n) for n in keys]
            assert sizes == sorted(sizes), (hq, per, sizes)
            assert size(hq, 4, per, 70000) <= size(hq, 5, per, 70000)
            assert all(size(hq, 5, less, 70000) <= size(hq, 5, per, 70000) for less in range(1, per))


def test_workspace_is_required():
    lib = A.library()
    need = lib.gdn_attention_decode_workspace_size(cache(), 4, 2, 3, 64)
    wide = lib.gdn_attention_decode_workspace_size(cache(), 4, 2, 3, 1 << 20)
    if need:
        refused("gdn_attention_decode", decode(cache(), ws_bytes=need - 1), "workspace_bytes")
    if wide:
        refused("gdn_attention_decode", decode(cache(), width=1 << 16, ws_bytes=wide - 1), "workspace_bytes")
        refused("gdn_attention_decode", decode(cache(), width=1 << 16, ws=None), "workspace is NULL")
        refused("gdn_attention_decode", decode(cache(), width=1 << 16, ws=FAKE + 16), "workspace")
