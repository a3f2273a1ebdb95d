"""The layer operators' C ABI without a GPU: every symbol that include/gdn_layer.h declares is
exported and bound, and bad host arguments are refused with a message naming them before
anything is enqueued.

No call can reach a launch: besides the argument under test each one carries a second
invalid argument that is checked last (a NULL output)."""
import ctypes
import os
import re

import pytest

from gated_deltanet_rule_amd import binding as B
from gated_deltanet_rule_amd import layer as L

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdn_layer.h")
pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libgdn.so not built")

FAKE = 0x100000           # a 16-byte aligned stand-in address that is never dereferenced
INVALID, UNSUPPORTED = B.GDN_ERR_INVALID_ARGUMENT, B.GDN_ERR_UNSUPPORTED


def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdn_[a-z_]+)\s*\(", text))
    assert names == set(L.SIGNATURES)
    lib = ctypes.CDLL(B.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def refused(name, args, needle, code=INVALID):
    st = getattr(L.library(), name)(*args)
    assert st == code and needle in B.gdn_last_error(), (name, st, B.gdn_last_error())


def plan_args(**kw):
    a = dict(requests=4, decode=2, computed=FAKE, new=FAKE, table=FAKE, width=4, block=64, run=FAKE, kv=FAKE, kv_width=8,
             kv_block=16, tokens=100, exports=4, slot_in=FAKE, slot_out=FAKE, cu=FAKE, start=FAKE, init=FAKE, final=FAKE,
             offsets=None, slots=FAKE, req=FAKE, pos=FAKE, kvs=FAKE, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("change,needle", [
    (dict(requests=-1), "num_requests -1"), (dict(decode=5), "num_decode_rows 5"), (dict(decode=-1), "num_decode_rows -1"),
    (dict(block=0), "state_block 0"), (dict(block=100), "chunk size 64"), (dict(width=-2), "state_table_width -2"),
    (dict(kv=None), "without a kv_table"), (dict(kv_block=0), "kv_block 0"), (dict(kv_width=-1), "kv_table_width -1"),
    (dict(tokens=-1), "token_capacity -1"), (dict(tokens=1 << 31), "token_capacity"), (dict(exports=-1), "export_capacity -1"),
    (dict(computed=None), "computed is NULL"), (dict(new=FAKE + 2), "new_tokens"), (dict(run=None), "run_slot is NULL"),
    (dict(table=None), "state_table is NULL"), (dict(slot_in=None), "slot_in is NULL"), (dict(final=None), "final_slot is NULL"),
    (dict(kvs=FAKE + 4), "token_kv_slot"), (dict(pos=FAKE + 1), "token_position"), (dict(slots=None), "export_slots is NULL"),
    (dict(cu=None), "cu_seqlens is NULL"), (dict(), "export_offsets is NULL")])
def test_plan_refusals(change, needle):
    refused("gdn_step_plan", plan_args(**change), needle)


def conv_shape(channels=(64, 64, 128), l2=(64, 64, 0), width=4, dtype=1, act=1, eps=1e-6):
    return L.GdnConvShape((ctypes.c_int32 * 3)(*channels), (ctypes.c_int32 * 3)(*l2), width, dtype, act, eps)


def conv_prefill(shape=None, n=2, tokens=100, cu=FAKE, x=FAKE, stride=256, weight=FAKE, bias=FAKE, y0=FAKE, y1=FAKE, y2=None,
                 pool=FAKE, slots=8, init=FAKE, final=FAKE, start=FAKE, grid=0, states=FAKE, offsets=FAKE, eslots=None, count=0):
    return [shape or conv_shape(), n, tokens, cu, x, stride, weight, bias, y0, y1, y2, pool, slots, init, final, start, grid, states,
            offsets, eslots, count, None]


def conv_decode(shape=None, rows=4, x=FAKE, stride=256, y2=FAKE, pool=FAKE, slots=8, slot_in=FAKE, slot_out=None):
    return [shape or conv_shape(), rows, x, stride, FAKE, None, FAKE, FAKE, y2, pool, slots, slot_in, slot_out, None]


@pytest.mark.parametrize("shape,needle,code", [
    (conv_shape(channels=(60, 64, 128)), "channels[0] 60 is not a multiple of 8", UNSUPPORTED),
    (conv_shape(channels=(-8, 64, 128)), "channels[0] -8", INVALID), (conv_shape(channels=(0, 0, 0)), "no channels", INVALID),
    (conv_shape(channels=(1 << 20, 64, 128)), "exceed", UNSUPPORTED),
    (conv_shape(l2=(48, 0, 0)), "l2_dim[0] 48", UNSUPPORTED), (conv_shape(l2=(0, 128, 0)), "l2_dim[1] 128", INVALID),
    (conv_shape(width=1), "width 1", UNSUPPORTED), (conv_shape(width=5), "width 5", UNSUPPORTED),
    (conv_shape(dtype=3), "dtype 3", UNSUPPORTED), (conv_shape(act=2), "activation 2", UNSUPPORTED),
    (conv_shape(eps=float("nan")), "l2_eps", INVALID), (conv_shape(eps=-1.0), "l2_eps", INVALID)])
def test_conv_shapes(shape, needle, code):
    refused("gdn_causal_conv_prefill", conv_prefill(shape=shape), needle, code)
    refused("gdn_causal_conv_decode", conv_decode(shape=shape), needle, code)


@pytest.mark.parametrize("change,needle,code", [
    (dict(n=-1), "num_seqs -1", INVALID), (dict(tokens=-5), "total_tokens -5", INVALID), (dict(tokens=1 << 31), "total_tokens", UNSUPPORTED),
    (dict(slots=-1), "num_slots -1", INVALID), (dict(grid=100), "export_grid 100", INVALID), (dict(grid=-64), "export_grid", INVALID),
    (dict(count=-1), "num_export_states", INVALID), (dict(cu=None), "cu_seqlens is NULL", INVALID), (dict(init=None), "init_slot is NULL", INVALID),
    (dict(final=FAKE + 1), "final_slot", INVALID), (dict(start=FAKE + 2), "start_pos", INVALID), (dict(pool=None), "pool is NULL", INVALID),
    (dict(grid=64, offsets=None), "export_offsets is NULL", INVALID), (dict(grid=64, count=3, states=None), "export_states is NULL", INVALID),
    (dict(grid=64, count=3, eslots=FAKE + 1), "export_slots", INVALID), (dict(stride=255), "x_stride 255", INVALID),
    (dict(stride=260), "x_stride 260", INVALID), (dict(x=FAKE + 4), "x (", INVALID), (dict(weight=None), "weight is NULL", INVALID),
    (dict(bias=FAKE + 4), "bias", INVALID), (dict(y1=None), "y1 is NULL", INVALID), (dict(), "y2 is NULL", INVALID)])
def test_conv_prefill_refusals(change, needle, code):
    refused("gdn_causal_conv_prefill", conv_prefill(**change), needle, code)


@pytest.mark.parametrize("change,needle", [
    (dict(rows=-1), "num_rows -1"), (dict(slots=-3), "num_slots -3"), (dict(stride=8), "x_stride 8"), (dict(y2=None), "y2 is NULL"),
    (dict(pool=None), "conv_pool is NULL"), (dict(slot_in=None), "slot_in is NULL"), (dict(), "slot_out is NULL")])
def test_conv_decode_refusals(change, needle):
    refused("gdn_causal_conv_decode", conv_decode(**change), needle)


def params(A=FAKE, bias=FAKE, D=FAKE):
    return L.GdnSsmParams(A, bias, D, 1)


def ssm_prefill(shape=None, p=None, n=2, tokens=100, c=FAKE, dt=FAKE, y=None, pool=FAKE, slots=8, grid=0, offsets=FAKE, count=0,
                states=FAKE, ws=None, ws_bytes=0):
    return [shape or B.make_shape(2, 4, 64, 64, 1, 1.0), p or params(), n, tokens, FAKE, c, FAKE, FAKE, dt, y, pool, slots, FAKE, FAKE,
            None, grid, states, offsets, None, count, ws, ws_bytes, None]


def ssm_decode(shape=None, p=None, rows=4, c=FAKE, y=FAKE, pool=FAKE, slots=8, slot_out=None):
    return [shape or B.make_shape(2, 4, 64, 64, 1, 1.0), p or params(), rows, c, FAKE, FAKE, FAKE, y, pool, slots, FAKE, slot_out, None]


@pytest.mark.parametrize("shape,p,needle,code", [
    (B.make_shape(3, 4, 64, 64, 1, 1.0), None, "multiple of num_k_heads", UNSUPPORTED),
    (B.make_shape(2, 4, 96, 64, 1, 1.0), None, "64 or 128", UNSUPPORTED), (B.make_shape(2, 4, 64, 64, 5, 1.0), None, "dtype 5", UNSUPPORTED),
    (B.make_shape(2, 4, 64, 64, 1, float("inf")), None, "scale", INVALID), (None, params(A=None), "A is NULL", INVALID),
    (None, params(bias=FAKE + 2), "dt_bias", INVALID), (None, params(D=FAKE + 1), "D is not", INVALID)])
def test_ssm_shapes(shape, p, needle, code):
    refused("gdn_ssm_chunk_prefill", ssm_prefill(shape=shape, p=p), needle, code)
    refused("gdn_ssm_recurrent_decode", ssm_decode(shape=shape, p=p), needle, code)


@pytest.mark.parametrize("change,needle", [
    (dict(n=-2), "num_seqs -2"), (dict(tokens=-1), "total_tokens -1"), (dict(grid=65), "export_grid 65"), (dict(pool=None), "pool is NULL"),
    (dict(c=FAKE + 8), "c ("), (dict(dt=None), "dt is NULL"), (dict(grid=64, offsets=None), "export_offsets is NULL"),
    (dict(grid=64, count=2, states=None), "export_states is NULL"), (dict(), "y is NULL")])
def test_ssm_prefill_refusals(change, needle):
    refused("gdn_ssm_chunk_prefill", ssm_prefill(**change), needle)


@pytest.mark.parametrize("change,needle", [
    (dict(rows=-1), "num_rows -1"), (dict(slots=-1), "num_slots -1"), (dict(c=None), "c is NULL"), (dict(pool=FAKE + 4), "state_pool"),
    (dict(y=None), "y is NULL"), (dict(), "slot_out is NULL")])
def test_ssm_decode_refusals(change, needle):
    refused("gdn_ssm_recurrent_decode", ssm_decode(**change), needle)


def gated(rows=4, groups=2, dim=64, dtype=1, x=FAKE, xs=128, z=FAKE, zs=128, w=FAKE, eps=1e-6, act=1, y=None):
    return [rows, groups, dim, dtype, x, xs, z, zs, w, 0, eps, 0, act, y, None]


def residual(rows=4, dim=64, dtype=1, rdt=0, x=FAKE, xs=64, post=FAKE, gate=FAKE, gs=64, act=1, scale=1.0, res=FAKE, out=None, pre=FAKE,
             eps=1e-6, y=FAKE):
    return [rows, dim, dtype, rdt, x, xs, post, gate, gs, act, scale, res, out, pre, eps, y, None]


@pytest.mark.parametrize("change,needle,code", [
    (dict(rows=-1), "num_rows -1", INVALID), (dict(groups=0), "num_groups 0", INVALID), (dict(dim=0), "dim 0", INVALID),
    (dict(dim=20000), "dim 20000", UNSUPPORTED), (dict(rows=1 << 31), "launch grid", UNSUPPORTED), (dict(dtype=2), "dtype 2", UNSUPPORTED),
    (dict(act=3), "activation 3", UNSUPPORTED), (dict(eps=-1.0), "eps", INVALID), (dict(xs=100), "x_stride 100", INVALID),
    (dict(zs=100), "z_stride 100", INVALID), (dict(x=None), "x is NULL", INVALID), (dict(z=FAKE + 1), "z is not", INVALID),
    (dict(w=None), "weight is NULL", INVALID), (dict(), "y is NULL", INVALID)])
def test_gated_norm_refusals(change, needle, code):
    refused("gdn_gated_norm", gated(**change), needle, code)


@pytest.mark.parametrize("change,needle,code", [
    (dict(rows=-1), "num_rows -1", INVALID), (dict(dim=0), "dim 0", INVALID), (dict(rdt=2), "residual_dtype 2", UNSUPPORTED),
    (dict(dtype=0, rdt=1), "residual_dtype 1", UNSUPPORTED), (dict(scale=float("inf")), "residual_scale", INVALID), (dict(xs=32), "x_stride 32", INVALID),
    (dict(gs=32), "gate_stride 32", INVALID), (dict(pre=None), "pre_weight is NULL", INVALID), (dict(y=FAKE + 1), "y (", INVALID),
    (dict(post=FAKE + 2), "post_weight", INVALID), (dict(gate=FAKE + 1), "gate", INVALID), (dict(res=None), "residual is NULL", INVALID),
    (dict(), "residual_out is NULL", INVALID)])
def test_residual_norm_refusals(change, needle, code):
    refused("gdn_residual_norm", residual(**change), needle, code)


def test_empty_calls_are_no_ops():
    lib = L.library()
    assert lib.gdn_causal_conv_decode(*conv_decode(rows=0)) == B.GDN_OK
    assert lib.gdn_causal_conv_prefill(*conv_prefill(n=0, tokens=0, cu=None, init=None, final=None)) == B.GDN_OK
    assert lib.gdn_ssm_chunk_prefill(*ssm_prefill(n=0, tokens=0)) == B.GDN_OK
    assert lib.gdn_ssm_recurrent_decode(*ssm_decode(rows=0)) == B.GDN_OK
    assert lib.gdn_gated_norm(*gated(rows=0)) == B.GDN_OK
    assert lib.gdn_residual_norm(*residual(rows=0)) == B.GDN_OK
    assert B.gdn_last_error() == ""


def test_binding_checks_tensors_before_calling():
    import torch
    t = torch.zeros(2, 1, 64)
    with pytest.raises(ValueError, match="HIP device"):
        L.gdn_gated_norm(t, None, torch.ones(64), t)
    with pytest.raises(ValueError, match="HIP device"):
        L.gdn_residual_norm(t[:, 0], t[:, 0], t[:, 0])
    with pytest.raises(ValueError, match="HIP device"):
        L.gdn_ssm_recurrent_decode(t, t, t, t[:, :, 0], t[0, :, 0], t, t, t, t)
    cpu = torch.device("cpu")
    with pytest.raises(ValueError, match="shape"):
        L._dense(t, "t", torch.float32, cpu, 2, 1, 63)
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        L._dense(t, "t", torch.bfloat16, cpu, 2, 1, 64)
    with pytest.raises(ValueError, match="contiguous"):
        L._dense(t[:, :, ::2], "t", torch.float32, cpu, 2, 1, 32)
    with pytest.raises(ValueError, match="dense rows"):
        L._rows(t[:, :, ::2], "t", torch.float32, cpu, 2, 1, 32)
    wide = torch.zeros(3, 40)
    assert L._rows(wide[:, 8:24], "t", torch.float32, cpu, 3, 16) == (wide.data_ptr() + 32, 40)
    with pytest.raises(ValueError, match="activation"):
        L._activation("gelu")
