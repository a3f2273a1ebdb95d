"""ctypes binding of the layer operators of libgdn.so (``include/gdn_layer.h``) for torch
tensors: the step plan, the short causal convolution, the selective state space scan and
the norms around a recurrent block.

Argument marshalling only, by the same rules as ``binding``: functions carry the C entry
points' names, outputs are the caller's tensors, the call is enqueued on ``stream``
(default: torch's current stream on that device) and returns without synchronising, and
there is no other implementation to fall back to.  Tensors are contiguous except where a
row stride is taken (the convolution's x; x, z and gate of the norms): there the rows may
be columns of a wider matrix.  Weights and per-head parameters are float32.
"""
from __future__ import annotations

import ctypes
import functools
import threading
from typing import Optional, Sequence

import torch

from . import binding
from .binding import GDN_BF16, GDN_F32, GdnError, GdnShape  # noqa: F401  (GdnError: what a refused call raises)

ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "sigmoid": 2}


class GdnConvShape(ctypes.Structure):
    _fields_ = [("channels", ctypes.c_int32 * 3), ("l2_dim", ctypes.c_int32 * 3), ("width", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("l2_eps", ctypes.c_float)]


class GdnSsmParams(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p), ("D", ctypes.c_void_p),
                ("dt_softplus", ctypes.c_int32)]


_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_conv, _shape, _ssm = ctypes.POINTER(GdnConvShape), ctypes.POINTER(GdnShape), ctypes.POINTER(GdnSsmParams)

SIGNATURES = {
    "gdn_step_plan": (ctypes.c_int, [_i32, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _i32, _i64, _i64]
                      + [_vp] * 12),
    "gdn_causal_conv_prefill": (ctypes.c_int, [_conv, _i32, _i64, _vp, _vp, _i64] + [_vp] * 6 + [_i32, _vp, _vp, _vp, _i32]
                                + [_vp] * 3 + [_i64, _vp]),
    "gdn_causal_conv_decode": (ctypes.c_int, [_conv, _i32, _vp, _i64] + [_vp] * 6 + [_i32] + [_vp] * 3),
    "gdn_ssm_chunk_prefill_workspace_size": (_sz, [_shape, _i32, _i64]),
    "gdn_ssm_chunk_prefill_workspace_bound": (_sz, [_shape, _i32, _i64]),
    "gdn_ssm_chunk_prefill": (ctypes.c_int, [_shape, _ssm, _i32, _i64] + [_vp] * 7 + [_i32, _vp, _vp, _vp, _i32]
                              + [_vp] * 3 + [_i64, _vp, _sz, _vp]),
    "gdn_ssm_recurrent_decode": (ctypes.c_int, [_shape, _ssm, _i32] + [_vp] * 6 + [_i32] + [_vp] * 3),
    "gdn_gated_norm": (ctypes.c_int, [_i64, _i32, _i32, _i32, _vp, _i64, _vp, _i64, _vp, _i32, _f32, _i32, _i32, _vp, _vp]),
    "gdn_residual_norm": (ctypes.c_int, [_i64, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _i32, _f32, _vp, _vp, _vp,
                                         _f32, _vp, _vp]),
}

_lock = threading.Lock()
_lib = None
_entry = {}          # the declared entry points by name, once the library is loaded


def library():
    """libgdn.so with this module's entry points declared."""
    global _lib
    if _lib is None:
        with _lock:
            lib = binding.library()
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
                _entry[name] = fn
            _lib = lib
    return _lib


# ---------------------------------------------------------------- marshalling

# A small call's time is its marshalling, not its kernel: tensors are checked in one condition
# (the reason is worked out only for a refusal), shapes are kept as C structures by their values,
# and the current stream is taken as the handle it is instead of through a Stream object.

_raw_stream = torch._C._cuda_getCurrentRawStream


def _enqueue(name, device, stream, *args):
    fn = _entry.get(name) or getattr(library(), name)
    index = device.index
    if torch.cuda.current_device() == index:
        status = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if status:
        binding._check(status)


def _device(t, name):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError("%s must be on a HIP device, got %s" % (name, dev))
    return dev


def _code(t, name="tensors"):
    if t.dtype is torch.bfloat16:
        return GDN_BF16
    if t.dtype is torch.float32:
        return GDN_F32
    raise ValueError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))


def _refuse(t, name, dtype, device, shape):
    if t.dtype is not dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _dense(t, name, dtype, device, *shape):
    """Address of a contiguous tensor of this dtype, device and shape."""
    if t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, device, shape)
    raise ValueError("%s must be contiguous" % name)


def _maybe(t, name, dtype, device, *shape):
    return None if t is None else _dense(t, name, dtype, device, *shape)


def _rows(t, name, dtype, device, *shape):
    """Address and row stride of a tensor whose rows are dense but may be part of wider ones."""
    if t.dtype is not dtype or t.device != device or t.shape != shape:
        _refuse(t, name, dtype, device, shape)
    strides = t.stride()
    width = 1
    for size, step in zip(shape[:0:-1], strides[:0:-1]):
        if size != 1 and step != width:
            raise ValueError("%s must have dense rows, got strides %s" % (name, strides))
        width *= size
    return t.data_ptr(), strides[0] if shape[0] > 1 else -(-width // 8) * 8


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError("activation must be one of %s, got %r" % (list(ACTIVATIONS), name)) from None


def _exports(device, num_seqs, export_grid, export_states, export_offsets, export_slots, dtype, entry):
    """(states, offsets, slots, count) of a prefill's exports; entry: the shape of one state."""
    if not export_grid:
        return None, None, None, 0
    if export_offsets is None:
        raise ValueError("export_offsets is required with an export_grid")
    offsets = _dense(export_offsets, "export_offsets", torch.int32, device, num_seqs + 1)
    if export_slots is not None:
        n = export_slots.shape[0]
        return None, offsets, _dense(export_slots, "export_slots", torch.int32, device, n), n
    if export_states is None:
        return None, offsets, None, 0
    n = export_states.shape[0]
    return _dense(export_states, "export_states", dtype, device, n, *entry), offsets, None, n


# ---------------------------------------------------------------- step plan

def alloc_step_plan(num_requests: int, num_decode_rows: int, token_capacity: int, export_capacity: int, device,
                    kv: bool = True) -> dict:
    """The output tensors of gdn_step_plan, by the names it takes them under."""
    n = num_requests - num_decode_rows
    sizes = dict(slot_in=num_decode_rows, slot_out=num_decode_rows, cu_seqlens=n + 1, start_pos=n, init_slot=n, final_slot=n,
                 export_offsets=n + 1, export_slots=export_capacity, token_request=token_capacity, token_position=token_capacity)
    out = {k: torch.empty(v, dtype=torch.int32, device=device) for k, v in sizes.items()}
    if kv:
        out["token_kv_slot"] = torch.empty(token_capacity, dtype=torch.int64, device=device)
    return out


def gdn_step_plan(computed, new_tokens, state_table, run_slot, *, num_decode_rows: int, state_block: int, slot_in, slot_out,
                  cu_seqlens, start_pos, init_slot, final_slot, export_offsets, export_slots=None, token_request=None,
                  token_position=None, token_kv_slot=None, kv_table=None, kv_block: int = 0, stream=None) -> None:
    """One step's slots, packed offsets, export list and token maps from the requests' lengths
    and block tables (see include/gdn_layer.h; outputs: alloc_step_plan).  A decode row continues
    a cached state (computed >= 1); a request's first token is planned as a prefill."""
    dev = _device(computed, "computed")
    i32 = torch.int32
    r, b = computed.shape[0], int(num_decode_rows)
    if not 0 <= b <= r:
        raise ValueError("num_decode_rows %d is not in [0, %d]" % (b, r))
    n = r - b
    if state_table.dim() != 2 or (kv_table is not None and kv_table.dim() != 2):
        raise ValueError("state_table and kv_table must have 2 dims")
    width = state_table.shape[1]
    kv_width = 0 if kv_table is None else kv_table.shape[1]
    tokens = 0
    for t in (token_request, token_position, token_kv_slot):
        if t is not None:
            tokens = t.shape[0]
    exports = 0 if export_slots is None else export_slots.shape[0]
    _enqueue("gdn_step_plan", dev, stream, r, b, _dense(computed, "computed", i32, dev, r),
             _dense(new_tokens, "new_tokens", i32, dev, r), _dense(state_table, "state_table", i32, dev, r, width), width,
             int(state_block), _dense(run_slot, "run_slot", i32, dev, r),
             _maybe(kv_table, "kv_table", i32, dev, r, kv_width), kv_width, int(kv_block), tokens, exports,
             _dense(slot_in, "slot_in", i32, dev, b), _dense(slot_out, "slot_out", i32, dev, b),
             _dense(cu_seqlens, "cu_seqlens", i32, dev, n + 1), _dense(start_pos, "start_pos", i32, dev, n),
             _dense(init_slot, "init_slot", i32, dev, n), _dense(final_slot, "final_slot", i32, dev, n),
             _dense(export_offsets, "export_offsets", i32, dev, n + 1),
             _maybe(export_slots, "export_slots", i32, dev, exports),
             _maybe(token_request, "token_request", i32, dev, tokens),
             _maybe(token_position, "token_position", i32, dev, tokens),
             _maybe(token_kv_slot, "token_kv_slot", torch.int64, dev, tokens))


# ---------------------------------------------------------------- short causal convolution

_OUTS = ("outs[0]", "outs[1]", "outs[2]")


@functools.lru_cache(maxsize=256)
def _conv_shape(channels, l2_dim, width, dtype, activation, l2_eps):
    return GdnConvShape(channels, l2_dim, width, dtype, activation, l2_eps)


@functools.lru_cache(maxsize=256)
def _head_shape(groups, heads, d_k, d_v, dtype, scale):
    return GdnShape(groups, heads, d_k, d_v, dtype, scale)


def _conv_common(x, weight, bias, outs, conv_pool, activation, l2_dims, l2_eps):
    dev = _device(x, "x")
    if x.dim() != 2 or weight.dim() != 2 or conv_pool.dim() != 3:
        raise ValueError("x and weight must have 2 dims and conv_pool 3")
    if not 1 <= len(outs) <= 3 or len(l2_dims) < len(outs):
        raise ValueError("one to three outputs are taken, with an l2_dims entry for each")
    (tokens, channels), width, dtype = x.shape, weight.shape[1], x.dtype
    y, runs, l2 = [None, None, None], [0, 0, 0], [0, 0, 0]
    for i, o in enumerate(outs):
        runs[i], l2[i] = o.shape[-1], int(l2_dims[i])
        y[i] = _dense(o, _OUTS[i], dtype, dev, tokens, runs[i])
    if sum(runs) != channels:
        raise ValueError("the outputs hold %d channels, x has %d" % (sum(runs), channels))
    shape = _conv_shape(tuple(runs), tuple(l2), width, _code(x, "x"), _activation(activation), float(l2_eps))
    px, stride = _rows(x, "x", dtype, dev, tokens, channels)
    slots = conv_pool.shape[0]
    return dev, shape, tokens, (px, stride, _dense(weight, "weight", torch.float32, dev, channels, width),
                                _maybe(bias, "bias", torch.float32, dev, channels), *y,
                                _dense(conv_pool, "conv_pool", dtype, dev, slots, width - 1, channels), slots), (width - 1, channels)


def gdn_causal_conv_prefill(x, weight, bias, outs: Sequence[torch.Tensor], conv_pool, cu_seqlens, init_slot, final_slot, *,
                            activation: Optional[str] = "silu", l2_dims: Sequence[int] = (0, 0, 0), l2_eps: float = 1e-6,
                            start_pos=None, export_grid: int = 0, export_states=None, export_offsets=None, export_slots=None,
                            stream=None) -> None:
    """Short causal convolution of packed sequences: x [T, C] into outs, dense [T, c_i] each, the
    tails of the inputs in conv_pool [num_slots, width - 1, C] (see include/gdn_layer.h)."""
    dev, shape, tokens, args, entry = _conv_common(x, weight, bias, outs, conv_pool, activation, l2_dims, l2_eps)
    n = cu_seqlens.shape[0] - 1
    i32 = torch.int32
    states, offsets, slots, count = _exports(dev, n, export_grid, export_states, export_offsets, export_slots, x.dtype, entry)
    _enqueue("gdn_causal_conv_prefill", dev, stream, shape, n, tokens, _dense(cu_seqlens, "cu_seqlens", i32, dev, n + 1), *args,
             _dense(init_slot, "init_slot", i32, dev, n), _dense(final_slot, "final_slot", i32, dev, n),
             _maybe(start_pos, "start_pos", i32, dev, n), int(export_grid), states, offsets, slots, count)


def gdn_causal_conv_decode(x, weight, bias, outs: Sequence[torch.Tensor], conv_pool, slot_in, slot_out, *,
                           activation: Optional[str] = "silu", l2_dims: Sequence[int] = (0, 0, 0), l2_eps: float = 1e-6,
                           stream=None) -> None:
    """The convolution of one token of each of x.shape[0] cached rows (see include/gdn_layer.h)."""
    dev, shape, rows, args, _ = _conv_common(x, weight, bias, outs, conv_pool, activation, l2_dims, l2_eps)
    _enqueue("gdn_causal_conv_decode", dev, stream, shape, rows, *args, _dense(slot_in, "slot_in", torch.int32, dev, rows),
             _dense(slot_out, "slot_out", torch.int32, dev, rows))


# ---------------------------------------------------------------- selective state space scan

def _ssm_common(c, b, x, dt, A, y, state_pool, dt_bias, D, dt_softplus, scale):
    dev = _device(x, "x")
    if x.dim() != 3 or c.dim() != 3:
        raise ValueError("x and c must have 3 dims, got %s and %s" % (tuple(x.shape), tuple(c.shape)))
    (tokens, heads, d_v), groups, d_k, dtype, f32 = x.shape, c.shape[1], c.shape[2], x.dtype, torch.float32
    shape = _head_shape(groups, heads, d_k, d_v, _code(x, "x"), float(scale))
    params = GdnSsmParams(_dense(A, "A", f32, dev, heads), _maybe(dt_bias, "dt_bias", f32, dev, heads),
                          _maybe(D, "D", f32, dev, heads), 1 if dt_softplus else 0)
    slots = state_pool.shape[0]
    return dev, shape, params, tokens, (
        _dense(c, "c", dtype, dev, tokens, groups, d_k), _dense(b, "b", dtype, dev, tokens, groups, d_k),
        _dense(x, "x", dtype, dev, tokens, heads, d_v), _dense(dt, "dt", f32, dev, tokens, heads),
        _dense(y, "y", dtype, dev, tokens, heads, d_v),
        _dense(state_pool, "state_pool", f32, dev, slots, heads, d_k, d_v), slots), (heads, d_k, d_v)


def alloc_ssm_workspace(c, x, num_seqs: int, *, smaller_calls: bool = False) -> Optional[torch.Tensor]:
    """A uint8 device buffer of the size gdn_ssm_chunk_prefill needs for these inputs and
    num_seqs sequences, or None when it needs none.  With smaller_calls it serves every call
    with at most as many sequences and tokens too (which may need more than this one)."""
    shape = GdnShape(c.shape[1], x.shape[1], c.shape[2], x.shape[2], _code(x, "x"), 1.0)
    query = library().gdn_ssm_chunk_prefill_workspace_bound if smaller_calls else library().gdn_ssm_chunk_prefill_workspace_size
    with torch.cuda.device(_device(x, "x")):
        n = int(query(shape, int(num_seqs), x.shape[0]))
    return torch.empty(n, dtype=torch.uint8, device=x.device) if n else None


def gdn_ssm_chunk_prefill(c, b, x, dt, A, y, cu_seqlens, state_pool, init_slot, final_slot, *, dt_bias=None, D=None,
                          dt_softplus: bool = True, scale: float = 1.0, workspace=None, start_pos=None, export_grid: int = 0,
                          export_states=None, export_offsets=None, export_slots=None, stream=None) -> None:
    """Selective state space scan of packed sequences (see include/gdn_layer.h; workspace:
    alloc_ssm_workspace)."""
    dev, shape, params, tokens, args, entry = _ssm_common(c, b, x, dt, A, y, state_pool, dt_bias, D, dt_softplus, scale)
    n = cu_seqlens.shape[0] - 1
    i32 = torch.int32
    states, offsets, slots, count = _exports(dev, n, export_grid, export_states, export_offsets, export_slots, torch.float32, entry)
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
        ws = _dense(workspace, "workspace", workspace.dtype, dev, *workspace.shape)
    _enqueue("gdn_ssm_chunk_prefill", dev, stream, shape, params, n, tokens,
             _dense(cu_seqlens, "cu_seqlens", i32, dev, n + 1), *args, _dense(init_slot, "init_slot", i32, dev, n),
             _dense(final_slot, "final_slot", i32, dev, n), _maybe(start_pos, "start_pos", i32, dev, n), int(export_grid),
             states, offsets, slots, count, ws, ws_bytes)


def gdn_ssm_recurrent_decode(c, b, x, dt, A, y, state_pool, slot_in, slot_out, *, dt_bias=None, D=None,
                             dt_softplus: bool = True, scale: float = 1.0, stream=None) -> None:
    """The scan of one token of each of x.shape[0] cached rows (see include/gdn_layer.h)."""
    dev, shape, params, rows, args, _ = _ssm_common(c, b, x, dt, A, y, state_pool, dt_bias, D, dt_softplus, scale)
    _enqueue("gdn_ssm_recurrent_decode", dev, stream, shape, params, rows, *args,
             _dense(slot_in, "slot_in", torch.int32, dev, rows), _dense(slot_out, "slot_out", torch.int32, dev, rows))


# ---------------------------------------------------------------- norms

def gdn_gated_norm(x, z, weight, y, *, eps: float = 1e-6, gate_first: bool = False, activation: Optional[str] = "silu",
                   stream=None) -> None:
    """Gated RMS norm over the last dim of x [T, groups, dim]; z the gate (or None), weight [dim] or
    [groups, dim], y dense (see include/gdn_layer.h)."""
    dev = _device(x, "x")
    if x.dim() != 3:
        raise ValueError("x must have 3 dims, got shape %s" % (tuple(x.shape),))
    (rows, groups, dim), dtype = x.shape, x.dtype
    px, xs = _rows(x, "x", dtype, dev, rows, groups, dim)
    pz, zs = (None, 0) if z is None else _rows(z, "z", dtype, dev, rows, groups, dim)
    per_group = weight.dim() == 2
    pw = _dense(weight, "weight", torch.float32, dev, *((groups, dim) if per_group else (dim,)))
    _enqueue("gdn_gated_norm", dev, stream, rows, groups, dim, _code(x, "x"), px, xs, pz, zs, pw, 1 if per_group else 0, eps,
             1 if gate_first else 0, _activation(activation), _dense(y, "y", dtype, dev, rows, groups, dim))


def gdn_residual_norm(x, residual, residual_out, y=None, *, post_weight=None, gate=None, activation: Optional[str] = "silu",
                      residual_scale: float = 1.0, pre_weight=None, eps: float = 1e-6, stream=None) -> None:
    """residual_out = residual + residual_scale act(gate) rms(x) post_weight and, with y,
    y = rms(residual_out) pre_weight (see include/gdn_layer.h)."""
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must have 2 dims, got shape %s" % (tuple(x.shape),))
    (rows, dim), dtype, f32 = x.shape, x.dtype, torch.float32
    if y is not None and pre_weight is None:
        raise ValueError("pre_weight is required with y")
    px, xs = _rows(x, "x", dtype, dev, rows, dim)
    pg, gs = (None, 0) if gate is None else _rows(gate, "gate", dtype, dev, rows, dim)
    _enqueue("gdn_residual_norm", dev, stream, rows, dim, _code(x, "x"), _code(residual, "residual"), px, xs,
             _maybe(post_weight, "post_weight", f32, dev, dim), pg, gs, _activation(activation), residual_scale,
             _dense(residual, "residual", residual.dtype, dev, rows, dim),
             _dense(residual_out, "residual_out", residual.dtype, dev, rows, dim),
             _maybe(pre_weight, "pre_weight", f32, dev, dim), eps, _maybe(y, "y", dtype, dev, rows, dim))
