"""ctypes binding of the attention layers' operators of libgdn.so (``include/gdn_attention.h``)
for torch tensors: rotary positions, the paged key/value cache in its formats, attention of
prompts and of decode rows over it.

Argument marshalling by the rules of ``binding`` and ``layer``: functions carry the C entry
points' names, outputs are the caller's tensors, the call is enqueued on ``stream`` (default:
torch's current stream on that device) and returns without synchronising.  A cache is two
tensors [num_rows, heads, head_dim] (``alloc_kv_cache``): of the activations' dtype, or
torch.float8_e4m3fn or torch.int8 with float32 scales [num_rows, heads] beside them.

Two helpers compute on the host what a model keeps: ``rotary_frequencies`` and ``tree_masks``.
"""
from __future__ import annotations

import ctypes
import math
import threading
from typing import Optional, Sequence, Tuple

import torch

from . import binding, layer
from .binding import GdnError  # noqa: F401  (what a refused call raises)
from .layer import _code, _dense, _device, _maybe, _rows

GDN_CACHE_PLAIN, GDN_CACHE_E4M3, GDN_CACHE_INT8 = 0, 1, 2
FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_FORMAT_CODES = {torch.float8_e4m3fn: GDN_CACHE_E4M3, torch.int8: GDN_CACHE_INT8}


class GdnKvCache(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("format", ctypes.c_int32),
                ("num_rows", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class GdnRotaryShape(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float)]


_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_cache_p, _rotary_p = ctypes.POINTER(GdnKvCache), ctypes.POINTER(GdnRotaryShape)

SIGNATURES = {
    "gdn_rotary": (ctypes.c_int, [_rotary_p, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]),
    "gdn_kv_cache_write": (ctypes.c_int, [_cache_p, _i64, _vp, _i64, _vp, _i64, _vp, _vp]),
    "gdn_kv_cache_read": (ctypes.c_int, [_cache_p, _i64, _vp, _vp, _vp, _vp]),
    "gdn_attention_prefill": (ctypes.c_int, [_cache_p, _i32, _f32, _i32, _i64, _vp, _vp, _vp, _i64, _vp, _i32, _i32, _vp, _vp]),
    "gdn_attention_decode_workspace_size": (_sz, [_cache_p, _i32, _i32, _i32, _i64]),
    "gdn_attention_decode": (ctypes.c_int, [_cache_p, _i32, _f32, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _i32, _i32, _i64, _vp, _vp,
                                            _sz, _vp]),
}

_lock = threading.Lock()
_lib = None


def library():
    """libgdn.so with this module's entry points declared."""
    global _lib
    if _lib is None:
        with _lock:
            lib = layer.library()
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
                layer._entry[name] = fn
            _lib = lib
    return _lib


def _enqueue(name, device, stream, *args):
    if _lib is None:
        library()
    layer._enqueue(name, device, stream, *args)


# ---------------------------------------------------------------- what a model keeps

def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: Optional[str] = None, factor: float = 1.0,
                       original_length: int = 0, turns: Tuple[float, float] = (1.0, 32.0), device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq, attention_factor) of gdn_rotary: float32 [rotary_dim / 2] frequencies base^(-2 i / rotary_dim), formed in
    64 bits, and what the turned part is multiplied with.  ``scaling`` stretches them for contexts `factor` times as long:

      None          as they are
      "linear"      all divided by factor
      "base"        base times factor^(r / (r - 2)): the fastest pair keeps its frequency, the slowest is divided by factor
      "ramp"        by the turns a pair makes over original_length: at least turns[1] keep theirs, at most turns[0] are divided by
                    factor, linear in the pair's number in between (Peng et al., YaRN); attention_factor 0.1 ln(factor) + 1
      "wavelength"  the same borders, linear in the number of turns in between
    """
    r = int(rotary_dim)
    if r < 2 or r % 2:
        raise ValueError("rotary_dim must be an even number of at least 2, got %r" % (rotary_dim,))
    if not (base > 1.0 and factor >= 1.0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base must be above 1 and factor at least 1, got %r and %r" % (base, factor))
    pair = torch.arange(0, r, 2, dtype=torch.float64) / r
    freq, attention_factor = float(base) ** -pair, 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "base":
        if r > 2:
            freq = (base * factor ** (r / (r - 2.0))) ** -pair
    elif scaling in ("ramp", "wavelength"):
        slow, fast = (float(t) for t in turns)
        if original_length < 1 or not 0.0 < slow < fast:
            raise ValueError("scaling %r needs original_length and 0 < turns[0] < turns[1], got %r and %r" % (scaling, original_length, turns))
        if scaling == "ramp":
            def number(t):      # of the pair that makes t turns over the original length
                return r * math.log(original_length / (t * 2.0 * math.pi)) / (2.0 * math.log(base))

            low, high = max(math.floor(number(fast)), 0), min(math.ceil(number(slow)), r - 1)
            keep = 1.0 - ((torch.arange(r // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
            attention_factor = 0.1 * math.log(factor) + 1.0
        else:
            keep = ((original_length * freq / (2.0 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
    elif scaling is not None:
        raise ValueError("scaling must be None, 'linear', 'base', 'ramp' or 'wavelength', got %r" % (scaling,))
    return freq.to(torch.float32).to(device), attention_factor


def tree_masks(parents: Sequence[Sequence[int]], device=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(tree_mask, depth) of gdn_attention_decode for rows of drafted tokens: parents[b][i] is the number of token i's
    parent in row b, below i, or -1 for a child of the context.  tree_mask int64 and depth int32, both
    [rows * tokens]; token i's rotary position is computed[b] + depth."""
    masks, depths = [], []
    for row in parents:
        if len(row) != len(parents[0]) or not 1 <= len(row) <= 64:
            raise ValueError("rows must hold the same number of tokens, 1 to 64")
        seen, depth = [], []
        for i, p in enumerate(row):
            if not -1 <= p < i:
                raise ValueError("the parent of token %d must be -1 or an earlier token, got %r" % (i, p))
            seen.append((1 << i) | (seen[p] if p >= 0 else 0))
            depth.append(depth[p] + 1 if p >= 0 else 0)
        masks += [m - (1 << 64) if m >> 63 else m for m in seen]
        depths += depth
    return torch.tensor(masks, dtype=torch.int64, device=device), torch.tensor(depths, dtype=torch.int32, device=device)


# ---------------------------------------------------------------- rotary positions

def _head_rows(t, name, dtype, device, tokens, heads, dim):
    """layer._rows of [tokens, heads, dim], in one condition where the heads are dense."""
    if t.dtype is dtype and t.get_device() == device.index and t.shape == (tokens, heads, dim):
        row, head, one = t.stride()
        if one == 1 and head == dim and tokens > 1:
            return t.data_ptr(), row
    return _rows(t, name, dtype, device, tokens, heads, dim)


def gdn_rotary(q, k, positions, inv_freq, *, q_out=None, k_out=None, interleaved: bool = False, attention_factor: float = 1.0,
               stream=None) -> None:
    """Rotary positions of q [T, heads, head_dim] and k (either may be None) into q_out and k_out, in place where those are None
    (see include/gdn_attention.h; inv_freq: rotary_frequencies)."""
    first = k if q is None else q
    if first is None:
        raise ValueError("q or k is required")
    dev, dtype, size = _device(first, "k" if q is None else "q"), first.dtype, first.shape
    if len(size) != 3:
        raise ValueError("q and k must have 3 dims, got shape %s" % (tuple(size),))
    tokens, q_heads, head_dim = size
    pq = sq = oq = soq = pk = sk = ok = sok = None
    k_heads = 0
    if q is not None:
        pq, sq = _head_rows(q, "q", dtype, dev, tokens, q_heads, head_dim)
        oq, soq = (pq, sq) if q_out is None else _head_rows(q_out, "q_out", dtype, dev, tokens, q_heads, head_dim)
    else:
        q_heads = sq = soq = 0
        if q_out is not None:
            raise ValueError("q_out is given without q")
    if k is not None:
        if k.dim() != 3 or k.shape[2] != head_dim:
            raise ValueError("q and k must be [T, heads, %d], k is %s" % (head_dim, tuple(k.shape)))
        k_heads = k.shape[1]
        pk, sk = _head_rows(k, "k", dtype, dev, tokens, k_heads, head_dim)
        ok, sok = (pk, sk) if k_out is None else _head_rows(k_out, "k_out", dtype, dev, tokens, k_heads, head_dim)
    else:
        sk = sok = 0
        if k_out is not None:
            raise ValueError("k_out is given without k")
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must have 1 dim, got shape %s" % (tuple(inv_freq.shape),))
    shape = GdnRotaryShape(q_heads, k_heads, head_dim, 2 * inv_freq.shape[0], _code(first, "q and k"), 1 if interleaved else 0,
                           attention_factor)
    _enqueue("gdn_rotary", dev, stream, shape, tokens, _dense(positions, "positions", torch.int32, dev, tokens),
             _dense(inv_freq, "inv_freq", torch.float32, dev, inv_freq.shape[0]), pq, sq, pk, sk, oq, soq, ok, sok)


# ---------------------------------------------------------------- the cache

def alloc_kv_cache(num_rows: int, num_heads: int, head_dim: int, dtype: torch.dtype, device, format: Optional[str] = None) -> dict:
    """The tensors of a cache of num_rows rows (pages times kv_block), by the names the entry points take them under:
    format None (values of `dtype`), "e4m3" or "int8".  Not initialised: a row is written before it is read."""
    if format is not None and format not in FORMATS:
        raise ValueError("format must be None or one of %s, got %r" % (list(FORMATS), format))
    stored = dtype if format is None else FORMATS[format]
    out = {n: torch.empty(num_rows, num_heads, head_dim, dtype=stored, device=device) for n in ("k_cache", "v_cache")}
    for n in ("k_scale", "v_scale"):
        out[n] = None if format is None else torch.empty(num_rows, num_heads, dtype=torch.float32, device=device)
    return out


def _cache(k_cache, v_cache, k_scale, v_scale, like, device):
    """The C description of a cache for activations like `like`."""
    size = k_cache.shape
    if len(size) != 3:
        raise ValueError("k_cache must have 3 dims, got shape %s" % (tuple(size),))
    rows, heads, head_dim = size
    stored, dtype = k_cache.dtype, _code(like, "activations")
    form = GDN_CACHE_PLAIN if stored is like.dtype else _FORMAT_CODES.get(stored)
    if form is None:
        raise ValueError("k_cache must be %s, torch.float8_e4m3fn or torch.int8, got %s" % (like.dtype, stored))
    ks = vs = None
    if form != GDN_CACHE_PLAIN:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        ks = _dense(k_scale, "k_scale", torch.float32, device, rows, heads)
        vs = _dense(v_scale, "v_scale", torch.float32, device, rows, heads)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale are given for a cache that has none")
    return GdnKvCache(heads, head_dim, dtype, form, rows, _dense(k_cache, "k_cache", stored, device, rows, heads, head_dim),
                      _dense(v_cache, "v_cache", stored, device, rows, heads, head_dim), ks, vs)


def gdn_kv_cache_write(k, v, slots, k_cache, v_cache, *, k_scale=None, v_scale=None, stream=None) -> None:
    """k, v [T, heads, head_dim] into cache rows slots [T] (int64, see include/gdn_attention.h)."""
    dev = _device(k, "k")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, k, dev)
    tokens = k.shape[0]
    shape = (tokens, cache.num_heads, cache.head_dim)
    pk, sk = _head_rows(k, "k", k.dtype, dev, *shape)
    pv, sv = _head_rows(v, "v", k.dtype, dev, *shape)
    _enqueue("gdn_kv_cache_write", dev, stream, cache, tokens, pk, sk, pv, sv, _dense(slots, "slots", torch.int64, dev, tokens))


def gdn_kv_cache_read(slots, k_cache, v_cache, k_out, v_out, *, k_scale=None, v_scale=None, stream=None) -> None:
    """The values of cache rows slots [T] into k_out and v_out, dense (see include/gdn_attention.h)."""
    dev = _device(k_out, "k_out")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, k_out, dev)
    shape = (slots.shape[0], cache.num_heads, cache.head_dim)
    _enqueue("gdn_kv_cache_read", dev, stream, cache, shape[0], _dense(slots, "slots", torch.int64, dev, shape[0]),
             _dense(k_out, "k_out", k_out.dtype, dev, *shape), _dense(v_out, "v_out", k_out.dtype, dev, *shape))


# ---------------------------------------------------------------- attention

def _attention(q, k_cache, v_cache, k_scale, v_scale, o, kv_table, sequences):
    dev = _device(q, "q")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, q, dev)
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError("q must be [T, heads, %d], got shape %s" % (cache.head_dim, tuple(shape)))
    if kv_table.dim() != 2:
        raise ValueError("kv_table must have 2 dims, got shape %s" % (tuple(kv_table.shape),))
    pq, sq = _head_rows(q, "q", q.dtype, dev, *shape)
    width = kv_table.shape[1]
    return dev, cache, pq, sq, _dense(kv_table, "kv_table", torch.int32, dev, sequences, width), width, \
        _dense(o, "o", q.dtype, dev, *shape)


def gdn_attention_prefill(q, k_cache, v_cache, o, cu_seqlens, start_pos, kv_table, *, kv_block: int, scale: float, k_scale=None,
                          v_scale=None, stream=None) -> None:
    """Causal attention of packed prompts q [T, heads, head_dim] over their cached keys (see include/gdn_attention.h);
    start_pos [N] or None."""
    n = cu_seqlens.shape[0] - 1
    dev, cache, pq, sq, table, width, po = _attention(q, k_cache, v_cache, k_scale, v_scale, o, kv_table, n)
    _enqueue("gdn_attention_prefill", dev, stream, cache, q.shape[1], scale, n, q.shape[0],
             _dense(cu_seqlens, "cu_seqlens", torch.int32, dev, n + 1), _maybe(start_pos, "start_pos", torch.int32, dev, n), pq, sq, table,
             width, int(kv_block), po)


def alloc_attention_workspace(q, k_cache, *, tokens_per_row: int, max_keys: int) -> Optional[torch.Tensor]:
    """A uint8 device buffer that gdn_attention_decode takes for q and every call with fewer rows, tokens of each or keys, or
    None when it needs none."""
    cache = GdnKvCache(k_cache.shape[1], k_cache.shape[2], _code(q, "q"), GDN_CACHE_PLAIN, 0, None, None, None, None)
    with torch.cuda.device(_device(q, "q")):
        n = int(library().gdn_attention_decode_workspace_size(cache, q.shape[1], q.shape[0] // int(tokens_per_row), int(tokens_per_row),
                                                              int(max_keys)))
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def gdn_attention_decode(q, k_cache, v_cache, o, computed, kv_table, *, kv_block: int, scale: float, tokens_per_row: int = 1,
                         tree_mask=None, max_keys: int = 0, workspace=None, k_scale=None, v_scale=None, stream=None) -> None:
    """Attention of tokens_per_row tokens of each of len(computed) cached rows, q [rows * tokens, heads, head_dim], over their
    cached keys: one token, a chain or a tree of drafted tokens (see include/gdn_attention.h; tree_mask: tree_masks,
    workspace: alloc_attention_workspace)."""
    rows, per = computed.shape[0], int(tokens_per_row)
    dev, cache, pq, sq, table, width, po = _attention(q, k_cache, v_cache, k_scale, v_scale, o, kv_table, rows)
    if q.shape[0] != rows * per:
        raise ValueError("q has %d tokens, expected %d rows of %d" % (q.shape[0], rows, per))
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
        ws = _dense(workspace, "workspace", workspace.dtype, dev, *workspace.shape)
    _enqueue("gdn_attention_decode", dev, stream, cache, q.shape[1], scale, rows, per, _dense(computed, "computed", torch.int32, dev, rows),
             _maybe(tree_mask, "tree_mask", torch.int64, dev, rows * per), pq, sq, table, width, int(kv_block), int(max_keys), po, ws,
             ws_bytes)
