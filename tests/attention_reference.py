"""The attention layers' operators in 64 bits (test infrastructure): rotary positions, cache codes
from their definition, attention with the error bound of the kernels' arithmetic."""
import math

import torch

F64 = torch.float64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}      # largest relative rounding, eps / 2
TOP = {"e4m3": 448.0, "int8": 127.0}
STORED = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def rotary(x, positions, inv_freq, factor, interleaved):
    """x [T, H, d] turned, in 64 bits."""
    half = inv_freq.shape[0]
    angle = positions.to(F64)[:, None] * inv_freq.to(F64)
    cos, sin = (torch.cos(angle) * factor)[:, None], (torch.sin(angle) * factor)[:, None]
    y = x.to(F64).clone()
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    u, v = x[..., a].to(F64), x[..., b].to(F64)
    y[..., a], y[..., b] = u * cos - v * sin, v * cos + u * sin
    return y


def quantise(x, fmt):
    """(code values, scales) of x [..., d] from the definition; the code values as 64-bit numbers."""
    x = x.to(F64)
    most = x.abs().amax(-1, keepdim=True)
    scale = (most.clamp(min=2.0 ** -100) / TOP[fmt]).to(torch.float32)
    # a quotient of two fp32 numbers rounded to 64 bits and then to 32 is the correctly rounded fp32 quotient
    v = (x / scale.to(F64)).to(torch.float32).to(F64)
    if fmt == "int8":
        code = v.round().clamp(-127, 127)
    else:
        # the step of each value's binade, 2^-9 below the smallest normal number 2^-6; from a list, so that powers are exact
        powers = torch.tensor([2.0 ** i for i in range(-9, 8)], dtype=F64, device=x.device)
        step = powers[torch.frexp(v).exponent.clamp(-5, 11).long() + 5]
        code = ((v / step).round() * step).clamp(-448, 448)
    bad = ~torch.isfinite(most)
    nan = torch.full((), math.nan, dtype=torch.float32, device=x.device)
    return torch.where(bad, torch.zeros((), dtype=F64, device=x.device), code), torch.where(bad, nan, scale)[..., 0]


def code_values(cache):
    """A cache tensor's codes as 64-bit numbers."""
    return cache.to(torch.float32).to(F64) if cache.dtype != torch.int8 else cache.to(F64)


def attend(q, k, v, seen, scale):
    """(o, bound) of queries q [T, G, d] over keys k, v [n, d] (64-bit values), seen [T, n]; the bound is that of the kernels'
    arithmetic on outputs of q's dtype, element by element:
      output rounding               u |o|
      weights rounded (bf16 only)   2^-8 sum_p w |v|
      scores: (d + 8) 2^-24 A in the exponent, A the largest sum |q_i k_i| scale, and 16 roundings of the exponential, the scales and
      their products, numerator and denominator
      sums over n keys              2 (n + 64) 2^-24 sum_p w |v|
    """
    u = HALF_STEP[q.dtype]
    q64 = q.to(F64)
    t, g, d = q64.shape
    o, bound = torch.zeros_like(q64), torch.full_like(q64, 1e-30)
    any_seen = seen.any(1)
    used = seen.any(0)
    if not bool(any_seen.any()):
        return o, bound
    k, v, seen = k[used], v[used], seen[:, used]
    score = torch.matmul(q64.reshape(t * g, d), k.t().contiguous()).view(t, g, -1) * scale
    score = score.masked_fill(~seen[:, None], -math.inf)
    w = torch.softmax(score, -1)
    w = torch.where(seen[:, None], w, torch.zeros((), dtype=F64, device=w.device))
    # what a token does not see counts for nothing, whatever it holds
    clean = torch.nan_to_num(v, 0.0, 0.0, 0.0)
    o = torch.matmul(w.view(t * g, -1), clean).view(t, g, d)
    spread = torch.matmul(w.view(t * g, -1), clean.abs()).view(t, g, d)
    size = torch.matmul(q64.abs().reshape(t * g, d), k.abs().nan_to_num(0.0, 0.0, 0.0).t().contiguous()).view(t, g, -1)
    size = size.masked_fill(~seen[:, None], 0.0).amax(-1, keepdim=True) * abs(scale)
    eps = 2.0 ** -24 * ((d + 8) * size + 16)
    weights = 2.0 ** -8 if q.dtype == torch.bfloat16 else 0.0
    bound = u * o.abs() + (weights + 2 * eps + 2 * (k.shape[0] + 64) * 2.0 ** -24) * spread + 1e-30
    o = torch.where(any_seen[:, None, None], o, torch.zeros((), dtype=F64, device=o.device))
    return o, bound


def attention(q, cache, table, kv_block, past, new, scale, tree=None):
    """(o, bound) for requests of `past` cached and `new` new tokens, packed in order.  tree: a visibility mask [new, new] for each
    request, or None (causal)."""
    k_cache, v_cache = cache["k_cache"], cache["v_cache"]
    heads, rows = k_cache.shape[1], k_cache.shape[0]
    group = q.shape[1] // heads
    os, bounds, lo = [], [], 0
    for i, (p, n) in enumerate(zip(past, new)):
        qs = q[lo: lo + n]
        lo += n
        key = torch.arange(p + n, device=q.device)
        page = key // kv_block
        entry = torch.where(page < table.shape[1], table[i][page.clamp(max=max(0, table.shape[1] - 1))].long() if table.shape[1] else key * 0 - 1,
                            torch.full_like(key, -1))
        row = entry * kv_block + key % kv_block
        present = (entry >= 0) & (row < rows)
        seen = torch.zeros(n, p + n, dtype=torch.bool, device=q.device)
        seen[:, :p] = True
        seen[:, p:] = torch.ones(n, n, dtype=torch.bool, device=q.device).tril() if tree is None else tree[i]
        seen &= present
        at = row.clamp(0, max(0, rows - 1))
        o, b = torch.zeros(n, q.shape[1], q.shape[2], dtype=F64, device=q.device), torch.full((n, q.shape[1], q.shape[2]), 1e-30, dtype=F64, device=q.device)
        for h in range(heads if n and rows else 0):
            k, v = (code_values(c.view(torch.uint8)[at, h].view(c.dtype) if c.dtype == torch.float8_e4m3fn else c[at, h]) for c in (k_cache, v_cache))
            if cache["k_scale"] is not None:
                k, v = k * cache["k_scale"][at, h, None].to(F64), v * cache["v_scale"][at, h, None].to(F64)
            mine = slice(h * group, (h + 1) * group)
            o[:, mine], b[:, mine] = attend(qs[:, mine], k, v, seen, scale)
        os.append(o)
        bounds.append(b)
    return torch.cat(os), torch.cat(bounds)


def check(name, got, ref, bound):
    got = got.to(F64)
    assert torch.isfinite(got).all(), "%s: %d values are not finite" % (name, int((~torch.isfinite(got)).sum()))
    over = (got - ref).abs() - bound
    worst = int(over.argmax())
    assert float(over.max()) <= 0.0, "%s: off by %.3g where %.3g is allowed, at %d of %s (got %.6g, exact %.6g)" % (
        name, float((got - ref).abs().flatten()[worst]), float(bound.flatten()[worst]), worst, tuple(got.shape), float(got.flatten()[worst]),
        float(ref.flatten()[worst]))
