"""Plain fp64 forms of the layer operators (include/gdn_layer.h), one request, token or
row at a time in numpy, and the error bounds the GPU tests hold the kernels to.

A bound counts roundings.  U = 2^-24 is half a step of fp32, HALF[dtype] half a step of the
stored type, both relative; a sum of n terms rounded at each step is off by at most n U
times the sum of their magnitudes, an exp of an exponent known to e is off by e relative."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


ACT = {"none": lambda v: v, "silu": lambda v: v * sigmoid(v), "sigmoid": sigmoid}


# ---------------------------------------------------------------- step plan

def plan(computed, new, state_table, run_slot, B, block, kv_table, kv_block, token_capacity, export_capacity):
    R = len(computed)
    computed = [max(0, int(c)) for c in computed]
    new = [int(n) for n in new]

    def slot(r, p):
        if p <= 0:
            return -1
        if p % block:
            return int(run_slot[r])
        j = p // block - 1
        return int(state_table[r][j]) if j < state_table.shape[1] else -1

    out = dict(slot_in=[], slot_out=[], cu_seqlens=[0], start_pos=[], init_slot=[], final_slot=[], export_offsets=[0])
    exports, owner, pos = [], [], []
    for r in range(B):
        live = new[r] > 0
        out["slot_in"].append(slot(r, computed[r]) if live else -1)
        out["slot_out"].append(slot(r, computed[r] + 1) if live else -1)
        owner.append(r if live else -1)
        pos.append(computed[r] if live else -1)
    for r in range(B, R):
        s, n = computed[r], max(0, new[r])
        out["cu_seqlens"].append(out["cu_seqlens"][-1] + n)
        out["start_pos"].append(s)
        out["init_slot"].append(slot(r, s))
        out["final_slot"].append(slot(r, s + n))
        for p in range((s // block + 1) * block, s + n + 1, block):
            exports.append(-1 if p == s + n else slot(r, p))
        out["export_offsets"].append(len(exports))
        owner += [r] * n
        pos += list(range(s, s + n))
    kv = []
    for r, p in zip(owner, pos):
        j = p // kv_block if kv_block else 0
        if r < 0 or kv_table is None or j >= kv_table.shape[1] or kv_table[r][j] < 0:
            kv.append(-1)
        else:
            kv.append(int(kv_table[r][j]) * kv_block + p % kv_block)

    def fill(v, n):
        return (v + [-1] * max(0, n - len(v)))[:n]

    out["export_slots"] = fill(exports, export_capacity)
    out["token_request"], out["token_position"] = fill(owner, token_capacity), fill(pos, token_capacity)
    out["token_kv_slot"] = fill(kv, token_capacity)
    return out


# ---------------------------------------------------------------- short causal convolution

def conv(x, lengths, tails, weight, bias, act, channels, l2, eps, dtype):
    """x [T, C] float64, tails [n, W - 1, C]: (outputs, their bounds, joined inputs of each sequence).
    Roundings of a: W products and additions and the bias; of the activation: an exp (its
    argument's error enters relative), an addition, a division; of the norm: d / 2 for the sum
    under the root, and four more."""
    W, C = weight.shape[1], x.shape[1]
    ys, es, joined, at = [], [], [], 0
    for i, n in enumerate(lengths):
        j = np.concatenate([tails[i], x[at:at + n]])
        joined.append(j)
        at += n
        a = np.zeros((n, C)) + (0.0 if bias is None else bias)
        mag = np.abs(a)
        for k in range(W):
            a = a + weight[:, k] * j[k:k + n]
            mag = mag + np.abs(weight[:, k] * j[k:k + n])
        ea = (W + 1) * U * mag
        y = ACT[act](a)
        e = 1.1 * ea + (12 + 2 * np.abs(a)) * U * np.abs(y) if act == "silu" else ea   # |silu'| <= 1.1
        ys.append(y)
        es.append(e)
    y, e = np.concatenate(ys), np.concatenate(es)
    outs, bounds, at = [], [], 0
    for c, d in zip(channels, l2):
        yy, ee = y[:, at:at + c], e[:, at:at + c]
        at += c
        if d:
            yy, ee = yy.reshape(len(yy), -1, d), ee.reshape(len(ee), -1, d)
            norm = np.sqrt((yy * yy).sum(-1, keepdims=True) + eps)
            en = np.sqrt((ee * ee).sum(-1, keepdims=True))
            ee = (ee + np.abs(yy) * (en / norm + (d / 2 + 4) * U)) / norm
            yy = yy / norm
            yy, ee = yy.reshape(len(yy), c), ee.reshape(len(ee), c)
        outs.append(yy)
        bounds.append(HALF[dtype] * np.abs(yy) + 1.01 * ee + 1e-30)
    return outs, bounds, joined


# ---------------------------------------------------------------- selective state space scan

def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def scan(c, b, x, dt, A, dt_bias, D, use_softplus, scale, S0, dtype, chunked=True):
    """One sequence of one head token by token: c, b [T, N], x [T, P], dt [T], S0 [N, P].
    Returns y, its bound, the states after every token [T + 1, N, P] and their bound.

    The bound follows the recurrence.  Each token: a step size and an exponent off by some
    (6 + 2 |g|) U relative, which the decayed magnitudes carry on; a product of three factors.
    Within a 64-token chunk up to 3 x 64 partial sums of the state's products (three terms
    carry an fp32 weight on 16-bit operands) and exponents off by 4 U times the chunk's sum.
    Outputs of the 16-bit path: scores and state rounded once to bf16, then the output; sums
    over N and 64 tokens in fp32."""
    T, N = c.shape
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    d = softplus(raw) if use_softplus else raw
    d_err = 8 * U * (np.abs(d) + (np.abs(raw) * np.abs(d) if use_softplus else np.abs(raw)))
    g = d * A
    span = max([0.0] + [float(np.abs(g[i:i + 64]).sum()) for i in range(0, T, 1)]) if T else 0.0
    S, E, M = S0.copy(), np.zeros_like(S0), np.abs(S0)
    states, errs, ys, bounds = [S.copy()], [E.copy()], [], []
    half = HALF[dtype]
    for t in range(T):
        a = np.exp(g[t])
        term = d[t] * np.outer(b[t], x[t])
        ga = (6 + 2 * abs(g[t])) * U + abs(A) * d_err[t]
        E = a * E + ga * a * M + 10 * U * np.abs(term) + np.abs(np.outer(b[t], x[t])) * d_err[t]
        S, M = a * S + term, a * M + np.abs(term)
        chunk_err = (200 + 4 * span) * U * M if chunked else 2 * U * M
        states.append(S.copy())
        errs.append(E + chunk_err)
        mag = np.abs(c[t]) @ M * abs(scale)
        skip = 0.0 if D is None else D * x[t]
        ys.append(scale * (c[t] @ S) + skip)
        # |E| through c, sums of N and 64 terms in fp32, and for 16-bit inputs one rounding of
        # every score and of the state before the products
        narrow = half if dtype == "bf16" else 0.0
        bounds.append(abs(scale) * (np.abs(c[t]) @ (E + chunk_err)) + mag * (narrow * 1.01 + (N + 64 + 8 + 4 * span) * U)
                      + 4 * U * np.abs(skip) + half * np.abs(ys[-1]) + 1e-30)
    shape = (T, x.shape[1])
    return np.array(ys).reshape(shape), np.array(bounds).reshape(shape), np.array(states), np.array(errs)


# ---------------------------------------------------------------- norms

def _rms(v, eps):
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def gated_norm(x, z, w, eps, gate_first, act, dtype):
    """Roundings: dim / 2 for the mean under the root (a sum of squares, all positive), the gate's
    exp, addition and division, and six products."""
    gate = 1.0 if z is None else ACT[act](z)
    eg = 0.0 if z is None else 4 + 2 * np.abs(z)
    y = _rms(x * gate, eps) * w if gate_first else _rms(x, eps) * w * gate
    k = x.shape[-1] / 2 + 8 + eg + (0.0 if z is None or not gate_first else (eg.max(-1, keepdims=True)))
    return y, HALF[dtype] * np.abs(y) + 1.01 * k * U * np.abs(y) + 1e-30


def residual_norm(x, residual, post, gate, act, scale, pre, eps, dtype, res_dtype):
    """As gated_norm; the second norm is of the stored residual, whose own error e enters by
    element and through the root (its share of the row's norm)."""
    dim = x.shape[-1]
    v, k = x, np.zeros_like(x)
    if post is not None:
        v, k = _rms(v, eps) * post, k + dim / 2 + 6
    if gate is not None:
        v, k = v * ACT[act](gate), k + 6 + 2 * np.abs(gate)
    r = residual + scale * v
    e = (k + 2) * U * np.abs(scale * v) + 2 * U * np.abs(r) + HALF[res_dtype] * np.abs(r) * 1.01
    norm = np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    y = None if pre is None else r / norm * pre
    if pre is None:
        return r, e + 1e-30, None, None
    en = np.sqrt((e * e).mean(-1, keepdims=True))
    ey = np.abs(pre) * (e + np.abs(r) * en / norm) / norm + (dim / 2 + 8) * U * np.abs(y)
    return r, e + 1e-30, y, HALF[dtype] * np.abs(y) * 1.01 + 1.05 * ey + 1e-30
