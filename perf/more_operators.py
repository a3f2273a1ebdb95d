"""Cases, inputs and plain forms of the attention layers' operators.

Three operators of the full-attention layers between the recurrent ones, over the token maps of
the step plan (positions, rows of a paged key/value cache):

  rotary     rotary positions of q and k: half or interleaved pairs, the whole head or its first
             part, angles of positions past a million
  cache      keys and values written into a paged cache, quantised to 8 bits for each head of a
             token (or kept as they are), and a prefix read back
  attention  decode rows of one or more tokens (a chain or a tree of drafted tokens) over their
             cached contexts, and packed prompts, fresh or behind a cached past

``run`` computes an operator in elementary torch operations, or, where ``own`` is true,
through ``gated_deltanet_rule_amd.attention``.  Both take the same state.
"""
import itertools
import math

import torch

own = False

DEVICE = "cuda"
E4M3 = torch.float8_e4m3fn
TOP = {"e4m3": 448.0, "int8": 127.0}      # the largest code of each 8-bit format


def _attention():
    from gated_deltanet_rule_amd import attention
    return attention


# ---------------------------------------------------------------- cases

# Heads of the attention layers: 32 query heads over 8 key/value heads of the standard width, and
# the wide layout, 16 over 2 heads of 256.
HEADS = dict(H_q=32, H_kv=8, d=128)
WIDE = dict(H_q=16, H_kv=2, d=256)


def listed():
    return [
        # the rotation of a decode step of 64 running requests: all latency
        dict(name="rotary_decode", op="rotary", tokens=64, max_pos=8192, rotary=128, interleaved=False, factor=1.0, pad=0,
             dtype="bf16", **HEADS),
        # the rotation of a whole long prefill, 16 prompts of 8192 tokens, read from a projection's rows
        dict(name="rotary_long", op="rotary", tokens=131072, max_pos=0, rotary=128, interleaved=False, factor=1.0, pad=1024,
             dtype="bf16", **HEADS),
        # a quarter of each wide head in interleaved pairs, positions stretched for a context of a million tokens, in fp32
        dict(name="rotary_part_f32", op="rotary", tokens=4099, max_pos=1000000, rotary=64, interleaved=True, factor=32.0, pad=512,
             dtype="f32", **WIDE),
        # a decode step's keys and values into an 8-bit cache: 64 tokens
        dict(name="cache_decode", op="cache", tokens=64, past=0, format="e4m3", dtype="bf16", pad=0, **HEADS),
        # a prompt chunk of 8192 tokens into the cache, and its request's prefix of 32768 read back
        dict(name="cache_prefix", op="cache", tokens=8192, past=24576, format="int8", dtype="bf16", pad=4096, **HEADS),
        # a whole long prefill written and read back: 16 prompts of 8192 tokens
        dict(name="cache_long", op="cache", tokens=131072, past=0, format="e4m3", dtype="bf16", pad=4096, **HEADS),
        # the standard decode batch: 64 requests with contexts up to 8192 tokens
        dict(name="attention_decode", op="attention", kind="decode", rows=64, tokens=1, min_ctx=1024, max_ctx=8192, tree=False,
             kv_block=16, format="plain", dtype="bf16", **HEADS),
        # one request alone with a long context in 8 bits: few rows, a long axis
        dict(name="attention_decode_long", op="attention", kind="decode", rows=1, tokens=1, min_ctx=131072, max_ctx=131072,
             tree=False, kv_block=64, format="e4m3", dtype="bf16", **HEADS),
        # trees of 32 drafted tokens of 16 requests, 8-bit integers in the cache
        dict(name="attention_tree", op="attention", kind="decode", rows=16, tokens=32, min_ctx=1024, max_ctx=8192, tree=True,
             kv_block=16, format="int8", dtype="bf16", **HEADS),
        # one short fp32 sequence with one head: the smallest prompt
        dict(name="attention_single_f32", op="attention", kind="prefill", seqs=1, min_len=256, max_len=256, past=0, kv_block=16,
             format="plain", dtype="f32", H_q=1, H_kv=1, d=64),
        # eight fresh prompts of 64 to 4096 tokens
        dict(name="attention_varlen", op="attention", kind="prefill", seqs=8, min_len=64, max_len=4096, past=0, kv_block=16,
             format="plain", dtype="bf16", **HEADS),
        # the last 8192 tokens of a prompt of 32768, wide heads over an 8-bit cache
        dict(name="attention_resume", op="attention", kind="prefill", seqs=1, min_len=8192, max_len=8192, past=24576, kv_block=64,
             format="e4m3", dtype="bf16", **WIDE),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["rotary", "cache", "attention", "attention", "attention"])
    d = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    heads = dict(H_q=kv * rng.choice([1, 2, 3, 4, 7, 8]), H_kv=kv, d=d)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "rotary":
        heads["d"] = d = rng.choice([64, 80, 96, 128, 128, 256])
        rotary = rng.choice([d, d, d // 2, d // 4 // 2 * 2])
        return dict(op=op, tokens=_log_int(rng, 1, (1 << 28) // ((heads["H_q"] + kv) * d)), max_pos=rng.choice([0, 8192, _log_int(rng, 2, 2000000)]),
                    rotary=rotary, interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 32.0]), pad=rng.choice([0, 8, 1024]),
                    dtype=dtype, **heads)
    fmt = rng.choice(["plain", "e4m3", "e4m3", "int8"])
    if op == "cache":
        most = (1 << 27) // (kv * d)
        return dict(op=op, tokens=_log_int(rng, 1, most), past=rng.choice([0, _log_int(rng, 1, most)]), format=fmt, dtype=dtype,
                    pad=rng.choice([0, 8, 1024]), **heads)
    common = dict(op=op, kv_block=rng.choice([1, 16, 16, 24, 64, 256]), format=fmt, dtype=dtype, **heads)
    if rng.random() < 0.55:
        tokens = rng.choice([1, 1, 1, _log_int(rng, 2, 64)])
        rows = _log_int(rng, 1, 64)
        ctx = _log_int(rng, 1, min(131072, (1 << 29) // (rows * kv * d)))
        return dict(common, kind="decode", rows=rows, tokens=tokens, min_ctx=rng.choice([0, ctx // 2, ctx]), max_ctx=ctx,
                    tree=tokens > 1 and rng.random() < 0.7)
    seqs = _log_int(rng, 1, 16)
    length = _log_int(rng, 1, 4096)
    most = (1 << 31) // (seqs * heads["H_q"] * length)           # keys, so that the plain form's scores fit
    past = rng.choice([0, 0, _log_int(rng, 1, 32768)])
    length = min(length, max(1, most // 2))
    return dict(common, kind="prefill", seqs=seqs, min_len=rng.choice([0, 1, length]), max_len=length, past=max(0, min(past, most - length)))


# ---------------------------------------------------------------- inputs

def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _between(lo, hi, n):
    """n whole numbers from lo to hi, the same for every seed; the largest is among them."""
    got = torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(n + hi)).tolist()
    return got[:-1] + [hi]


def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEVICE).to(dtype)


def _columns(gen, tokens, runs, pad, d, dtype):
    """Runs of heads as columns of one projection's rows, `pad` more columns behind them."""
    wide = _normal(gen, tokens, sum(runs) * d + pad, dtype=dtype)
    parts, at = [], 0
    for n in runs:
        parts.append(wide[:, at: at + n * d].unflatten(1, (n, d)))
        at += n * d
    return parts


def _prepare_rotary(case, gen, host):
    tokens, dtype, d, r = case["tokens"], _dt(case["dtype"]), case["d"], case["rotary"]
    q, k = _columns(gen, tokens, (case["H_q"], case["H_kv"]), case["pad"], d, dtype)
    if case["max_pos"]:          # running requests, each at its own position
        positions = torch.randint(0, case["max_pos"], (tokens,), generator=host).to(DEVICE, torch.int32)
    else:                        # prompts of 8192 tokens, one behind the other
        positions = (torch.arange(tokens, device=DEVICE) % 8192).to(torch.int32)
    freq = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r) / case["factor"]
    return dict(q=q, k=k, positions=positions, inv_freq=freq.to(DEVICE, torch.float32), interleaved=case["interleaved"],
                attention_factor=0.1 * math.log(case["factor"]) + 1.0,
                q_out=torch.empty(tokens, case["H_q"], d, dtype=dtype, device=DEVICE),
                k_out=torch.empty(tokens, case["H_kv"], d, dtype=dtype, device=DEVICE))


def _empty_cache(rows, case):
    """K and V rows of a cache and their scales (None where the format has none)."""
    dtype = {"plain": _dt(case["dtype"]), "e4m3": E4M3, "int8": torch.int8}[case["format"]]
    made = {n: torch.zeros(rows, case["H_kv"], case["d"], dtype=dtype, device=DEVICE) for n in ("k_cache", "v_cache")}
    for n in ("k_scale", "v_scale"):
        made[n] = None if case["format"] == "plain" else torch.zeros(rows, case["H_kv"], device=DEVICE)
    return made


def _prepare_cache(case, gen, host):
    tokens, past, d, dtype = case["tokens"], case["past"], case["d"], _dt(case["dtype"])
    rows = tokens + past + 100
    state = _empty_cache(rows, case)
    place = torch.randperm(rows, generator=gen, device=DEVICE)
    old, new = place[:past], place[past: past + tokens].contiguous()
    for name in ("k", "v"):
        _plain_write(state, name, _normal(gen, past, case["H_kv"], d, dtype=dtype), old)
    k, v = _columns(gen, tokens, (case["H_kv"], case["H_kv"]), case["pad"], d, dtype)
    out = [torch.empty(past + tokens, case["H_kv"], d, dtype=dtype, device=DEVICE) for _ in range(2)]
    return dict(state, k=k, v=v, slots=new, prefix=place[: past + tokens].contiguous(), k_out=out[0], v_out=out[1])


def _pages(lengths, kv_block, gen):
    """A block table [n, width] of shuffled pages for requests of these lengths, and the cache's rows."""
    counts = [-(-length // kv_block) for length in lengths]
    pages = torch.randperm(sum(counts) + 4, generator=gen, device=DEVICE).to(torch.int32)
    width = max(1, max(counts))
    first = torch.tensor(list(itertools.accumulate(counts, initial=0))[:-1], device=DEVICE)
    column = torch.arange(width, device=DEVICE)
    live = column < torch.tensor(counts, device=DEVICE)[:, None]
    at = (first[:, None] + column).clamp(max=pages.shape[0] - 1)
    return torch.where(live, pages[at], torch.full_like(pages[at], -1)).contiguous(), pages.shape[0] * kv_block


def _trees(rows, tokens, host):
    """Random trees: the parent of each drafted token is an earlier one or the context; a bit for each ancestor and for itself."""
    parents = (torch.rand(rows, tokens, generator=host) * (torch.arange(tokens) + 1)).long().tolist()     # 0: the context, i + 1: token i
    masks = []
    for row in parents:
        seen = []
        for i, p in enumerate(row):
            m = (1 << i) | (seen[p - 1] if p else 0)
            seen.append(m)
        masks += [m - (1 << 64) if m >> 63 else m for m in seen]
    return torch.tensor(masks, dtype=torch.int64, device=DEVICE)


def _lengths(case):
    """(cached tokens, new tokens) of each request of an attention case."""
    if case["kind"] == "decode":
        past = _between(case["min_ctx"], case["max_ctx"], case["rows"])
        return past, [case["tokens"]] * len(past)
    new = _between(case["min_len"], case["max_len"], case["seqs"])
    return [case["past"]] * len(new), new


def _prepare_attention(case, gen, host):
    dtype, d, past, new = _dt(case["dtype"]), case["d"], *_lengths(case)
    order = torch.randperm(len(past), generator=host).tolist()
    past, new = [past[i] for i in order], [new[i] for i in order]
    keys = [p + n for p, n in zip(past, new)]
    table, rows = _pages(keys, case["kv_block"], gen)
    state = _empty_cache(rows, case)
    everywhere = torch.arange(rows, device=DEVICE)
    for name in ("k", "v"):
        _plain_write(state, name, _normal(gen, rows, case["H_kv"], d, dtype=dtype), everywhere)
    tokens, cu = sum(new), list(itertools.accumulate(new, initial=0))
    state.update(q=_normal(gen, tokens, case["H_q"], d, dtype=dtype), o=torch.empty(tokens, case["H_q"], d, dtype=dtype, device=DEVICE),
                 computed=_i32(past), cu_seqlens=_i32(cu), table=table, kv_block=case["kv_block"], scale=d ** -0.5, max_keys=max(keys),
                 max_new=max(new), past=past, new=new, cu=cu, tokens=case.get("tokens", 0))
    state["mask"] = _trees(case["rows"], case["tokens"], host) if case.get("tree") else None
    return state


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    state = dict(rotary=_prepare_rotary, cache=_prepare_cache, attention=_prepare_attention)[case["op"]](case, gen, host)
    state.update(op=case["op"], kind=case.get("kind", ""), format=case.get("format", ""))
    return state


# ---------------------------------------------------------------- the framework's operators

def _run_own(s):
    attention = _attention()
    if s["op"] == "rotary":
        attention.gdn_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], q_out=s["q_out"], k_out=s["k_out"],
                             interleaved=s["interleaved"], attention_factor=s["attention_factor"])
        return s["q_out"], s["k_out"]
    cache = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "cache":
        attention.gdn_kv_cache_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], **cache)
        attention.gdn_kv_cache_read(s["prefix"], s["k_cache"], s["v_cache"], s["k_out"], s["v_out"], **cache)
        return s["k_out"], s["v_out"]
    if s["kind"] == "prefill":
        attention.gdn_attention_prefill(s["q"], s["k_cache"], s["v_cache"], s["o"], s["cu_seqlens"], s["computed"], s["table"],
                                        kv_block=s["kv_block"], scale=s["scale"], **cache)
        return s["o"]
    if "workspace" not in s:
        s["workspace"] = attention.alloc_attention_workspace(s["q"], s["k_cache"], tokens_per_row=s["tokens"], max_keys=s["max_keys"])
    attention.gdn_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["o"], s["computed"], s["table"], kv_block=s["kv_block"],
                                   tokens_per_row=s["tokens"], tree_mask=s["mask"], scale=s["scale"], max_keys=s["max_keys"],
                                   workspace=s["workspace"], **cache)
    return s["o"]


# ---------------------------------------------------------------- plain forms

def _run_rotary(s):
    """Angles in 64 bits: a far position times a frequency is many turns."""
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos = (torch.cos(angle) * s["attention_factor"]).float()[:, None]
    sin = (torch.sin(angle) * s["attention_factor"]).float()[:, None]
    half = cos.shape[-1]
    outs = []
    for x in (s["q"], s["k"]):
        v = x.float()
        if s["interleaved"]:
            a, b = v[..., 0: 2 * half: 2], v[..., 1: 2 * half: 2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = v[..., :half], v[..., half: 2 * half]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        outs.append(torch.cat([turned, v[..., 2 * half:]], -1).to(x.dtype))
    return tuple(outs)


def _plain_write(s, name, x, slots):
    """x [T, H, d] into rows `slots` of cache `name`: a scale for each head of a token, codes rounded to nearest even."""
    cache, scales = s[name + "_cache"], s[name + "_scale"]
    if scales is None:
        cache[slots] = x
        return
    x = x.float()
    top = 448.0 if cache.dtype == E4M3 else 127.0
    largest = x.abs().amax(-1).clamp(min=2.0 ** -100)
    scale = largest / torch.full_like(largest, top)           # a division: by a plain number it would be a product with the inverse
    v = (x / scale[..., None]).clamp(-top, top)
    codes = v.to(E4M3).view(torch.uint8) if cache.dtype == E4M3 else torch.round(v).to(torch.int8).view(torch.uint8)
    cache.view(torch.uint8)[slots] = codes
    scales[slots] = scale


def _plain_read(s, name, rows):
    """The values at these rows of cache `name`, in 32 bits."""
    cache, scales = s[name + "_cache"], s[name + "_scale"]
    if scales is None:
        return cache[rows].float()
    return cache.view(torch.uint8)[rows].view(cache.dtype).float() * scales[rows][..., None]


def _run_cache(s):
    _plain_write(s, "k", s["k"], s["slots"])
    _plain_write(s, "v", s["v"], s["slots"])
    return _plain_read(s, "k", s["prefix"]).to(s["k"].dtype), _plain_read(s, "v", s["prefix"]).to(s["v"].dtype)


def _run_attention(s):
    q, block = s["q"], s["kv_block"]
    past = s["computed"].long()
    n, keys, h, d = past.shape[0], s["max_keys"], s["k_cache"].shape[1], q.shape[2]
    group = q.shape[1] // h
    key = torch.arange(keys, device=q.device)
    rows = (s["table"].long()[:, key // block] * block + key % block).clamp(min=0)                # [n, keys]
    # queries laid out by request, [n, heads, tokens x group, d], and the keys that each token sees, [n, tokens, keys]
    cu = s["cu_seqlens"].long()
    local = torch.arange(s["max_new"], device=q.device)
    at = (cu[:-1, None] + local).clamp(max=max(0, q.shape[0] - 1))
    if q.shape[0] == 0:
        return torch.zeros_like(q)
    laid = q[at].float().view(n, -1, h, group, d).transpose(1, 2).reshape(n, h, -1, d)
    if s["mask"] is None:
        seen = key <= (past[:, None] + local)[..., None]
    else:
        j = key - past[:, None]                                                                   # [n, keys]
        bits = s["mask"].view(n, -1, 1) >> j.clamp(0, 63)[:, None]
        seen = (j < 0)[:, None] | ((bits & 1).bool() & ((j >= 0) & (j < s["max_new"]))[:, None])
    k = _plain_read(s, "k", rows).permute(0, 2, 3, 1).contiguous()                                # [n, h, d, keys]
    scores = torch.matmul(laid, k).view(n, h, -1, group, keys)
    del k
    scores *= s["scale"]
    scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True).clamp(min=-3e38)
    weights = scores.exp_().view(n, h, -1, keys)
    total = weights.sum(-1, keepdim=True)
    v = _plain_read(s, "v", rows).transpose(1, 2).contiguous()
    o = torch.matmul(weights, v) / total.clamp(min=1e-30)                                         # a token that sees nothing: zeros
    o = o.view(n, h, -1, group, d).transpose(1, 2).reshape(n, -1, h * group, d)
    t = torch.arange(q.shape[0], device=q.device)
    owner = torch.searchsorted(cu, t, right=True) - 1
    return o[owner, t - cu[owner]].to(q.dtype)


def run(state):
    if own:
        return _run_own(state)
    return dict(rotary=_run_rotary, cache=_run_cache, attention=_run_attention)[state["op"]](state)


# ---------------------------------------------------------------- work

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    h, hkv, d = case["H_q"], case["H_kv"], case["d"]
    if case["op"] == "rotary":
        n = case["tokens"] * (h + hkv) * d
        return dict(bytes=2 * n * size + case["tokens"] * 4, flops=3 * n * case["rotary"] // d)
    stored = hkv * (d * size if case["format"] == "plain" else d + 4)          # a cache row of K or V, its scales with it
    if case["op"] == "cache":
        t, read = case["tokens"], case["tokens"] + case["past"]
        return dict(bytes=(t + read) * (2 * hkv * d * size + 2 * stored + 8), flops=(3 * t + read) * 2 * hkv * d)
    past, new = _lengths(case)
    keys, tokens = sum(p + n for p, n in zip(past, new) if n), sum(new)
    if case.get("tree"):        # the context and, of a random tree, itself and about log n ancestors
        pairs = sum(n * (p + 1 + math.log(n)) for p, n in zip(past, new))
    else:
        pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(past, new))
    return dict(bytes=2 * keys * stored + 2 * tokens * h * d * size, flops=4 * d * h * pairs)


# ---------------------------------------------------------------- values in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions, in 64 bits."""

    def rotary(s):
        r = case["rotary"]
        both = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            for i in range(r // 2):
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
                turn = torch.polar(torch.full((x.shape[0],), s["attention_factor"], dtype=torch.float64, device=x.device),
                                   s["positions"].double() * s["inv_freq"][i].double())[:, None]
                z = torch.complex(x[..., a].double(), x[..., b].double()) * turn
                y[..., a], y[..., b] = z.real, z.imag
            both.append(y)
        return tuple(both)

    def stored(x, fmt):
        """The values that a row's codes stand for.  Scale and quotient are fp32 numbers by definition."""
        x = x.double()
        if fmt == "plain":
            return x
        largest = x.abs().max(-1, keepdim=True).values
        scale = (torch.where(largest < 2.0 ** -100, torch.full_like(largest, 2.0 ** -100), largest) / TOP[fmt]).float().double()
        v = (x / scale).float().double()
        if fmt == "int8":
            return v.round().clamp(-127, 127) * scale
        # the step of each value's binade, 2^-9 below the smallest normal number 2^-6; from a list, so that powers are exact
        powers = torch.tensor([2.0 ** i for i in range(-9, 8)], dtype=torch.float64, device=v.device)
        step = powers[torch.frexp(v).exponent.clamp(-5, 11).long() + 5]
        return ((v / step).round() * step).clamp(-448, 448) * scale

    def cache(s):
        both = []
        for name in ("k", "v"):
            old = s[name + "_cache"]
            table = old.to(torch.float64)
            if s[name + "_scale"] is not None:
                table = table * s[name + "_scale"].double()[..., None]
            table[s["slots"]] = stored(s[name], case["format"])
            both.append(table[s["prefix"]])
        return tuple(both)

    def values(s, name, at, g):
        """Head g of rows `at` of a cache."""
        table, scale = s[name + "_cache"], s[name + "_scale"]
        if scale is None:
            return table[at, g].double()
        return table.view(torch.uint8)[at, g].view(table.dtype).to(torch.float64) * scale[at, g, None].double()

    def attention(s):
        q = s["q"].double()
        o = torch.zeros_like(q)
        hkv = case["H_kv"]
        group = case["H_q"] // hkv
        for i, (past, new) in enumerate(zip(s["past"], s["new"])):
            position = torch.arange(past + new, device=q.device)
            at = s["table"][i][position // s["kv_block"]].long() * s["kv_block"] + position % s["kv_block"]
            lo = s["cu"][i]
            for g in range(hkv if new else 0):
                k, v = values(s, "k", at, g), values(s, "v", at, g)
                kt = k.t().contiguous()
                for first in range(0, new, 1024):
                    n = min(1024, new - first)
                    own_rows = slice(lo + first, lo + first + n)
                    rows = q[own_rows, g * group: (g + 1) * group].reshape(n * group, -1)
                    allowed = torch.ones(n, past + new, dtype=torch.bool, device=q.device)
                    if s["mask"] is None:
                        allowed[:, past:] = torch.ones(new, new, dtype=torch.bool, device=q.device).tril()[first: first + n]
                    else:
                        drafted = torch.arange(new, device=q.device)
                        allowed[:, past:] = (s["mask"][own_rows, None] >> drafted) % 2 == 1
                    score = (rows @ kt).mul_(s["scale"]).view(n, group, -1)
                    score.masked_fill_(~allowed[:, None], -math.inf)
                    p = torch.softmax(score, -1).nan_to_num(0.0).flatten(0, 1)
                    o[own_rows, g * group: (g + 1) * group] = (p @ v).view(n, group, -1)
        return o

    return dict(rotary=rotary, cache=cache, attention=attention)[case["op"]](prepare(case, seed))
