"""Cases, inputs and plain forms of the operators around the gated delta rule.

Four operators of a recurrent layer's serving step, over packed sequences (cu_seqlens),
cache slots and the absolute 64-token chunk grid of the rule itself:

  plan   cache-slot maps, packed offsets and per-token maps of one step, from the
         requests' lengths and block tables
  conv   short causal convolution with SiLU and per-head L2 norm: packed prompts with
         cached tails, and single tokens
  scan   selective state space scan (scalar decay per head): packed prompts, and single
         tokens over cached fp32 states
  norm   the gated RMS norm behind the recurrence, and the residual norm between blocks

``run`` computes an operator in elementary torch operations, or, where ``own`` is true,
through ``gated_deltanet_rule_amd.layer``.  Both take the same state.
"""
import itertools
import math

import torch

own = False

CHUNK = 64
DEVICE = "cuda"


def _layer():
    from gated_deltanet_rule_amd import layer
    return layer


# ---------------------------------------------------------------- cases

# The standard head layout of the repository's workloads: 16 key heads, 32 value heads, 128 wide.
HEADS = dict(H_k=16, H_v=32, d_k=128, d_v=128)


def listed():
    return [
        # a decode-only step of 64 running requests: the smallest plan, all latency
        dict(name="plan_decode", op="plan", requests=64, decode=64, max_len=0, max_past=8192, block=1088, kv_block=16),
        # a large step: 448 running requests ahead of 64 prompts of up to 4096 tokens
        dict(name="plan_mixed", op="plan", requests=512, decode=448, max_len=4096, max_past=32768, block=1088, kv_block=16),
        # the convolution of the standard decode batch, read from a wider projection's rows
        dict(name="conv_decode", op="conv", kind="decode", rows=64, slots=256, width=4, dtype="bf16", l2=True, pad=4096, **HEADS),
        # eight prompts of 64 to 4096 tokens, tails kept every 64 tokens for the prefix cache
        dict(name="conv_varlen", op="conv", kind="prefill", seqs=8, min_len=64, max_len=4096, start=0, grid=64, width=4,
             dtype="bf16", l2=True, pad=4096, **HEADS),
        # one short fp32 sequence with one head: the smallest prompt
        dict(name="conv_single_f32", op="conv", kind="prefill", seqs=1, min_len=256, max_len=256, start=0, grid=0, width=4,
             dtype="f32", l2=True, pad=0, H_k=1, H_v=1, d_k=64, d_v=64),
        # the scan of the standard decode batch: 64 cached states of 2 MiB
        dict(name="scan_decode", op="scan", kind="decode", rows=64, slots=256, dtype="bf16", **HEADS),
        # one short fp32 sequence with one head
        dict(name="scan_single_f32", op="scan", kind="prefill", seqs=1, min_len=256, max_len=256, start=0, grid=0,
             dtype="f32", H_k=1, H_v=1, d_k=64, d_v=64),
        # one long prompt alone on the card: few chains, a long axis
        dict(name="scan_prompt", op="scan", kind="prefill", seqs=1, min_len=8192, max_len=8192, start=0, grid=1088,
             dtype="bf16", **HEADS),
        # the long prefill: 16 prompts of 8192 tokens, states kept on the 1088-token grid
        dict(name="scan_long", op="scan", kind="prefill", seqs=16, min_len=8192, max_len=8192, start=0, grid=1088,
             dtype="bf16", **HEADS),
        # the gated norm behind the rule in a decode step
        dict(name="norm_gated_decode", op="norm", kind="gated", rows=64, groups=32, dim=128, dtype="bf16", gate_first=False,
             per_group=False, pad=8192),
        # the gated norm behind the rule over a whole long prefill
        dict(name="norm_gated_long", op="norm", kind="gated", rows=131072, groups=32, dim=128, dtype="bf16", gate_first=False,
             per_group=False, pad=0),
        # the join of two blocks: norm after, gate, residual in fp32, norm before the next
        dict(name="norm_residual", op="norm", kind="residual", rows=16384, dim=4096, dtype="bf16", res_dtype="f32",
             post=True, gate=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_heads(rng):
    H_k = rng.choice([1, 2, 4, 8, 16])
    return dict(H_k=H_k, H_v=H_k * rng.choice([1, 2, 4] if H_k < 16 else [1, 2]), d_k=rng.choice([64, 128]), d_v=rng.choice([64, 128]))


def draw(rng):
    op = rng.choice(["plan", "conv", "scan", "scan", "norm", "norm"])
    if op == "plan":
        requests = _log_int(rng, 1, 512)
        decode = rng.choice([0, requests, rng.randint(0, requests)])
        return dict(op=op, requests=requests, decode=decode, max_len=_log_int(rng, 1, 131072 // max(1, requests - decode)),
                    max_past=_log_int(rng, 1, 32768), block=64 * _log_int(rng, 1, 17), kv_block=rng.choice([1, 16, 24, 64]))
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if rng.random() < 0.5:
            dim = rng.choice([64, 128, 128, 100, 4096, _log_int(rng, 1, 8192)])
            rows = _log_int(rng, 1, max(1, (1 << 24) // dim))
            groups = rng.choice([1, 1, 4]) if dim > 256 else rng.choice([1, 7, 32])
            return dict(op=op, kind="gated", rows=max(1, rows // groups), groups=groups, dim=dim, dtype=dtype,
                        gate_first=rng.random() < 0.5, per_group=rng.random() < 0.5, pad=rng.choice([0, 8 * groups, 3]))
        dim = rng.choice([1024, 2048, 4096, 5000, _log_int(rng, 1, 8192)])
        return dict(op=op, kind="residual", rows=_log_int(rng, 1, max(1, (1 << 25) // dim)), dim=dim, dtype=dtype,
                    res_dtype="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]), post=rng.random() < 0.5, gate=rng.random() < 0.5)
    heads = _draw_heads(rng)
    common = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), **heads)
    if op == "conv":
        common.update(width=rng.choice([2, 3, 4, 4]), l2=rng.random() < 0.7, pad=rng.choice([0, 8, 1024]))
    if rng.random() < 0.4:
        rows = _log_int(rng, 1, 128)
        return dict(common, kind="decode", rows=rows, slots=2 * rows + rng.randint(0, 64))
    seqs = _log_int(rng, 1, 16)
    max_len = _log_int(rng, 1, 4096)
    return dict(common, kind="prefill", seqs=seqs, min_len=rng.choice([0, 1, max_len]), max_len=max_len,
                start=rng.choice([0, 0, 64, 37]), grid=rng.choice([0, 64, 1088]))


# ---------------------------------------------------------------- inputs

def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _sequences(case, host):
    """Lengths, start positions and slots of a packed prefill: slots 0..n-1 hold the initial states, the next n take the final ones.
    A case's prompts are the same for every seed, their order and values are the seed's."""
    n = case["seqs"]
    lengths = torch.randint(case["min_len"], case["max_len"] + 1, (n,), generator=torch.Generator().manual_seed(n)).tolist()
    order = torch.randperm(n, generator=host).tolist()
    lengths, starts = [lengths[i] for i in order], [case["start"] * (i + 1) for i in order]
    grid = case["grid"]
    offsets = list(itertools.accumulate(((s + length) // grid - s // grid if grid else 0 for s, length in zip(starts, lengths)), initial=0))
    cu = list(itertools.accumulate(lengths, initial=0))
    return dict(lengths=lengths, starts=starts, offsets=offsets, cu=cu, cu_seqlens=_i32(cu), start_pos=_i32(starts),
                export_offsets=_i32(offsets), init_slot=_i32([i if s > 0 else -1 for i, s in enumerate(starts)]),
                final_slot=_i32([n + i for i in range(n)]))


def _prepare_plan(case, gen, host):
    n, b = case["requests"], case["decode"]
    past = torch.randint(0, case["max_past"] + 1, (n,), generator=host)
    past[:b] = past[:b].clamp(min=1)
    new = torch.randint(0, case["max_len"] + 1, (n,), generator=host)
    new[:b] = 1
    last = case["max_past"] + max(1, case["max_len"])
    width, kv_width = last // case["block"] + 1, last // case["kv_block"] + 1
    tokens = b + (n - b) * max(1, case["max_len"])      # what the step's buffers hold: the prompts need not fill it
    exports = (n - b) * (max(1, case["max_len"]) // case["block"] + 1)
    int32 = dict(dtype=torch.int32, device=DEVICE)
    return dict(computed=past.to(**int32), new_tokens=new.to(**int32), decode=b, block=case["block"], kv_block=case["kv_block"],
                state_table=torch.randperm(n * width, generator=gen, device=DEVICE).to(torch.int32).view(n, width),
                run_slot=torch.arange(n * width, n * width + n, **int32),
                kv_table=torch.randperm(n * kv_width, generator=gen, device=DEVICE).to(torch.int32).view(n, kv_width),
                out=dict(slot_in=torch.empty(b, **int32), slot_out=torch.empty(b, **int32), cu_seqlens=torch.empty(n - b + 1, **int32),
                         start_pos=torch.empty(n - b, **int32), init_slot=torch.empty(n - b, **int32),
                         final_slot=torch.empty(n - b, **int32), export_offsets=torch.empty(n - b + 1, **int32),
                         export_slots=torch.empty(exports, **int32), token_request=torch.empty(tokens, **int32),
                         token_position=torch.empty(tokens, **int32),
                         token_kv_slot=torch.empty(tokens, dtype=torch.int64, device=DEVICE)))


def _channels(case):
    return [case["H_k"] * case["d_k"], case["H_k"] * case["d_k"], case["H_v"] * case["d_v"]]


def _prepare_conv(case, gen, host):
    dtype, chan = _dt(case["dtype"]), _channels(case)
    c, w = sum(chan), case["width"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=DEVICE) * std

    seq = _sequences(case, host) if case["kind"] == "prefill" else None
    tokens = seq["cu"][-1] if seq else case["rows"]
    slots = 2 * case["seqs"] if seq else case["slots"]
    rows = torch.empty(tokens, c + case["pad"], dtype=dtype, device=DEVICE)
    rows.copy_(normal(tokens, c + case["pad"]))
    state = dict(x=rows[:, :c], weight=normal(c, w, std=w ** -0.5), bias=normal(c, std=0.1),
                 l2=(case["d_k"], case["d_k"], 0) if case["l2"] else (0, 0, 0), eps=1e-6, pool=normal(slots, w - 1, c).to(dtype),
                 outs=[torch.empty(tokens, n, dtype=dtype, device=DEVICE) for n in chan], seq=seq, grid=case.get("grid", 0))
    if seq:
        state["exports"] = torch.zeros(seq["offsets"][-1], w - 1, c, dtype=dtype, device=DEVICE)
    else:
        order = torch.randperm(slots, generator=host).to(torch.int32)[: 2 * tokens].to(DEVICE)
        state["slot_in"], state["slot_out"] = order[:tokens].contiguous(), order[tokens:].contiguous()
    return state


def _prepare_scan(case, gen, host):
    dtype, h, g = _dt(case["dtype"]), case["H_v"], case["H_k"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=DEVICE) * std

    seq = _sequences(case, host) if case["kind"] == "prefill" else None
    tokens = seq["cu"][-1] if seq else case["rows"]
    slots = 2 * case["seqs"] if seq else case["slots"]
    # the customary initial steps: log-uniform in [0.001, 0.1], kept as the bias whose softplus they are
    step = torch.exp(torch.rand(h, generator=gen, device=DEVICE) * math.log(100.0) + math.log(1e-3))
    state = dict(c=normal(tokens, g, case["d_k"]).to(dtype), b=normal(tokens, g, case["d_k"]).to(dtype),
                 x=normal(tokens, h, case["d_v"]).to(dtype), dt=normal(tokens, h), dt_bias=step + torch.log(-torch.expm1(-step)),
                 A=-(1.0 + 15.0 * torch.rand(h, generator=gen, device=DEVICE)), D=1.0 + normal(h, std=0.1),
                 scale=1.0, pool=normal(slots, h, case["d_k"], case["d_v"], std=0.1),
                 y=torch.empty(tokens, h, case["d_v"], dtype=dtype, device=DEVICE), seq=seq, grid=case.get("grid", 0))
    if seq:
        state["exports"] = torch.zeros(seq["offsets"][-1], h, case["d_k"], case["d_v"], device=DEVICE)
    else:
        order = torch.randperm(slots, generator=host).to(torch.int32)[: 2 * tokens].to(DEVICE)
        state["slot_in"], state["slot_out"] = order[:tokens].contiguous(), order[tokens:].contiguous()
    return state


def _prepare_norm(case, gen, host):
    dtype, rows, dim = _dt(case["dtype"]), case["rows"], case["dim"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=DEVICE) * std

    if case["kind"] == "gated":
        groups = case["groups"]
        wide = torch.empty(rows, groups * dim + case["pad"], dtype=dtype, device=DEVICE)     # the gate: columns of a wider projection
        wide.copy_(normal(rows, groups * dim + case["pad"]))
        return dict(x=normal(rows, groups, dim).to(dtype), z=wide[:, : groups * dim].unflatten(1, (groups, dim)),
                    weight=1.0 + (normal(groups, dim, std=0.1) if case["per_group"] else normal(dim, std=0.1)), eps=1e-6,
                    y=torch.empty(rows, groups, dim, dtype=dtype, device=DEVICE))
    res = _dt(case["res_dtype"])
    return dict(x=normal(rows, dim).to(dtype), residual=normal(rows, dim).to(res), scale=0.22, eps=1e-6,
                post=1.0 + normal(dim, std=0.1) if case["post"] else None, gate=normal(rows, dim).to(dtype) if case["gate"] else None,
                pre=1.0 + normal(dim, std=0.1), residual_out=torch.empty(rows, dim, dtype=res, device=DEVICE),
                y=torch.empty(rows, dim, dtype=dtype, device=DEVICE))


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    make = dict(plan=_prepare_plan, conv=_prepare_conv, scan=_prepare_scan, norm=_prepare_norm)[case["op"]]
    state = make(case, gen, host)
    state.update(op=case["op"], kind=case.get("kind", ""), gate_first=case.get("gate_first", False))
    return state


# ---------------------------------------------------------------- the framework's operators

def _run_own(s):
    layer = _layer()
    op, seq = s["op"], s.get("seq")
    if op == "plan":
        layer.gdn_step_plan(s["computed"], s["new_tokens"], s["state_table"], s["run_slot"], num_decode_rows=s["decode"],
                            state_block=s["block"], kv_table=s["kv_table"], kv_block=s["kv_block"], **s["out"])
        return s["out"]
    if op == "norm":
        if s["kind"] == "gated":
            layer.gdn_gated_norm(s["x"], s["z"], s["weight"], s["y"], eps=s["eps"], gate_first=s["gate_first"])
            return s["y"]
        layer.gdn_residual_norm(s["x"], s["residual"], s["residual_out"], s["y"], post_weight=s["post"], gate=s["gate"],
                                residual_scale=s["scale"], pre_weight=s["pre"], eps=s["eps"])
        return s["residual_out"], s["y"]
    exports = dict(start_pos=seq["start_pos"], export_grid=s["grid"], export_states=s["exports"],
                   export_offsets=seq["export_offsets"]) if seq else {}
    if op == "conv":
        if s["kind"] == "decode":
            layer.gdn_causal_conv_decode(s["x"], s["weight"], s["bias"], s["outs"], s["pool"], s["slot_in"], s["slot_out"],
                                         l2_dims=s["l2"], l2_eps=s["eps"])
            return s["outs"], s["pool"]
        layer.gdn_causal_conv_prefill(s["x"], s["weight"], s["bias"], s["outs"], s["pool"], seq["cu_seqlens"], seq["init_slot"],
                                      seq["final_slot"], l2_dims=s["l2"], l2_eps=s["eps"], **exports)
        return s["outs"], s["pool"], s["exports"]
    if s["kind"] == "decode":
        layer.gdn_ssm_recurrent_decode(s["c"], s["b"], s["x"], s["dt"], s["A"], s["y"], s["pool"], s["slot_in"], s["slot_out"],
                                       dt_bias=s["dt_bias"], D=s["D"], scale=s["scale"])
        return s["y"], s["pool"]
    if "workspace" not in s:
        s["workspace"] = layer.alloc_ssm_workspace(s["c"], s["x"], seq["cu_seqlens"].shape[0] - 1)
    layer.gdn_ssm_chunk_prefill(s["c"], s["b"], s["x"], s["dt"], s["A"], s["y"], seq["cu_seqlens"], s["pool"], seq["init_slot"],
                                seq["final_slot"], dt_bias=s["dt_bias"], D=s["D"], scale=s["scale"], workspace=s["workspace"], **exports)
    return s["y"], s["pool"], s["exports"]


# ---------------------------------------------------------------- plain forms

def _slot_at(s, request, position):
    """The cache slot of a request's state after `position` tokens: its block's on a block border, its running slot elsewhere."""
    block = s["block"]
    border = s["state_table"][request, (position // block - 1).clamp(min=0)].long()
    slot = torch.where(position % block == 0, border, s["run_slot"][request].long())
    return torch.where(position > 0, slot, torch.full_like(slot, -1))


def _run_plan(s):
    b, kv_block, out = s["decode"], s["kv_block"], s["out"]
    past, new = s["computed"].long(), s["new_tokens"].long()
    n, device = past.shape[0], past.device
    request = torch.arange(n, device=device)
    first, last = _slot_at(s, request, past), _slot_at(s, request, past + new)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=device), torch.cumsum(new[b:], 0)])
    count = (past[b:] + new[b:]) // s["block"] - past[b:] // s["block"]
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=device), torch.cumsum(count, 0)])
    # one entry for each export, then padding: its request, its grid point, and that block's slot unless the final state is that block's
    e = torch.arange(out["export_slots"].shape[0], device=device)
    owner = (torch.searchsorted(offsets, e, right=True) - 1 + b).clamp(max=n - 1)
    point = (past[owner] // s["block"] + 1 + e - offsets[(owner - b).clamp(min=0)]) * s["block"]
    slots = _slot_at(s, owner, point.clamp(max=s["state_table"].shape[1] * s["block"]))
    slots = torch.where((point == past[owner] + new[owner]) | (e >= offsets[-1]), torch.full_like(slots, -1), slots)
    # one entry for each token: decode rows, then the packed prompts, then padding
    t = torch.arange(out["token_request"].shape[0], device=device)
    owner = torch.where(t < b, t, torch.searchsorted(cu, t - b, right=True) - 1 + b)
    live = t - b < cu[-1]
    owner = owner.clamp(max=n - 1)
    position = past[owner] + torch.where(t < b, torch.zeros_like(t), t - b - cu[(owner - b).clamp(min=0)])
    position = torch.where(live, position, torch.zeros_like(t))
    kv = s["kv_table"][owner, position // kv_block].long() * kv_block + position % kv_block
    none = torch.full_like(t, -1)
    made = dict(slot_in=first[:b], slot_out=last[:b], cu_seqlens=cu, start_pos=past[b:], init_slot=first[b:], final_slot=last[b:],
                export_offsets=offsets, export_slots=slots, token_request=torch.where(live, owner, none),
                token_position=torch.where(live, position, none), token_kv_slot=torch.where(live, kv, none))
    return {k: v.to(out[k].dtype) for k, v in made.items()}


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _conv_outputs(s, taps):
    """Outputs from the taps [T, C, W] of every token, oldest first."""
    act = _silu((taps * s["weight"]).sum(-1) + s["bias"])
    parts = torch.split(act, [o.shape[1] for o in s["outs"]], dim=1)

    def normalised(p, dim):
        heads = p.unflatten(1, (-1, dim))
        return (heads / torch.sqrt((heads * heads).sum(-1, keepdim=True) + s["eps"])).flatten(1)

    return [(normalised(p, dim) if dim else p).to(o.dtype) for p, dim, o in zip(parts, s["l2"], s["outs"])]


def _run_conv(s):
    x, pool = s["x"], s["pool"]
    w = s["weight"].shape[1]
    if s["kind"] == "decode":
        window = torch.cat([pool[s["slot_in"].long()], x[:, None]], 1)           # [B, W, C]
        outs = _conv_outputs(s, window.float().transpose(1, 2))
        pool[s["slot_out"].long()] = window[:, 1:]
        return outs, pool
    seq, device = s["seq"], x.device
    cu, starts = seq["cu_seqlens"].long(), seq["start_pos"].long()
    n, tokens = starts.shape[0], x.shape[0]
    # every sequence's cached tail (zeros without one), then all tokens: rows of one table
    init = seq["init_slot"].long()
    tails = torch.where((init >= 0)[:, None, None], pool[init.clamp(min=0)], torch.zeros((), dtype=x.dtype, device=device))
    table = torch.cat([tails.reshape(n * (w - 1), -1), x])
    back = torch.arange(1 - w, 1, device=device)

    def rows(owner, local):
        """Table rows of the w inputs of owner's sequence that end at its local token."""
        rel = local[:, None] + back
        return torch.where(rel < 0, owner[:, None] * (w - 1) + w - 1 + rel, n * (w - 1) + cu[owner][:, None] + rel)

    t = torch.arange(tokens, device=device)
    owner = torch.searchsorted(cu, t, right=True) - 1
    outs = _conv_outputs(s, table[rows(owner, t - cu[owner])].float().transpose(1, 2))
    each = torch.arange(n, device=device)
    pool[seq["final_slot"].long()] = table[rows(each, cu[1:] - cu[:-1] - 1)[:, 1:]]
    exports = s["exports"]
    if s["grid"]:
        e = torch.arange(exports.shape[0], device=device)
        offsets = seq["export_offsets"].long()
        owner = torch.searchsorted(offsets, e, right=True) - 1
        point = (starts[owner] // s["grid"] + 1 + e - offsets[owner]) * s["grid"]
        exports.copy_(table[rows(owner, point - starts[owner] - 1)[:, 1:]])
    return outs, pool, exports


def _steps(s):
    """The positive step sizes softplus(dt + bias), in 64 bits: their sums are exponents."""
    v = s["dt"].double() + s["dt_bias"].double()
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _run_scan(s):
    pool, scale = s["pool"], s["scale"]
    x, b, c = s["x"].float(), s["b"].float(), s["c"].float()
    h, per = x.shape[1], x.shape[1] // b.shape[1]
    dt = _steps(s)
    if s["kind"] == "decode":
        b, c = b.repeat_interleave(per, 1), c.repeat_interleave(per, 1)
        old = pool[s["slot_in"].long()]
        decay = torch.exp(dt * s["A"].double()).float()
        state = decay[..., None, None] * old + (dt.float()[..., None] * b)[..., None] * x[:, :, None, :]
        y = scale * (c[..., None] * state).sum(2) + s["D"][:, None] * x
        pool[s["slot_out"].long()] = state
        return y.to(s["y"].dtype), pool
    seq, device = s["seq"], x.device
    cu, starts = seq["cu_seqlens"].long(), seq["start_pos"].long()
    n, q = starts.shape[0], CHUNK
    # sequences laid out on the absolute chunk grid: [n, chunks, 64, ...], zero steps where there is no token
    skew = starts % q
    chunks = max(1, max((st % q + length + q - 1) // q for st, length in zip(seq["starts"], seq["lengths"])))
    local = torch.arange(chunks * q, device=device) - skew[:, None]
    live = (local >= 0) & (local < (cu[1:] - cu[:-1])[:, None])
    at = (cu[:-1, None] + local).clamp(0, max(0, x.shape[0] - 1))
    keep = live.view(n, chunks, q)

    def laid(v):
        if v.shape[0] == 0:
            return v.new_zeros((n, chunks, q) + v.shape[1:])
        got = v[at].view((n, chunks, q) + v.shape[1:])
        return torch.where(keep.view((n, chunks, q) + (1,) * (v.dim() - 1)), got, torch.zeros((), dtype=v.dtype, device=device))

    dt = laid(dt).transpose(2, 3)                                            # [n, chunks, H, 64], 64 bits
    total = torch.cumsum(dt * s["A"].double()[:, None], -1)                  # G, inclusive
    xc = laid(x).transpose(2, 3).contiguous()                                # [n, chunks, H, 64, P]
    bc = laid(b).transpose(2, 3).contiguous()                                # [n, chunks, groups, 64, N]
    cc = laid(c).transpose(2, 3).contiguous()
    lower = torch.ones(q, q, dtype=torch.bool, device=device).tril()
    decay = torch.exp((total[..., :, None] - total[..., None, :]).masked_fill(~lower, -math.inf).float())
    scores = torch.matmul(cc, bc.transpose(-1, -2).contiguous()).repeat_interleave(per, 2)
    scores = scores * decay * dt.float()[..., None, :]
    y = torch.matmul(scores, xc)
    del scores, decay
    # what each chunk adds to the state, then the states at all chunk borders
    last = total[..., -1]                                                    # [n, chunks, H]
    weight = (torch.exp(last[..., None] - total) * dt).float()
    added = torch.matmul((bc.repeat_interleave(per, 2) * weight[..., None]).transpose(-1, -2).contiguous(), xc)
    init = seq["init_slot"].long()
    first = torch.where((init >= 0)[:, None, None, None], pool[init.clamp(min=0)], torch.zeros((), device=device))
    steps = torch.cat([first[:, None], added], 1).transpose(1, 2).flatten(3)          # [n, H, chunks + 1, N P]
    del added
    run = torch.cat([torch.zeros(n, 1, h, dtype=torch.float64, device=device), torch.cumsum(last, 1)], 1).transpose(1, 2)
    reach = torch.ones(chunks + 1, chunks + 1, dtype=torch.bool, device=device).tril()
    carry = torch.exp((run[..., :, None] - run[..., None, :]).masked_fill(~reach, -math.inf)).float()
    borders = torch.matmul(carry, steps).unflatten(3, first.shape[2:])                # [n, H, chunks + 1, N, P]
    del steps
    inter = torch.matmul(cc.repeat_interleave(per, 2), borders[:, :, :-1].transpose(1, 2).contiguous())
    y = scale * (y + torch.exp(total).float()[..., None] * inter) + s["D"][:, None, None] * xc
    y = y.transpose(2, 3).flatten(1, 2)[live].to(s["y"].dtype)
    pool[seq["final_slot"].long()] = borders[:, :, -1]
    exports = s["exports"]
    if s["grid"]:
        e = torch.arange(exports.shape[0], device=device)
        offsets = seq["export_offsets"].long()
        owner = torch.searchsorted(offsets, e, right=True) - 1
        point = (starts[owner] // s["grid"] + 1 + e - offsets[owner]) * s["grid"]
        exports.copy_(borders[owner, :, point // q - starts[owner] // q])
    return y, pool, exports


def _rms(v, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def _run_norm(s):
    x = s["x"].float()
    if s["kind"] == "gated":
        gate = _silu(s["z"].float())
        y = _rms(x * gate, s["eps"]) * s["weight"] if s["gate_first"] else _rms(x, s["eps"]) * s["weight"] * gate
        return y.to(s["y"].dtype)
    if s["post"] is not None:
        x = _rms(x, s["eps"]) * s["post"]
    if s["gate"] is not None:
        x = x * _silu(s["gate"].float())
    residual = (s["residual"].float() + s["scale"] * x).to(s["residual"].dtype)
    return residual, (_rms(residual.float(), s["eps"]) * s["pre"]).to(s["y"].dtype)


def run(state):
    if own:
        return _run_own(state)
    return dict(plan=_run_plan, conv=_run_conv, scan=_run_scan, norm=_run_norm)[state["op"]](state)


# ---------------------------------------------------------------- work

def _expected(case):
    """Tokens and exports of a packed prefill: those of the mean length, exact where all lengths are the same."""
    mean = (case["min_len"] + case["max_len"]) / 2
    tokens = case["seqs"] * mean
    exports = 0.0
    if case["grid"]:
        exports = sum((case["start"] * (i + 1) + mean) // case["grid"] - case["start"] * (i + 1) // case["grid"] for i in range(case["seqs"]))
    return tokens, exports


def work(case):
    size = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "plan":
        n, b = case["requests"], case["decode"]
        tokens = b + (n - b) * case["max_len"] / 2
        # lengths and slots of each request, one table entry for each block of either table, 16 bytes a token
        return dict(bytes=n * 40 + tokens * 16 + tokens / case["kv_block"] * 4 + tokens / case["block"] * 8, flops=0)
    if case["op"] == "norm":
        if case["kind"] == "gated":
            n = case["rows"] * case["groups"] * case["dim"]
            return dict(bytes=3 * n * size, flops=12 * n)
        n, res = case["rows"] * case["dim"], 2 if case["res_dtype"] == "bf16" else 4
        return dict(bytes=n * (2 * size + 2 * res + (size if case["gate"] else 0)), flops=16 * n)
    if case["op"] == "conv":
        c, w = sum(_channels(case)), case["width"]
        if case["kind"] == "decode":
            return dict(bytes=case["rows"] * c * size * (2 + 2 * (w - 1)) + c * (w + 1) * 4, flops=case["rows"] * c * (2 * w + 10))
        tokens, exports = _expected(case)
        states = case["seqs"] * (2 if case["start"] else 1) + exports
        return dict(bytes=(2 * tokens + states * (w - 1)) * c * size + c * (w + 1) * 4, flops=tokens * c * (2 * w + 10))
    h, g, n, p = case["H_v"], case["H_k"], case["d_k"], case["d_v"]
    per_token = (2 * g * n + 2 * h * p) * size + h * 4
    if case["kind"] == "decode":
        return dict(bytes=case["rows"] * (per_token + 8 * h * n * p), flops=case["rows"] * h * n * p * 5)
    tokens, exports = _expected(case)
    states = case["seqs"] * (2 if case["start"] else 1) + exports
    # the chunked form: scores shared by a group's heads, half of each square masked; then scores x, C S and B x for each head
    flops = tokens * (g * CHUNK * n + h * (CHUNK * p + 4 * n * p))
    return dict(bytes=tokens * per_token + states * h * n * p * 4, flops=flops)


# ---------------------------------------------------------------- values in 64 bits


def exact(case, seed):
    """What run() returns, from the definitions, in 64 bits."""
    if case["op"] == "plan":
        return None                                    # whole numbers: held to equality

    def conv(s):
        x, weight, bias = s["x"].double(), s["weight"].double(), s["bias"].double()
        w, pool = weight.shape[1], s["pool"].double()

        def act(joined):
            """Outputs for the rows of `joined` from row w - 1 on."""
            m = joined.shape[0] - (w - 1)
            a = bias.expand(m, -1).clone()
            for j in range(w):
                a += weight[:, j] * joined[j:j + m]
            return a * torch.sigmoid(a)

        def parts(u):
            done, at = [], 0
            for o, dim in zip(s["outs"], s["l2"]):
                p = u[:, at:at + o.shape[1]].clone()
                at += o.shape[1]
                for k in range(0, p.shape[1] if dim else 0, dim or 1):
                    p[:, k:k + dim] /= (p[:, k:k + dim].square().sum(1, keepdim=True) + s["eps"]).sqrt()
                done.append(p)
            return done

        if s["kind"] == "decode":
            after, rows = pool.clone(), []
            for i, (a, b) in enumerate(zip(s["slot_in"].tolist(), s["slot_out"].tolist())):
                joined = torch.cat([pool[a], x[i:i + 1]])
                rows.append(act(joined))
                after[b] = joined[1:]
            return parts(torch.cat(rows)), after
        seq, after, rows = s["seq"], pool.clone(), [x[:0]]
        exports = torch.zeros_like(s["exports"], dtype=torch.float64)
        for i, length in enumerate(seq["lengths"]):
            start, lo = seq["starts"][i], seq["cu"][i]
            joined = torch.cat([pool[i] if start > 0 else torch.zeros_like(pool[0]), x[lo:lo + length]])
            if length:
                rows.append(act(joined))
            after[len(seq["lengths"]) + i] = joined[length:]
            at = seq["offsets"][i]
            for p in range(start + 1, start + length + 1) if s["grid"] else ():
                if p % s["grid"] == 0:
                    exports[at] = joined[p - start:p - start + w - 1]
                    at += 1
        return parts(torch.cat(rows)), after, exports

    def scan(s):
        """Token by token: the recurrence as it is defined, all sequences in step."""
        pool = s["pool"].double()
        per = s["x"].shape[1] // s["b"].shape[1]
        A, D = s["A"].double(), s["D"].double()
        raw = s["dt"].double() + s["dt_bias"].double()
        dt = torch.logaddexp(raw, torch.zeros_like(raw))

        def step(state, rows):
            x = s["x"][rows].double()
            b = s["b"][rows].double().repeat_interleave(per, 1)
            c = s["c"][rows].double().repeat_interleave(per, 1)
            d = dt[rows]
            state = torch.exp(d * A)[..., None, None] * state + (d[..., None] * b)[..., None] * x[:, :, None]
            y = s["scale"] * torch.matmul(c[:, :, None], state)[:, :, 0] + D[:, None] * x
            return state, y

        if s["kind"] == "decode":
            state, y = step(pool[s["slot_in"].long()], torch.arange(s["x"].shape[0], device=pool.device))
            pool[s["slot_out"].long()] = state
            return y, pool
        seq = s["seq"]
        n = len(seq["lengths"])
        state = torch.zeros((n,) + tuple(pool.shape[1:]), dtype=torch.float64, device=pool.device)
        for i in range(n):
            if seq["starts"][i] > 0:
                state[i] = pool[i]
        y = torch.zeros(s["x"].shape, dtype=torch.float64, device=pool.device)
        exports = torch.zeros_like(s["exports"], dtype=torch.float64)
        order = sorted(range(n), key=lambda i: -seq["lengths"][i])
        state = state[torch.tensor(order, device=pool.device)]
        base = torch.tensor([seq["cu"][i] for i in order], device=pool.device)
        taken = [0] * n
        for t in range(max(seq["lengths"])):
            m = sum(length > t for length in seq["lengths"])                     # the m longest still run
            state[:m], y[base[:m] + t] = step(state[:m], base[:m] + t)
            for k in range(m if s["grid"] else 0):
                i = order[k]
                if (seq["starts"][i] + t + 1) % s["grid"] == 0:
                    exports[seq["offsets"][i] + taken[i]] = state[k]
                    taken[i] += 1
        for k, i in enumerate(order):
            pool[n + i] = state[k]
        return y, pool, exports

    def norm(s):
        def unit(v):
            return v * torch.rsqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + s["eps"])

        x = s["x"].double()
        if s["kind"] == "gated":
            z, w = s["z"].double(), s["weight"].double()
            z = z * torch.sigmoid(z)
            return unit(x * z) * w if s["gate_first"] else unit(x) * z * w
        if s["post"] is not None:
            x = unit(x) * s["post"].double()
        if s["gate"] is not None:
            g = s["gate"].double()
            x = g * torch.sigmoid(g) * x
        residual = s["residual"].double() + s["scale"] * x
        return residual, unit(residual) * s["pre"].double()

    return dict(conv=conv, scan=scan, norm=norm)[case["op"]](prepare(case, seed))
