"""The selective state space scan on the GPU against the fp64 recurrence, token by token:
packed prompts, initial states, exports, decode rows, and the invariances of the rule."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_amd import binding, layer
from tests import layer_reference as R

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
SHAPES = [("bf16", 2, 4, 128, 128), ("bf16", 1, 3, 64, 64), ("bf16", 2, 2, 128, 64), ("bf16", 1, 4, 64, 128), ("f32", 1, 1, 64, 64),
          ("f32", 2, 4, 128, 128), ("f32", 1, 2, 64, 128), ("f32", 1, 1, 128, 64)]


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def inputs(seed, tokens, Hk, Hv, dk, dv, dtype, slots, D=True, bias=True, rate=8.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)
    return dict(c=n(tokens, Hk, dk).to(TD[dtype]).cuda(), b=n(tokens, Hk, dk).to(TD[dtype]).cuda(), x=n(tokens, Hv, dv).to(TD[dtype]).cuda(),
                dt=n(tokens, Hv).cuda(), A=-(0.05 + rate * torch.rand(Hv, generator=g)).cuda(), bias=(n(Hv) - 3.0).cuda() if bias else None,
                D=n(Hv).cuda() if D else None, pool=n(slots, Hv, dk, dv).cuda(),
                y=torch.full((tokens, Hv, dv), float("nan"), dtype=TD[dtype], device="cuda"))


def prefill(d, lengths, init, final, scale=1.0, softplus=True, start=None, y=None, pool=None, rows=slice(None), stream=None, **kw):
    c, b, x, dt = d["c"][rows], d["b"][rows], d["x"][rows], d["dt"][rows]
    layer.gdn_ssm_chunk_prefill(c, b, x, dt, d["A"], d["y"] if y is None else y, i32(np.cumsum([0] + list(lengths))),
                                d["pool"] if pool is None else pool, i32(init), i32(final), dt_bias=d["bias"], D=d["D"], dt_softplus=softplus,
                                scale=scale, workspace=layer.alloc_ssm_workspace(c, x, len(lengths)), start_pos=None if start is None else i32(start),
                                stream=stream, **kw)


def within(name, got, ref, bound):
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all() and (err <= bound).all(), "%s: worst error / bound %.3g" % (name, np.max(err / bound))


def reference(d, before, i, h, lo, n, slot, scale, softplus, dtype, chunked=True):
    kh = h // (d["x"].shape[1] // d["c"].shape[1])
    S0 = before[slot, h] if 0 <= slot < len(before) else np.zeros(before.shape[2:])
    s = slice(lo, lo + n)
    return R.scan(f64(d["c"][s, kh]), f64(d["b"][s, kh]), f64(d["x"][s, h]), f64(d["dt"][s, h]), float(d["A"][h]),
                  None if d["bias"] is None else float(d["bias"][h]), None if d["D"] is None else float(d["D"][h]), softplus, scale, S0, dtype, chunked)


LENGTHS, STARTS = [130, 1, 0, 64, 200, 63, 65], [0, 5, 7, 64, 1000, 33, 63]


@pytest.mark.parametrize("dtype,Hk,Hv,dk,dv", SHAPES)
@pytest.mark.parametrize("variant", ["plain", "bare"])
def test_prefill(dtype, Hk, Hv, dk, dv, variant):
    n, tokens, grid = len(LENGTHS), sum(LENGTHS), 64
    bare = variant == "bare"                                      # no bias, no skip, dt taken as the step
    d = inputs(dk + dv + Hv, tokens, Hk, Hv, dk, dv, dtype, 3 * n, D=not bare, bias=not bare)
    if bare:
        d["dt"] = d["dt"].abs() * 0.05
    before = f64(d["pool"])
    init = [i if s else -1 for i, s in enumerate(STARTS)]
    final = [i if i % 2 else n + i for i in range(n)]             # odd sequences resume in place
    init[3], final[6] = 999, -1
    offs = binding.export_offsets(LENGTHS, STARTS, grid)
    exports = torch.full((offs[-1], Hv, dk, dv), float("nan"), device="cuda")
    scale = 0.5 if bare else 1.0
    prefill(d, LENGTHS, init, final, scale, not bare, STARTS, export_grid=grid, export_states=exports, export_offsets=i32(offs))
    lo = 0
    for i, length in enumerate(LENGTHS):
        for h in range(Hv):
            y, yb, S, Sb = reference(d, before, i, h, lo, length, init[i], scale, not bare, dtype)
            tag = "sequence %d head %d " % (i, h)
            if length:
                within(tag + "y", d["y"][lo:lo + length, h], y, yb)
            if 0 <= final[i] < 3 * n:
                within(tag + "state", d["pool"][final[i], h], S[-1], Sb[-1] + 1e-30)
            for m, p in enumerate(range((STARTS[i] // grid + 1) * grid, STARTS[i] + length + 1, grid)):
                within(tag + "export", exports[offs[i] + m, h], S[p - STARTS[i]], Sb[p - STARTS[i]] + 1e-30)
        lo += length
    untouched = [s for s in range(3 * n) if s not in final]
    assert np.array_equal(f64(d["pool"][untouched]), before[untouched])


@pytest.mark.parametrize("dtype,Hk,Hv,dk,dv", SHAPES)
def test_decode(dtype, Hk, Hv, dk, dv):
    rows = 6
    d = inputs(3, rows, Hk, Hv, dk, dv, dtype, 16)
    slot_in, slot_out = [3, -1, 5, 15, 16, 7], [3, 2, 6, -1, 4, 0]
    before = f64(d["pool"])
    layer.gdn_ssm_recurrent_decode(d["c"], d["b"], d["x"], d["dt"], d["A"], d["y"], d["pool"], i32(slot_in), i32(slot_out), dt_bias=d["bias"],
                                   D=d["D"], scale=0.7)
    for k in range(rows):
        if not 0 <= slot_in[k] < 16:
            assert (d["y"][k] == 0).all()
            continue
        for h in range(Hv):
            y, yb, S, Sb = reference(d, before, k, h, k, 1, slot_in[k], 0.7, True, dtype, chunked=False)
            within("row %d head %d y" % (k, h), d["y"][k:k + 1, h], y, yb)
            if 0 <= slot_out[k] < 16:
                within("row %d head %d state" % (k, h), d["pool"][slot_out[k], h], S[-1], Sb[-1])
    untouched = [s for s in range(16) if s not in (3, 6, 0)]
    assert np.array_equal(f64(d["pool"][untouched]), before[untouched])


@pytest.mark.parametrize("dtype,Hk,Hv,dk,dv", [("bf16", 2, 4, 128, 128), ("bf16", 1, 2, 64, 64), ("f32", 1, 2, 64, 64)])
def test_batch_mates_and_resumes_do_not_change_bits(dtype, Hk, Hv, dk, dv):
    """One long sequence alone, among few and among very many others, and resumed from each of its
    grid states: equal bits, whichever launch shape the call takes."""
    L, many = 700, 400
    d = inputs(11, L + 70 + many, Hk, Hv, dk, dv, dtype, many + 8)
    offs = L // 64
    alone, states = torch.empty_like(d["y"][:L]), torch.empty(offs, Hv, dk, dv, device="cuda")
    pool = d["pool"].clone()
    prefill(d, [L], [-1], [0], y=alone, pool=pool, rows=slice(0, L), export_grid=64, export_states=states, export_offsets=i32([0, offs]))
    for lengths in ([L, 70], [L, 70] + [1] * many):
        p, n, t = d["pool"].clone(), len(lengths), sum(lengths)
        y = torch.empty_like(d["y"][:t])
        e = torch.empty(offs + 1, Hv, dk, dv, device="cuda")
        prefill(d, lengths, [-1] * n, list(range(n)), y=y, pool=p, rows=slice(0, t), export_grid=64, export_states=e,
                export_offsets=i32([0, offs, offs + 1] + [offs + 1] * (n - 2)))
        assert torch.equal(y[:L], alone) and torch.equal(p[0], pool[0]) and torch.equal(e[:offs], states)
    for m in range(offs):
        t0 = 64 * (m + 1)
        p = d["pool"].clone()
        p[1] = states[m]
        y = torch.empty_like(d["y"][t0:L])
        prefill(d, [L - t0], [1], [2], start=[t0], y=y, pool=p, rows=slice(t0, L))
        assert torch.equal(y, alone[t0:]) and torch.equal(p[2], pool[0]), t0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_and_infinity_do_not_reach_earlier_tokens(dtype):
    """A poisoned token changes nothing before it, nor any other sequence."""
    d = inputs(4, 300, 1, 2, 64, 64, dtype, 4)
    args = ([200, 100], [-1, -1], [0, 1])
    clean = torch.empty_like(d["y"])
    prefill(d, *args, y=clean)
    state = d["pool"][1].clone()
    for name, t, value in (("x", 77, float("nan")), ("b", 130, float("inf")), ("c", 30, float("nan")), ("dt", 199, float("nan")),
                           ("x", 140, float("-inf"))):
        e = dict(d, **{name: d[name].clone()})
        e[name][t] = value
        y = torch.empty_like(clean)
        prefill(e, *args, y=y)
        assert torch.equal(y[:t], clean[:t]) and torch.equal(y[200:], clean[200:]) and torch.equal(d["pool"][1], state), (name, t)
        if name != "b":
            assert not torch.isfinite(y[t]).all(), (name, t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_decays(dtype):
    """No decay at all, and a decay that leaves nothing: S = d b x^T of the last token alone."""
    d = inputs(6, 150, 1, 2, 64, 64, dtype, 4, bias=False)
    d["dt"] = torch.full_like(d["dt"], 0.5)
    d["A"] = torch.tensor([0.0, -1000.0], device="cuda")
    before = f64(d["pool"])
    prefill(d, [150], [2], [3], softplus=False)
    for h in range(2):
        y, yb, S, Sb = reference(d, before, 0, h, 0, 150, 2, 1.0, False, dtype)
        within("y", d["y"][:, h], y, yb)
        within("state", d["pool"][3, h], S[-1], Sb[-1])


def test_long_sequence_few_chains():
    """One long prompt: the launch that spreads a sequence's chunks over the card."""
    T, Hk, Hv, dk, dv = 2100, 1, 2, 128, 128
    d = inputs(21, T, Hk, Hv, dk, dv, "bf16", 4)
    before = f64(d["pool"])
    prefill(d, [T], [1], [2], start=[64])
    for h in range(Hv):
        y, yb, S, Sb = reference(d, before, 0, h, 0, T, 1, 1.0, True, "bf16")
        within("y", d["y"][:, h], y, yb)
        within("state", d["pool"][2, h], S[-1], Sb[-1])


def test_exports_into_slots_and_far_slots():
    """Exports routed into pool slots, one of them dropped; a pool of more than 2^31 elements."""
    Hv, dk, dv = 2, 64, 64
    slots = (1 << 31) // (Hv * dk * dv) + 9
    d = inputs(8, 200, 1, Hv, dk, dv, "bf16", 4)
    pool = torch.empty(slots, Hv, dk, dv, device="cuda")
    pool[slots - 1] = d["pool"][0]
    prefill(d, [200], [slots - 1], [slots - 2], pool=pool, export_grid=64, export_offsets=i32([0, 3]), export_slots=i32([slots - 3, -1, 5]))
    want, y = torch.empty(3, Hv, dk, dv, device="cuda"), torch.empty_like(d["y"])
    prefill(d, [200], [0], [1], y=y, export_grid=64, export_states=want, export_offsets=i32([0, 3]))
    assert torch.equal(y, d["y"]) and torch.equal(pool[slots - 2], d["pool"][1])
    assert torch.equal(pool[slots - 3], want[0]) and torch.equal(pool[5], want[2])


def test_graph_and_side_stream():
    lengths = [150, 60, 90]
    d = inputs(12, 300, 2, 4, 128, 128, "bf16", 16)
    sin, sout = i32([3, 4, 5, -1]), i32([6, 7, 8, -1])
    ws = layer.alloc_ssm_workspace(d["c"], d["x"], 3)
    cu, init, fin = i32([0, 150, 210, 300]), i32([0, -1, 1]), i32([9, 10, 11])
    y1 = torch.empty_like(d["y"][:4])

    def step(s, y0, y, stream=None):
        layer.gdn_ssm_recurrent_decode(s["c"][:4], s["b"][:4], s["x"][:4], s["dt"][:4], s["A"], y0, s["pool"], sin, sout, dt_bias=s["bias"], D=s["D"],
                                       stream=stream)
        layer.gdn_ssm_chunk_prefill(s["c"], s["b"], s["x"], s["dt"], s["A"], y, cu, s["pool"], init, fin, dt_bias=s["bias"], D=s["D"],
                                    workspace=ws, stream=stream)

    step(d, y1, d["y"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(d, y1, d["y"])
    side = torch.cuda.Stream()
    for seed in range(3):
        e = inputs(30 + seed, 300, 2, 4, 128, 128, "bf16", 16)
        for k in ("c", "b", "x", "dt", "A", "bias", "D", "pool"):
            d[k].copy_(e[k])
        if seed == 1:                                             # another split of the same tokens
            cu.copy_(i32([0, 1, 1, 300]))
        ye = torch.empty_like(y1)
        side.wait_stream(torch.cuda.current_stream())
        step(e, ye, e["y"], stream=side)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d["y"], e["y"]) and torch.equal(y1, ye) and torch.equal(d["pool"], e["pool"])


def test_refusals():
    d = inputs(1, 8, 1, 2, 64, 64, "bf16", 4)
    s = i32([0])
    ok = dict(c=d["c"], b=d["b"], x=d["x"], dt=d["dt"], A=d["A"], y=d["y"], cu_seqlens=i32([0, 8]), state_pool=d["pool"], init_slot=s, final_slot=s,
              workspace=layer.alloc_ssm_workspace(d["c"], d["x"], 1))
    for change, err, text in [
            (dict(c=d["c"].float()), ValueError, "c must be"), (dict(b=d["b"][:4]), ValueError, "b must have shape"), (dict(dt=d["dt"].bfloat16()), ValueError, "dt"),
            (dict(A=d["A"][:1]), ValueError, "A must"), (dict(state_pool=d["pool"].bfloat16()), ValueError, "state_pool"),
            (dict(y=d["y"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError, "contiguous"), (dict(export_grid=96, export_offsets=i32([0, 0])), layer.GdnError, "export_grid 96"),
            (dict(scale=float("nan")), layer.GdnError, "scale")]:
        with pytest.raises(err, match=text):
            layer.gdn_ssm_chunk_prefill(**dict(ok, **change))
