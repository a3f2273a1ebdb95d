"""The scan's launch for calls with few chains (W and the decays in a launch of their own,
then strips of columns): sequences long enough on average to take it, with odd starts, single
tokens and empty ones among them, against the fp64 recurrence and against the other launch."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_amd import binding, layer
from tests.test_gpu_layer_ssm import TD, f64, i32, inputs, prefill, reference, within

pytestmark = pytest.mark.gpu
SHAPES = [("bf16", 1, 2, 128, 128), ("bf16", 1, 6, 64, 64), ("bf16", 2, 2, 128, 64), ("bf16", 1, 1, 64, 128),
          ("f32", 1, 2, 128, 128), ("f32", 1, 6, 64, 64), ("f32", 1, 1, 64, 128), ("f32", 2, 2, 128, 64)]
LENGTHS, STARTS = [470, 1, 0, 333, 64, 129], [0, 5, 7, 1000, 33, 63]


def workspace_bytes(d, seqs, tokens):
    ws = layer.alloc_ssm_workspace(d["c"][:tokens], d["x"][:tokens], seqs)
    return 0 if ws is None else ws.numel()


@pytest.mark.parametrize("dtype,Hk,Hv,dk,dv", SHAPES)
def test_strips(dtype, Hk, Hv, dk, dv):
    n, tokens, grid = len(LENGTHS), sum(LENGTHS), 128
    d = inputs(dk + 3 * dv + Hv, tokens, Hk, Hv, dk, dv, dtype, 3 * n)
    assert workspace_bytes(d, n, tokens) > 0                       # the call takes the strips
    before = f64(d["pool"])
    init = [i if s else -1 for i, s in enumerate(STARTS)]
    final = [i if i % 2 else n + i for i in range(n)]             # odd sequences resume in place
    init[4], final[5] = 999, -1
    offs = binding.export_offsets(LENGTHS, STARTS, grid)
    exports = torch.full((offs[-1], Hv, dk, dv), float("nan"), device="cuda")
    prefill(d, LENGTHS, init, final, 0.7, True, STARTS, export_grid=grid, export_states=exports, export_offsets=i32(offs))
    lo = 0
    for i, length in enumerate(LENGTHS):
        for h in range(Hv):
            y, yb, S, Sb = reference(d, before, i, h, lo, length, init[i], 0.7, True, dtype)
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
def test_both_launches_give_the_same_bits(dtype, Hk, Hv, dk, dv):
    """The same sequences alone and among single tokens enough to take the whole-heads launch."""
    n, tokens, many = len(LENGTHS), sum(LENGTHS), 600
    d = inputs(17 + dk, tokens + many, Hk, Hv, dk, dv, dtype, 2 * (n + many))
    assert workspace_bytes(d, n, tokens) > 0 and workspace_bytes(d, n + many, tokens + many) == 0
    got = []
    for lengths, starts in ((LENGTHS, STARTS), (LENGTHS + [1] * many, STARTS + [0] * many)):
        t, k = sum(lengths), len(lengths)
        pool, y = d["pool"].clone(), torch.empty_like(d["y"][:t])
        prefill(d, lengths, [i if i % 2 else -1 for i in range(k)], [k + i for i in range(k)], start=starts, pool=pool, y=y, rows=slice(0, t))
        got.append((y[:tokens], pool[k:k + n]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_poisoned_chunks(dtype):
    """NaN and infinity in x reach no earlier token, no other sequence and no other column's state."""
    d = inputs(9, 600, 1, 2, 64, 64, dtype, 4)
    assert workspace_bytes(d, 2, 600) > 0
    args = ([400, 200], [-1, -1], [0, 1])
    clean = torch.empty_like(d["y"])
    prefill(d, *args, y=clean)
    states = d["pool"][:2].clone()
    e = dict(d, x=d["x"].clone())
    e["x"][130, 1, 5], e["x"][131, 0, 40] = float("nan"), float("inf")
    y = torch.empty_like(clean)
    prefill(e, *args, y=y)
    assert torch.equal(y[:130], clean[:130]) and torch.equal(y[400:], clean[400:]) and torch.equal(d["pool"][1], states[1])
    assert torch.isnan(y[130:400, 1, 5]).all() and not torch.isfinite(y[131:400, 0, 40]).any()
    keep = torch.ones(2, 64, dtype=torch.bool, device="cuda")
    keep[1, 5] = keep[0, 40] = False
    assert torch.equal(y.transpose(0, 1)[keep.nonzero(as_tuple=True)[0], :, keep.nonzero(as_tuple=True)[1]],
                       clean.transpose(0, 1)[keep.nonzero(as_tuple=True)[0], :, keep.nonzero(as_tuple=True)[1]])
    cols = keep[:, None, :].expand(2, 64, 64)
    assert torch.equal(d["pool"][0][cols], states[0][cols])


def test_graph_with_other_splits():
    d = inputs(12, 900, 2, 4, 128, 128, "bf16", 8)
    ws = layer.alloc_ssm_workspace(d["c"], d["x"], 3)
    assert ws is not None
    cu, init, fin = i32([0, 450, 510, 900]), i32([0, -1, 1]), i32([5, 6, 7])

    def step(s, y):
        layer.gdn_ssm_chunk_prefill(s["c"], s["b"], s["x"], s["dt"], s["A"], y, cu, s["pool"], init, fin, dt_bias=s["bias"], D=s["D"], workspace=ws)

    step(d, d["y"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(d, d["y"])
    for seed, split in enumerate(([0, 450, 510, 900], [0, 1, 1, 900], [0, 64, 640, 900])):
        e = inputs(40 + seed, 900, 2, 4, 128, 128, "bf16", 8)
        for k in ("c", "b", "x", "dt", "A", "bias", "D", "pool"):
            d[k].copy_(e[k])
        cu.copy_(i32(split))
        step(e, e["y"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d["y"], e["y"]) and torch.equal(d["pool"], e["pool"])


def test_workspace_refusals():
    d = inputs(1, 300, 1, 2, 64, 64, "bf16", 4)
    s = i32([0])
    ok = dict(c=d["c"], b=d["b"], x=d["x"], dt=d["dt"], A=d["A"], y=d["y"], cu_seqlens=i32([0, 300]), state_pool=d["pool"], init_slot=s, final_slot=s)
    ws = layer.alloc_ssm_workspace(d["c"], d["x"], 1)
    for bad, text in ((None, "workspace_bytes 0"), (ws[:-1], "workspace_bytes"), (torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:], "workspace")):
        with pytest.raises(layer.GdnError, match=text):
            layer.gdn_ssm_chunk_prefill(**ok, workspace=bad)
