"""The step plan on the GPU against one request at a time in Python: whole numbers, equal."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_amd import layer
from tests import layer_reference as R

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def make(rng, requests, B, max_len, max_past, block, kv_block, width=None, kv_width=None):
    computed = rng.integers(0, max_past + 1, requests)
    new = rng.integers(0, max_len + 1, requests)
    new[:B] = 1
    last = max_past + max_len + 1
    width = last // block + 1 if width is None else width
    kv_width = last // kv_block + 1 if kv_width is None else kv_width
    return dict(computed=computed, new=new, state_table=rng.integers(0, 1 << 20, (requests, width)), run_slot=rng.integers(0, 1 << 20, requests),
                kv_table=rng.integers(0, 1 << 24, (requests, kv_width)))


def run(m, B, block, kv_block, tokens, exports, stream=None):
    out = layer.alloc_step_plan(len(m["computed"]), B, tokens, exports, "cuda", kv=m["kv_table"] is not None)
    for t in out.values():
        t.fill_(-7)
    layer.gdn_step_plan(i32(m["computed"]), i32(m["new"]), i32(m["state_table"]), i32(m["run_slot"]), num_decode_rows=B, state_block=block,
                        kv_table=None if m["kv_table"] is None else i32(m["kv_table"]), kv_block=kv_block, stream=stream, **out)
    return out


def check(m, B, block, kv_block, tokens, exports):
    got = run(m, B, block, kv_block, tokens, exports)
    ref = R.plan(m["computed"], m["new"], m["state_table"], m["run_slot"], B, block, m["kv_table"], kv_block, tokens, exports)
    for name, t in got.items():
        assert t.cpu().tolist() == ref[name], name


@pytest.mark.parametrize("requests,B,max_len,max_past,block,kv_block", [
    (1, 0, 1, 0, 64, 1), (1, 1, 1, 5, 64, 16), (5, 0, 300, 500, 64, 16), (64, 64, 1, 8192, 1088, 16), (33, 20, 700, 2000, 128, 24),
    (300, 0, 3, 200, 64, 7), (1500, 700, 40, 3000, 64, 16), (2500, 3, 9, 130, 64, 1), (3, 1, 9000, 5000, 1088, 64)])
def test_plan_matches_reference(requests, B, max_len, max_past, block, kv_block):
    rng = np.random.default_rng(requests + B)
    m = make(rng, requests, B, max_len, max_past, block, kv_block)
    need = B + int(m["new"][B:].sum())
    n_exp = int(((m["computed"] + m["new"]) // block - m["computed"] // block)[B:].sum())
    check(m, B, block, kv_block, need, n_exp)
    check(m, B, block, kv_block, need + 1000, n_exp + 70)         # padding past the end
    check(m, B, block, kv_block, max(0, need - 3), max(0, n_exp - 2))   # buffers that are too small drop the rest


def test_borders_padding_rows_and_empty_prompts():
    """Positions on and beside block borders, decode rows switched off, empty and negative
    lengths, tables that end before the position and negative entries."""
    block = 64
    computed = [0, 1, 63, 64, 65, 128, 127, 500] + [0, 0, 64, 63, 64, 128, 1, -5, 600]
    new = [1, 0, 1, 1, -3, 1, 1, 1] + [0, 64, 0, 1, 64, 129, 200, 10, 3]
    rng = np.random.default_rng(7)
    m = dict(computed=np.array(computed), new=np.array(new), state_table=rng.integers(0, 99, (17, 3)), run_slot=np.arange(100, 117),
             kv_table=rng.integers(-3, 50, (17, 11)))
    check(m, 8, block, 16, 600, 40)
    m["kv_table"] = None
    check(m, 8, block, 0, 600, 40)


def test_no_requests_writes_the_padding():
    m = dict(computed=np.zeros(0), new=np.zeros(0), state_table=np.zeros((0, 4)), run_slot=np.zeros(0), kv_table=np.zeros((0, 4)))
    check(m, 0, 64, 16, 130, 5)


def test_long_cache_slots_pass_32_bits():
    m = dict(computed=np.array([2 ** 31 - 70]), new=np.array([64]), state_table=np.array([[3]]), run_slot=np.array([9]),
             kv_table=np.full((1, 2 ** 31 // 4096), 2 ** 30, dtype=np.int64))
    check(m, 0, 1 << 20, 4096, 64, 0)


def test_plan_feeds_the_rule_as_a_graph():
    """Captured once and replayed with other lengths, each replay equal to the eager call."""
    rng = np.random.default_rng(3)
    B, block, kvb, tokens, exports = 6, 64, 16, 2000, 40
    base = make(rng, 12, B, 200, 300, block, kvb)
    static = {k: i32(v) for k, v in base.items()}
    out = layer.alloc_step_plan(12, B, tokens, exports, "cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.gdn_step_plan(static["computed"], static["new"], static["state_table"], static["run_slot"], num_decode_rows=B, state_block=block,
                            kv_table=static["kv_table"], kv_block=kvb, **out)
    for _ in range(3):
        m = make(rng, 12, B, 200, 300, block, kvb)
        for k, v in m.items():
            static[k].copy_(i32(v))
        eager = run(m, B, block, kvb, tokens, exports)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in out:
            assert torch.equal(out[name], eager[name]), name


def test_refusals():
    m = make(np.random.default_rng(1), 3, 1, 5, 5, 64, 16)
    with pytest.raises(ValueError, match="num_decode_rows"):
        run(m, 1, 64, 16, 10, 0) and layer.gdn_step_plan(i32(m["computed"]), i32(m["new"]), i32(m["state_table"]), i32(m["run_slot"]),
                                                         num_decode_rows=4, state_block=64, **layer.alloc_step_plan(4, 4, 1, 0, "cuda", kv=False))
    with pytest.raises(layer.GdnError, match="state_block 65"):
        run(m, 1, 65, 16, 10, 0)
    with pytest.raises(layer.GdnError, match="kv_block 0"):
        run(m, 1, 64, 0, 10, 0)
