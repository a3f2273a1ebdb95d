"""A request's first token, planned as a prefill of one token beside decode rows: its outputs and
its state are those of the prompt it begins."""
import pytest
import torch

from gated_deltanet_rule_amd import layer
from tests.test_gpu_layer_plan import i32
from tests.test_gpu_layer_ssm import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_first_token_beside_decode_rows(dtype):
    rows, block = 3, 64                                           # two decode rows, then the new request
    d = inputs(7, rows, 1, 2, 64, 64, dtype, 12)
    plan = layer.alloc_step_plan(rows, 2, rows, 1, "cuda", kv=False)
    layer.gdn_step_plan(i32([10, 63, 0]), i32([1, 1, 1]), i32([[0, 1], [2, 3], [4, 5]]), i32([6, 7, 8]), num_decode_rows=2, state_block=block, **plan)
    assert plan["slot_in"].tolist() == [6, 7] and plan["slot_out"].tolist() == [6, 2]
    assert plan["init_slot"].tolist() == [-1] and plan["final_slot"].tolist() == [8] and plan["cu_seqlens"].tolist() == [0, 1]
    par = dict(dt_bias=d["bias"], D=d["D"])
    pool = d["pool"].clone()
    part = lambda s: [d[k][s] for k in ("c", "b", "x", "dt")]
    layer.gdn_ssm_recurrent_decode(*part(slice(0, 2)), d["A"], d["y"][:2], pool, plan["slot_in"], plan["slot_out"], **par)
    layer.gdn_ssm_chunk_prefill(*part(slice(2, 3)), d["A"], d["y"][2:], plan["cu_seqlens"], pool, plan["init_slot"], plan["final_slot"], **par,
                                start_pos=plan["start_pos"], workspace=layer.alloc_ssm_workspace(d["c"][2:], d["x"][2:], 1))
    assert torch.isfinite(d["y"]).all() and not torch.equal(pool[8], d["pool"][8])
    # S = d b x^T of the one token: the outer product's rank-one form at fp32 accuracy
    raw = d["dt"][2].double() + d["bias"].double()
    step = torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0)
    want = step[:, None, None] * d["b"][2, 0].double()[None, :, None] * d["x"][2].double()[:, None, :]
    assert ((pool[8].double() - want).abs() <= 16 * 2.0 ** -24 * (1 + raw.abs())[:, None, None] * want.abs()).all()
