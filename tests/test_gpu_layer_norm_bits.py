"""A row's bits depend on its dim alone: the norms over aligned rows, and over the same values
at other alignments and row strides, are equal bit for bit."""
import pytest
import torch

from gated_deltanet_rule_amd import layer
from tests.test_gpu_layer_norm import TD, normal

pytestmark = pytest.mark.gpu
PLACES = ((0, 8), (1, 3), (3, 0), (8, 5))          # elements before a matrix of rows, elements between rows


def moved(t, off, pad):
    """The same rows at another alignment and row stride."""
    rows, dim = t.shape
    wide = torch.zeros(rows * (dim + pad) + off, dtype=t.dtype, device="cuda")[off:].view(rows, dim + pad)[:, :dim]
    wide.copy_(t)
    return wide


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("groups,dim", [(4, 8), (4, 128), (3, 256), (2, 1024), (1, 4096), (1, 16384)])
@pytest.mark.parametrize("gate_first", [False, True])
def test_gated_norm(dtype, groups, dim, gate_first):
    g = torch.Generator().manual_seed(dim)
    x, z, w = normal(g, 9, groups * dim, dtype=dtype), normal(g, 9, groups * dim, dtype=dtype), normal(g, dim)
    shape = (groups, dim)
    want = torch.empty(9, groups, dim, dtype=TD[dtype], device="cuda")
    layer.gdn_gated_norm(x.unflatten(1, shape), z.unflatten(1, shape), w, want, gate_first=gate_first)
    for off, pad in PLACES:
        got = moved(want.flatten(1), off, 0).view(9, groups, dim)
        got.fill_(float("nan"))
        layer.gdn_gated_norm(moved(x, off, pad).unflatten(1, shape), moved(z, off, pad).unflatten(1, shape), w, got, gate_first=gate_first)
        assert torch.equal(got, want), (off, pad)


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("dim", [8, 64, 256, 512, 2048, 4096, 8192, 16384])
@pytest.mark.parametrize("post,gate", [(True, True), (False, False)])
def test_residual_norm(dtype, res, dim, post, gate):
    g = torch.Generator().manual_seed(dim)
    x, r, z = normal(g, 9, dim, dtype=dtype), normal(g, 9, dim, dtype=res), normal(g, 9, dim, dtype=dtype)
    kw = dict(post_weight=normal(g, dim) if post else None, pre_weight=normal(g, dim), residual_scale=0.3)
    out, y = torch.empty_like(r), torch.empty_like(x)
    layer.gdn_residual_norm(x, r, out, y, gate=z if gate else None, **kw)
    for off, pad in PLACES:
        o2, y2 = moved(torch.zeros_like(r), off, 0), moved(torch.zeros_like(x), off, 0)
        layer.gdn_residual_norm(moved(x, off, pad), moved(r, off, 0), o2, y2, gate=moved(z, off, pad) if gate else None, **kw)
        assert torch.equal(o2, out) and torch.equal(y2, y), (off, pad)
