"""The gated norm and the residual norm on the GPU against fp64."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_amd import layer
from tests import layer_reference as R

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def normal(g, *shape, dtype="f32", pad=0):
    t = torch.randn(shape[:-1] + (shape[-1] + pad,), generator=g).to(TD[dtype]).cuda()
    return t[..., :shape[-1]]


def within(name, got, ref, bound):
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all() and (err <= bound).all(), "%s: worst error / bound %.3g" % (name, np.max(err / bound))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,groups,dim", [(1, 1, 1), (3, 32, 128), (5, 1, 4096), (2, 3, 100), (4, 7, 64), (33, 2, 513), (2, 1, 16384),
                                             (3, 1, 9999), (1, 1, 8), (65, 5, 256), (7, 1, 2056), (2, 2, 12)])
@pytest.mark.parametrize("gate_first,act,per_group", [(False, "silu", False), (True, "silu", True), (False, "sigmoid", True), (True, "none", False)])
def test_gated_norm(dtype, rows, groups, dim, gate_first, act, per_group):
    g = torch.Generator().manual_seed(dim)
    x = normal(g, rows, groups, dim, dtype=dtype)
    z = normal(g, rows, groups * dim, dtype=dtype, pad=8).unflatten(1, (groups, dim))
    w = normal(g, groups, dim) if per_group else normal(g, dim)
    y = torch.full((rows, groups, dim), float("nan"), dtype=TD[dtype], device="cuda")
    layer.gdn_gated_norm(x, z, w, y, eps=1e-5, gate_first=gate_first, activation=act)
    within("y", y, *R.gated_norm(f64(x), f64(z), f64(w), 1e-5, gate_first, act, dtype))
    # in place, and without a gate
    ref, bound = R.gated_norm(f64(x), None, f64(w), 1e-5, gate_first, act, dtype)
    layer.gdn_gated_norm(x, None, w, x, eps=1e-5, gate_first=gate_first, activation=act)
    within("in place", x, ref, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_norm_strides_and_alignment(dtype):
    """Rows that start off 16 bytes, row strides of any size, and the aligned case: equal bits
    for the same values."""
    g = torch.Generator().manual_seed(1)
    x, z, w = normal(g, 9, 4, 128, dtype=dtype), normal(g, 9, 4, 128, dtype=dtype), normal(g, 128)
    want = torch.empty_like(x)
    layer.gdn_gated_norm(x, z, w, want)
    for off, pad in ((0, 8), (1, 3), (3, 0), (8, 5)):
        wide = torch.zeros(9, 512 + off + pad, dtype=TD[dtype], device="cuda")
        xs, zs = wide[:, off:off + 512].unflatten(1, (4, 128)), wide.clone()[:, off:off + 512].unflatten(1, (4, 128))
        xs.copy_(x)
        zs.copy_(z)
        flat = torch.zeros(9 * 512 + off, dtype=TD[dtype], device="cuda")[off:].view(9, 4, 128)
        layer.gdn_gated_norm(xs, zs, w, flat)
        err = (flat.double() - want.double()).abs()
        assert (err <= 2 * R.HALF[dtype] * want.double().abs() + 300 * R.U * want.double().abs()).all()


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 4096), (2, 100), (17, 2048), (1, 16384), (2, 9999), (5, 5000), (40, 64)])
@pytest.mark.parametrize("post,gate,pre", [(True, True, True), (False, False, True), (True, False, False), (False, True, True)])
def test_residual_norm(dtype, res, rows, dim, post, gate, pre):
    g = torch.Generator().manual_seed(dim + post)
    x, r = normal(g, rows, dim, dtype=dtype, pad=24), normal(g, rows, dim, dtype=res)
    gt = normal(g, rows, dim, dtype=dtype, pad=1) if gate else None
    pw, nw = normal(g, dim) if post else None, normal(g, dim) if pre else None
    out = torch.full_like(r, float("nan"))
    y = torch.full((rows, dim), float("nan"), dtype=TD[dtype], device="cuda") if pre else None
    layer.gdn_residual_norm(x, r, out, y, post_weight=pw, gate=gt, residual_scale=0.3, pre_weight=nw, eps=1e-5)
    ref, bound, yref, ybound = R.residual_norm(f64(x), f64(r), f64(pw), f64(gt), "silu", 0.3, f64(nw), 1e-5, dtype, res)
    within("residual", out, ref, bound)
    if pre:
        within("y", y, yref, ybound)
    layer.gdn_residual_norm(x, r, r, y, post_weight=pw, gate=gt, residual_scale=0.3, pre_weight=nw, eps=1e-5)
    assert torch.equal(r, out)                                    # in place


def test_zero_rows_infinities_and_extremes():
    w = torch.ones(128, device="cuda")
    x = torch.zeros(4, 1, 128, device="cuda")
    x[1, 0, 5] = float("inf")
    x[2] = 1e-30
    x[3, 0, 0] = float("nan")
    z = torch.full((4, 1, 128), -3e38, device="cuda")             # the type's lowest values: a gate of zero
    y = torch.empty_like(x)
    layer.gdn_gated_norm(x, None, w, y, eps=1e-6)
    assert (y[0] == 0).all() and (y[2].double() - 1e-27).abs().max() < 1e-32 and torch.isnan(y[3, 0, 0])
    layer.gdn_gated_norm(torch.ones_like(x), z, w, y)
    assert (y == 0).all()
    layer.gdn_gated_norm(torch.ones_like(x), -z, w, y, activation="sigmoid")
    assert (y.double() - 1 / np.sqrt(1 + 1e-6)).abs().max() < 1e-6


def test_offsets_past_32_bits():
    rows, dim = 300_000, 8192                                     # 2.4e9 elements
    x = torch.empty(rows, 1, dim, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, 1, dim).to(torch.bfloat16)
    w = torch.rand(dim, device="cuda")
    y = torch.empty_like(x)
    layer.gdn_gated_norm(x, x, w, y)
    small = torch.empty_like(x[-3:])
    layer.gdn_gated_norm(x[-3:], x[-3:], w, small)
    assert torch.equal(y[-3:], small)


def test_rows_do_not_depend_on_their_call_and_graphs_replay():
    g = torch.Generator().manual_seed(3)
    x, z, w = normal(g, 64, 32, 128, dtype="bf16"), normal(g, 64, 32, 128, dtype="bf16"), normal(g, 128)
    y = torch.empty_like(x)
    layer.gdn_gated_norm(x, z, w, y)
    one = torch.empty_like(x[:1])
    layer.gdn_gated_norm(x[17:18], z[17:18], w, one)
    assert torch.equal(one[0], y[17])
    r, pre = normal(g, 64, 4096), normal(g, 4096)
    flat, out, n = x.flatten(1), torch.empty_like(r), torch.empty(64, 4096, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.gdn_gated_norm(x, z, w, y)
        layer.gdn_residual_norm(flat, r, out, n, gate=z.flatten(1), pre_weight=pre)
    for _ in range(3):
        x.copy_(torch.randn(64, 32, 128))
        r.copy_(torch.randn(64, 4096))
        eager = [torch.empty_like(t) for t in (y, out, n)]
        layer.gdn_gated_norm(x, z, w, eager[0])
        layer.gdn_residual_norm(flat, r, eager[1], eager[2], gate=z.flatten(1), pre_weight=pre)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (y, out, n)):
            assert torch.equal(a, b)


def test_refusals():
    x, w = torch.zeros(2, 3, 64, device="cuda"), torch.ones(64, device="cuda")
    for args, kw, err, text in [
            ((x.half(), None, w, x), {}, ValueError, "bfloat16 or float32"), ((x, x[:1], w, x), {}, ValueError, "z must have shape"),
            ((x, None, w[:32], x), {}, ValueError, "weight"), ((x[..., ::2], None, w[:32], x), {}, ValueError, "dense rows"),
            ((x, None, w, x.bfloat16()), {}, ValueError, "y must be"), ((x, None, w, x), dict(eps=-1.0), layer.GdnError, "eps"),
            ((x, None, w, x), dict(activation="relu"), ValueError, "activation")]:
        with pytest.raises(err, match=text):
            layer.gdn_gated_norm(*args, **kw)
    f = x[:, 0]
    with pytest.raises(ValueError, match="pre_weight"):
        layer.gdn_residual_norm(f, f.contiguous(), f.contiguous(), f.contiguous())
    with pytest.raises(layer.GdnError, match="residual_dtype"):
        layer.gdn_residual_norm(f, f.contiguous().bfloat16(), f.contiguous().bfloat16())


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("dim", [3, 7, 9, 37, 129, 999, 2051, 4099, 9999])
@pytest.mark.parametrize("post", [True, False])
def test_rows_that_end_inside_a_vector_in_place(dtype, res, dim, post):
    """Odd rows in place (the residual over itself, the gated norm over its input): the same bits as
    into other memory, and nothing past the last row."""
    g = torch.Generator().manual_seed(dim)
    rows = 70
    x, r = normal(g, rows, dim, dtype=dtype), normal(g, rows, dim, dtype=res)
    w = 1.0 + normal(g, dim, dtype="f32") * 0.1
    out, y = torch.empty_like(r), torch.empty_like(x)
    kw = dict(post_weight=w if post else None, pre_weight=w, residual_scale=0.5)
    layer.gdn_residual_norm(x, r, out, y, **kw)
    guard = torch.full((rows + 1, dim), 7.0, dtype=r.dtype, device="cuda")
    guard[:rows] = r
    y2 = torch.full((rows + 1, dim), 7.0, dtype=x.dtype, device="cuda")
    layer.gdn_residual_norm(x, guard[:rows], guard[:rows], y2[:rows], **kw)
    assert torch.equal(guard[:rows], out) and torch.equal(y2[:rows], y) and (guard[rows] == 7).all() and (y2[rows] == 7).all()
    layer.gdn_gated_norm(x[:, None], x[:, None], w, y[:, None])
    same = torch.full((rows + 1, dim), 7.0, dtype=x.dtype, device="cuda")
    same[:rows] = x
    layer.gdn_gated_norm(same[:rows, None], x[:, None], w, same[:rows, None])
    assert torch.equal(same[:rows], y) and (same[rows] == 7).all()
