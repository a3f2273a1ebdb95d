"""Rotary positions on the GPU against the formula in 64 bits."""
import pytest
import torch

from gated_deltanet_rule_amd import attention as A
from tests import attention_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def bound(x, y, factor, dtype, half, interleaved):
    """cos and sin: two units in the last place and the angle's rounding (2 pi 2^-25 of a turn's part), 2^-21 of a value in all;
    two products and a sum: 3 roundings; the output's."""
    pair = torch.zeros_like(y)
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    size = (x[..., a].double().abs() + x[..., b].double().abs()) * abs(factor)
    pair[..., a] = size
    pair[..., b] = size
    return R.HALF_STEP[dtype] * y.abs() + pair * (2.0 ** -21 + 3 * 2.0 ** -24) + 1e-30


def run(tokens, hq, hk, d, r, dtype, interleaved, positions, factor=1.0, pad=0, base=10000.0, offset=0):
    g = torch.Generator(device=DEV).manual_seed(tokens * 31 + d + r)
    wide = torch.randn(tokens, (hq + hk) * d + pad + offset, generator=g, device=DEV).to(dtype)[:, offset:]
    q, k = wide[:, : hq * d].unflatten(1, (hq, d)), wide[:, hq * d: (hq + hk) * d].unflatten(1, (hk, d))
    freq, _ = A.rotary_frequencies(r, base, device=DEV)
    qo, ko = torch.full((tokens, hq, d), 7.0, dtype=dtype, device=DEV), torch.full((tokens, hk, d), 7.0, dtype=dtype, device=DEV)
    A.gdn_rotary(q, k, positions, freq, q_out=qo, k_out=ko, interleaved=interleaved, attention_factor=factor)
    live = positions >= 0
    for x, out in ((q, qo), (k, ko)):
        y = R.rotary(x, positions, freq, factor, interleaved)
        R.check("rotary", out[live], y[live], bound(x, y, factor, dtype, r // 2, interleaved)[live])
        assert torch.equal(out[live][..., r:], x[live][..., r:])          # the rest of the head: the same bits
        assert (out[~live] == 7.0).all()
    # in place gives the same bits, and leaves the columns beside the heads alone
    before = wide.clone()
    A.gdn_rotary(q, k, positions, freq, interleaved=interleaved, attention_factor=factor)
    assert torch.equal(q[live], qo[live]) and torch.equal(k[live], ko[live])
    assert torch.equal(q[~live], before[:, : hq * d].unflatten(1, (hq, d))[~live])
    assert torch.equal(wide[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,hq,hk,d,r,pad", [
    (1, 1, 1, 64, 64, 0), (3, 32, 8, 128, 128, 0), (65, 16, 2, 256, 64, 64), (33, 5, 5, 80, 80, 8), (9, 4, 1, 96, 24, 8),
    (7, 3, 1, 10, 6, 3), (5, 2, 2, 512, 512, 0), (2, 1, 3, 128, 2, 0), (1200, 7, 1, 64, 32, 8)])
def test_shapes(tokens, hq, hk, d, r, pad, dtype, interleaved):
    positions = (torch.arange(tokens, device=DEV) * 37 % 8192).to(torch.int32)
    positions[tokens // 2] = -1 if tokens > 2 else 5
    run(tokens, hq, hk, d, r, dtype, interleaved, positions, pad=pad)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_unaligned_rows(dtype):
    run(11, 3, 2, 64, 64, dtype, False, torch.arange(11, dtype=torch.int32, device=DEV), pad=1, offset=1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """fp32 values at positions up to 2^31 - 1 are as exact as at 1."""
    positions = torch.tensor([0, 1, 2 ** 20 + 1, 10 ** 6, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    run(7, 2, 1, 128, 128, F32, interleaved, positions)
    run(7, 2, 1, 128, 128, F32, interleaved, positions, factor=1.3465, base=5e6)


def test_one_of_q_and_k():
    """q alone and k alone give the bits of both together."""
    q, k = torch.randn(5, 4, 64, device=DEV), torch.randn(5, 2, 64, device=DEV)
    positions, freq = torch.arange(5, dtype=torch.int32, device=DEV), A.rotary_frequencies(32, device=DEV)[0]
    qo, ko, q1, k1 = torch.empty_like(q), torch.empty_like(k), q.clone(), k.clone()
    A.gdn_rotary(q, k, positions, freq, q_out=qo, k_out=ko)
    A.gdn_rotary(q1, None, positions, freq)
    A.gdn_rotary(None, k1, positions, freq)
    assert torch.equal(q1, qo) and torch.equal(k1, ko)


def test_no_tokens():
    q, freq = torch.empty(0, 4, 64, device=DEV), A.rotary_frequencies(32, device=DEV)[0]
    A.gdn_rotary(q, None, torch.empty(0, dtype=torch.int32, device=DEV), freq)


def test_rows_do_not_depend_on_the_batch():
    q = torch.randn(5000, 8, 128, device=DEV).to(BF16)
    positions, freq = torch.arange(5000, dtype=torch.int32, device=DEV) * 3, A.rotary_frequencies(128, device=DEV)[0]
    whole, one = torch.empty_like(q), torch.empty_like(q)
    A.gdn_rotary(q, None, positions, freq, q_out=whole)
    for at in (0, 1, 777, 4999):
        A.gdn_rotary(q[at: at + 1], None, positions[at: at + 1], freq, q_out=one[at: at + 1])
        assert torch.equal(one[at], whole[at])
