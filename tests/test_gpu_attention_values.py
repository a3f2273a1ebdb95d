"""What attention makes of values on the GPU: rows that a few keys dominate, and infinities that a token sees."""
import math

import pytest
import torch

from gated_deltanet_rule_amd import attention as A
from tests import attention_cases as C
from tests import attention_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
FORMATS = [(BF16, None), (BF16, "e4m3"), (BF16, "int8"), (F32, None), (F32, "e4m3"), (F32, "int8")]


def prefill(q, cache, table, past, scale):
    o = torch.full_like(q, 5.0)
    A.gdn_attention_prefill(q, o=o, cu_seqlens=C.packed([q.shape[0]], DEV), start_pos=C.i32([past], DEV), kv_table=table, kv_block=16, scale=scale, **cache)
    return o


def decode(q, cache, table, past, scale):
    o = torch.full_like(q, 5.0)
    ws = A.alloc_attention_workspace(q, cache["k_cache"], tokens_per_row=q.shape[0], max_keys=past + q.shape[0])
    A.gdn_attention_decode(q, o=o, computed=C.i32([past], DEV), kv_table=table, kv_block=16, scale=scale, tokens_per_row=q.shape[0],
                           max_keys=past + q.shape[0], workspace=ws, **cache)
    return o


@pytest.mark.parametrize("hq,d,past,new,how", [(1, 64, 300, 1, decode), (16, 128, 700, 1, decode), (8, 256, 200, 2, decode), (16, 128, 300, 33, decode),
                                               (4, 64, 100, 40, prefill), (8, 128, 0, 200, prefill), (4, 256, 300, 50, prefill)])
def test_rounded_weights_cancel(hq, d, past, new, how):
    """The weights of a plain bf16 cache are rounded to bf16, and their sum is the sum of the rounded ones: with w_j (1 + e_j),
    |e_j| <= 2^-8, the output is off by sum_j p_j e_j (v_j - o) / (1 + sum_j p_j e_j), which vanishes where one key has
    nearly all of the weight, however far above the running maximum of its time it came."""
    table, rows = C.pages([past + new], 16, DEV, 3)
    at = C.owned_rows(table, 16, [past + new])
    cache = C.filled_cache(rows, 1, d, BF16, None, at, DEV, 3)
    # queries and keys of -1, 0 and 1: a score is a whole number, exact in fp32, of some 5 either way
    g = torch.Generator(device=DEV).manual_seed(8)
    q = torch.randint(-1, 2, (new, hq, d), generator=g, device=DEV).to(BF16)
    cache["k_cache"][at] = torch.randint(-1, 2, (past + new, 1, d), generator=g, device=DEV).to(BF16)
    scale = 1.0 if d <= 128 else 0.5
    o = how(q, cache, table, past, scale).double()
    k, v = cache["k_cache"][at, 0].double(), cache["v_cache"][at, 0].double()
    seen = torch.ones(new, past + new, dtype=torch.bool, device=DEV).tril(past)
    score = (torch.matmul(q.double().view(-1, d), k.t().contiguous()).view(new, hq, -1) * scale).masked_fill(~seen[:, None], -math.inf)
    p = torch.softmax(score, -1)
    exact = torch.matmul(p.view(new * hq, -1), v).view(new, hq, d)
    away, spread = torch.zeros_like(exact), torch.matmul(p.view(new * hq, -1), v.abs()).view(new, hq, d)
    for t in range(new):
        away[t] = (p[t][..., None] * (v - exact[t][:, None]).abs()).sum(1)
    # in the exponent: log2 e, the score's product, the largest score's and their difference rounded, each 2^-24 of at most
    # twice the largest; 16 roundings of the exponential and the inverse; sums over the keys
    largest = score.masked_fill(~seen[:, None], 0.0).abs().amax(-1, keepdim=True)
    eps = 2.0 ** -24 * (6 * 1.4427 * largest + 16)
    before = 2.0 ** -8 / (1 - 2.0 ** -8) * away + (2 * eps + 2 * (past + new + 64) * 2.0 ** -24) * spread
    # the output's rounding: half a step of the binade that the value before it may lie in
    half = torch.ldexp(torch.ones_like(exact), torch.frexp(exact.abs() + before).exponent - 9)
    off = (o - exact).abs()
    assert (off <= before + half).all(), "off by up to %.3g of what is allowed" % float((off / (before + half)).max())


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_infinities_that_are_seen(d, dtype, fmt):
    """An infinite value counts by its weight: an infinity where that is positive, NaN where it underflows to zero, wherever the
    token stands in its call.  (In 8 bits such a head is NaN.)"""
    n, first, second, block, hq = 260, 20, 140, 16, 2
    table, rows = C.pages([n], block, DEV, 5)
    own = C.owned_rows(table, block, [n])
    cache = C.filled_cache(rows, 1, d, dtype, fmt, own, DEV, 5)
    # query head 0's score is higher with key 10 than with any other by 288 powers of two; query head 1 sees all alike
    q = torch.ones(n, hq, d, dtype=dtype, device=DEV)
    q[:, 1] = 0
    k = torch.zeros(rows, 1, d, dtype=dtype, device=DEV)
    k[own[10]] = 1
    v = torch.ones(rows, 1, d, dtype=dtype, device=DEV)
    v[own[first], :, 3] = math.inf
    v[own[first], :, 4] = -math.inf
    v[own[second], :, 5] = math.inf
    A.gdn_kv_cache_write(k, v, torch.arange(rows, device=DEV), **cache)
    scale = 200.0 / d
    whole = prefill(q, cache, table, 0, scale)
    finite = torch.isfinite(whole.float())
    assert finite[:first].all()
    if fmt is None:
        assert whole[first:, 0, 3: 5].isnan().all() and whole[second:, 0, 5].isnan().all()
        assert (whole[first:, 1, 3] == math.inf).all() and (whole[first:, 1, 4] == -math.inf).all() and (whole[second:, 1, 5] == math.inf).all()
        assert finite[first: second, :, 5].all() and finite[:, :, 6:].all() and finite[:, :, :3].all()
    else:
        assert whole[first:].isnan().all()

    def same(a, b):
        return torch.equal(a.float().nan_to_num(7.0, 8.0, 9.0), b.float().nan_to_num(7.0, 8.0, 9.0))

    for cuts in ([0, 1, 20, 21, 64, 139, n], [0, 30, 31, 128, 141, n], [0, 70, 140, 200, n]):
        for a, b in zip(cuts, cuts[1:]):
            assert same(prefill(q[a:b], cache, table, a, scale), whole[a:b]), (a, b)
    # and in decode rows: a chain, where some tokens do not see the infinity or all do
    for start in (5, 15, 30, 100, 135, 150, 200):
        for per in (1, 7, 50):
            want = whole[start: start + per].float()
            got = decode(q[start: start + per].contiguous(), cache, table, start, scale).float()
            assert torch.equal(torch.isfinite(got), torch.isfinite(want)) and torch.equal(got.isnan(), want.isnan()), (start, per)


@pytest.mark.parametrize("dtype,fmt", [(BF16, "e4m3"), (BF16, "int8"), (F32, "e4m3"), (F32, "int8")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_infinite_scales(d, dtype, fmt):
    """A head of values whose scale is infinite is NaN to the tokens that see it, in whatever call, and nothing to others."""
    n, at = 200, 20
    table, rows = C.pages([n], 16, DEV, 5)
    own = C.owned_rows(table, 16, [n])
    cache = C.filled_cache(rows, 2, d, dtype, fmt, own, DEV, 5)
    q = C.queries(n, 4, d, dtype, DEV, 5)
    clean = prefill(q, cache, table, 0, 0.1)
    cache["v_scale"][own[at], 1] = math.inf
    cache["v_cache"].view(torch.uint8)[own[at], 1, :5] = 0          # codes of zero among them
    whole = prefill(q, cache, table, 0, 0.1)
    assert torch.equal(whole[:at], clean[:at]) and torch.equal(whole[:, :2], clean[:, :2]) and whole[at:, 2:].isnan().all()
    for a, b in ((0, 21), (19, 22), (21, 64), (64, 200), (70, 71), (130, 190)):
        part = prefill(q[a:b], cache, table, a, 0.1)
        assert torch.equal(part.nan_to_num(7.0), whole[a:b].nan_to_num(7.0)), (a, b)
    for start, per in ((5, 1), (5, 40), (15, 10), (21, 1), (30, 50), (150, 33)):
        got = decode(q[start: start + per].contiguous(), cache, table, start, 0.1)
        assert torch.equal(got.isnan(), whole[start: start + per].isnan()), (start, per)
