"""Attention over a paged cache on the GPU against the formula in 64 bits: packed prompts and decode rows, every
format, masks that leave rows empty, pages that end inside a tile, everything unowned poisoned."""
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


def setup(past, new, hq, hkv, d, dtype, fmt, kv_block, seed=1, pad=0):
    keys = [p + n for p, n in zip(past, new)]
    table, rows = C.pages(keys, kv_block, DEV, seed)
    own = C.owned_rows(table, kv_block, keys)
    cache = C.filled_cache(rows, hkv, d, dtype, fmt, own, DEV, seed)
    return table, cache, C.queries(sum(new), hq, d, dtype, DEV, seed + 100, pad)


def prefill(q, cache, table, kv_block, past, new, scale, extra=0, **kw):
    o = torch.full((q.shape[0] + extra, q.shape[1], q.shape[2]), 5.0, dtype=q.dtype, device=DEV)
    full = q if not extra else torch.cat([q, torch.full_like(q[:1], math.nan).expand(extra, -1, -1)])
    start = None if not any(past) else C.i32(past, DEV)
    A.gdn_attention_prefill(full, o=o, cu_seqlens=C.packed(new, DEV), start_pos=start, kv_table=table, kv_block=kv_block, scale=scale, **cache, **kw)
    assert (o[q.shape[0]:] == 5.0).all()          # rows behind the last sequence: left as they were
    return o[: q.shape[0]]


def decode(q, cache, table, kv_block, past, per, scale, mask=None, max_keys=0):
    o = torch.full(q.shape, 5.0, dtype=q.dtype, device=DEV)
    keys = max_keys or table.shape[1] * kv_block
    ws = A.alloc_attention_workspace(q, cache["k_cache"], tokens_per_row=per, max_keys=keys)
    if ws is not None:
        ws.fill_(0xff)                             # NaN: nothing that a call did not write may count
    A.gdn_attention_decode(q, o=o, computed=C.i32(past, DEV), kv_table=table, kv_block=kv_block, scale=scale, tokens_per_row=per, tree_mask=mask,
                           max_keys=max_keys, workspace=ws, **cache)
    return o


def visible(masks, rows, per):
    bits = masks.view(rows, per, 1) >> torch.arange(per, device=masks.device)
    return [(bits[b] & 1).bool() for b in range(rows)]


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("past,new,hq,hkv,d,kv_block", [
    ([0], [1], 1, 1, 64, 16), ([0], [256], 1, 1, 64, 16), ([0, 0, 0], [70, 1, 129], 8, 2, 128, 16),
    ([5, 100, 0, 63], [65, 0, 33, 64], 4, 4, 128, 24), ([200, 1], [130, 300], 16, 2, 256, 64), ([31], [97], 7, 1, 128, 1),
    ([1000, 77], [17, 3], 6, 2, 64, 256), ([129], [200], 3, 1, 256, 16), ([64, 64], [64, 128], 14, 2, 64, 1088)])
def test_prefill(past, new, hq, hkv, d, kv_block, dtype, fmt):
    table, cache, q = setup(past, new, hq, hkv, d, dtype, fmt, kv_block)
    o = prefill(q, cache, table, kv_block, past, new, d ** -0.5, extra=3)
    R.check("prefill", o, *R.attention(q, cache, table, kv_block, past, new, d ** -0.5))


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("past,per,hq,hkv,d,kv_block", [
    ([1], 1, 1, 1, 64, 16), ([0, 5, 31, 64], 1, 8, 2, 128, 16), ([300, 1, 1023], 1, 32, 8, 128, 16), ([2500, 77], 1, 16, 2, 256, 64),
    ([700], 1, 7, 1, 128, 24), ([129, 600], 1, 40, 1, 64, 1), ([5000], 1, 3, 3, 128, 1088), ([100, 0, 2000], 3, 8, 2, 128, 16),
    ([333], 17, 4, 2, 64, 16), ([64, 1500], 64, 8, 1, 128, 16), ([600], 9, 16, 2, 256, 24), ([40, 900], 33, 6, 2, 256, 16)])
def test_decode_and_chains(past, per, hq, hkv, d, kv_block, dtype, fmt):
    new = [per] * len(past)
    table, cache, q = setup(past, new, hq, hkv, d, dtype, fmt, kv_block)
    o = decode(q, cache, table, kv_block, past, per, d ** -0.5)
    R.check("decode", o, *R.attention(q, cache, table, kv_block, past, new, d ** -0.5))


def random_tree(rows, per, seed):
    g = torch.Generator().manual_seed(seed)
    parents = [[int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(per)] for _ in range(rows)]
    return A.tree_masks(parents, DEV)[0]


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("past,per,hq,hkv,d,kv_block", [
    ([0, 7], 5, 4, 2, 64, 16), ([500, 31], 8, 8, 2, 128, 16), ([1000, 0, 65], 32, 8, 8, 128, 24), ([700, 190], 64, 4, 1, 128, 16), ([320], 12, 16, 2, 256, 64),
    ([257], 64, 7, 1, 256, 1)])
def test_trees(past, per, hq, hkv, d, kv_block, dtype, fmt):
    rows = len(past)
    table, cache, q = setup(past, [per] * rows, hq, hkv, d, dtype, fmt, kv_block)
    mask = random_tree(rows, per, per)
    o = decode(q, cache, table, kv_block, past, per, d ** -0.5, mask)
    R.check("tree", o, *R.attention(q, cache, table, kv_block, past, [per] * rows, d ** -0.5, visible(mask, rows, per)))
    # bits from tokens_per_row on are not looked at
    if per < 64:
        assert torch.equal(decode(q, cache, table, kv_block, past, per, d ** -0.5, mask | (-1 << per)), o)


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("per,hq,hkv,d", [(6, 4, 2, 64), (40, 8, 2, 128), (7, 8, 1, 256)])
def test_rows_that_see_nothing(per, hq, hkv, d, dtype, fmt):
    """Padding rows, tokens with an empty mask in a row without a context, later tokens that an earlier one sees."""
    past, rows = [0, -1, 90, 0, -2 ** 31], 5
    table, cache, q = setup([max(p, 0) for p in past], [per] * rows, hq, hkv, d, dtype, fmt, 16)
    mask = random_tree(rows, per, 3).view(rows, per)
    mask[0, 1:4] = 0
    mask[2, 2] = 0
    mask[3] = 0
    mask[3, per - 1] = 1 << (per - 1)
    mask[3, 0] = 1 << (per - 1)
    seen = visible(mask.flatten(), rows, per)
    o = decode(q, cache, table, 16, past, per, d ** -0.5, mask.flatten().contiguous()).view(rows, per, hq, d)
    ref, bound = (t.view(rows, per, hq, d) for t in R.attention(q, cache, table, 16, [max(p, 0) for p in past], [per] * rows, d ** -0.5, seen))
    for b in (1, 4):
        ref[b], bound[b] = 0, 1e-30
    R.check("empty", o, ref, bound)
    assert (o[0, 1:4] == 0).all() and (o[3, 1: per - 1] == 0).all()


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_absent_pages(d, dtype, fmt):
    """Negative entries, entries behind the cache and tables that end early: those keys are seen by no token."""
    past, new, block = [100, 3, 250, 0], [30, 70, 5, 65], 16
    table, cache, q = setup(past, new, 4, 2, d, dtype, fmt, block)
    table[0, 2] = -1
    table[0, 3] = -7
    table[2, 10] = cache["k_cache"].shape[0] // block
    table[2, 0] = 2 ** 31 - 1
    table[3] = -1
    o = prefill(q, cache, table, block, past, new, d ** -0.5)
    R.check("absent", o, *R.attention(q, cache, table, block, past, new, d ** -0.5))
    assert (o[-65:] == 0).all()
    short = table[:, :5].contiguous()
    o = prefill(q, cache, short, block, past, new, d ** -0.5)
    R.check("short table", o, *R.attention(q, cache, short, block, past, new, d ** -0.5))
    q1 = q[:8]
    o = decode(q1, cache, table, block, past, 2, d ** -0.5)
    R.check("absent, decode", o, *R.attention(q1, cache, table, block, past, [2] * 4, d ** -0.5))
    o = decode(q1, cache, short, block, past, 2, d ** -0.5)
    R.check("short table, decode", o, *R.attention(q1, cache, short, block, past, [2] * 4, d ** -0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_cache(dtype):
    q = torch.randn(6, 4, 64, device=DEV).to(dtype)
    cache = A.alloc_kv_cache(0, 2, 64, dtype, DEV)
    table = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    assert (prefill(q, cache, table, 16, [4, 0], [3, 3], 1.0) == 0).all()
    assert (decode(q, cache, table, 16, [4, 0], 3, 1.0) == 0).all()
    none = torch.zeros(2, 0, dtype=torch.int32, device=DEV)
    full = C.filled_cache(48, 2, 64, dtype, None, torch.arange(48, device=DEV), DEV, 1)
    assert (prefill(q, full, none, 16, [4, 0], [3, 3], 1.0) == 0).all()
    assert (decode(q, full, none, 16, [4, 0], 3, 1.0) == 0).all()
    assert decode(q[:0], full, table[:0], 16, [], 3, 1.0).shape[0] == 0
    assert prefill(q[:0], full, table, 16, [4, 0], [0, 0], 1.0).shape[0] == 0


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_non_finite_places_that_are_not_seen(d, dtype, fmt):
    """Infinities and NaN in later tokens' keys and values, and in branches of a tree, leave other tokens as they were, bit for bit;
    the tokens that see them are not finite."""
    past, new, block, hq = [50, 3], [90, 40], 16, 4
    table, cache, q = setup(past, new, hq, 2, d, dtype, fmt, block)
    clean = prefill(q, cache, table, block, past, new, d ** -0.5)
    row = lambda b, p: int(table[b, p // block]) * block + p % block  # noqa: E731

    def poison(b, p, name, value, column=None):
        c, s = cache[name + "_cache"], cache[name + "_scale"]
        if fmt is None:
            c[row(b, p), :, slice(None) if column is None else column] = value
        elif fmt == "e4m3" and column is not None:
            c.view(torch.uint8)[row(b, p), :, column] = 0x7f
        else:
            s[row(b, p)] = value

    poison(0, 80, "v", math.nan, 5)
    poison(0, 81, "v", math.inf, d - 1)
    poison(0, 82, "v", -math.inf, d // 2)
    poison(0, 60 + 64, "k", math.nan)
    poison(1, 20, "k", math.inf, 3)
    poison(1, 21, "v", math.nan)
    o = prefill(q, cache, table, block, past, new, d ** -0.5)
    assert torch.equal(o[:30], clean[:30]) and torch.equal(o[90: 107], clean[90: 107])
    assert not torch.isfinite(o[30: 90].float()).all(2).all(1).any() and not torch.isfinite(o[108: 130].float()).all(2).all(1).any()
    # a tree of 24 tokens behind 76: the poisoned keys are tokens 4, 5, 6 (and 48 is out of it), each seen by itself and one child
    per = 24
    parents = [[-1] * 4 + [0, 1, 2, 4, 5, 6] + [3] * (per - 10)]
    mask = A.tree_masks(parents, DEV)[0]
    qt = q[:per]
    with_poison = decode(qt, cache, table[:1].contiguous(), block, [76], per, d ** -0.5, mask)
    hit = torch.zeros(per, dtype=torch.bool, device=DEV)
    hit[4:10] = True
    finite = torch.isfinite(with_poison.float()).all(2).all(1)
    assert torch.equal(finite, ~hit), finite
    for p, name in ((80, "v"), (81, "v"), (82, "v")):
        c, s = cache[name + "_cache"], cache[name + "_scale"]
        if fmt is None:
            c[row(0, p)] = 0
        else:
            s[row(0, p)] = 1.0
            c.view(torch.uint8)[row(0, p)] = 0
    without = decode(qt, cache, table[:1].contiguous(), block, [76], per, d ** -0.5, mask)
    assert torch.equal(with_poison[~hit], without[~hit])


@pytest.mark.parametrize("dtype,fmt", FORMATS)
def test_large_scores_and_one_hot(dtype, fmt):
    """Scores of hundreds either way: the softmax picks one key; the running maximum rises and falls along the keys."""
    d, n = 128, 700
    table, cache, q = setup([n], [8], 2, 1, d, dtype, fmt, 16)
    o = prefill(q * 8, cache, table, 16, [n], [8], 4.0)
    R.check("large", o, *R.attention(q * 8, cache, table, 16, [n], [8], 4.0))
    o = decode((q * 8)[:1], cache, table, 16, [n], 1, 4.0)
    R.check("large, decode", o, *R.attention((q * 8)[:1], cache, table, 16, [n], [1], 4.0))
    o = decode(q[:1], cache, table, 16, [n], 1, 0.0)
    R.check("even", o, *R.attention(q[:1], cache, table, 16, [n], [1], 0.0))
    o = decode(q[:1], cache, table, 16, [n], 1, -0.5)
    R.check("negative scale", o, *R.attention(q[:1], cache, table, 16, [n], [1], -0.5))


@pytest.mark.parametrize("dtype,fmt", [(BF16, None), (BF16, "e4m3"), (F32, None)])
def test_strided_queries(dtype, fmt):
    past, new = [40, 0], [33, 20]
    table, cache, q = setup(past, new, 4, 2, 128, dtype, fmt, 16, pad=24)
    assert not q.is_contiguous()
    assert torch.equal(prefill(q, cache, table, 16, past, new, 0.1), prefill(q.contiguous(), cache, table, 16, past, new, 0.1))
    assert torch.equal(decode(q[:4], cache, table, 16, past, 2, 0.1), decode(q[:4].contiguous(), cache, table, 16, past, 2, 0.1))


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (3, 1, 64), (16, 2, 256)])
def test_bits_do_not_depend_on_the_call(hq, hkv, d, dtype, fmt):
    """A prompt alone, beside others and in pieces; a decode row alone and beside others: the same bits."""
    past, new, block = [0, 37, 400], [333, 150, 90], 16
    table, cache, q = setup(past, new, hq, hkv, d, dtype, fmt, block)
    whole = prefill(q, cache, table, block, past, new, d ** -0.5)
    at = 0
    for i, n in enumerate(new):
        mine = table[i: i + 1].contiguous()
        assert torch.equal(prefill(q[at: at + n], cache, mine, block, [past[i]], [n], d ** -0.5), whole[at: at + n])
        done = 0
        for piece in (1, 63, 5, 17, n):
            piece = min(piece, n - done)
            got = prefill(q[at + done: at + done + piece], cache, mine, block, [past[i] + done], [piece], d ** -0.5)
            assert torch.equal(got, whole[at + done: at + done + piece]), (i, done, piece)
            done += piece
        at += n
    for per in (1, 4, 21):
        ctx = [300, 20, 469]
        rows = decode(q[: 3 * per], cache, table, block, ctx, per, d ** -0.5)
        for b in range(3):
            one = decode(q[b * per: (b + 1) * per], cache, table[b: b + 1].contiguous(), block, [ctx[b]], per, d ** -0.5, max_keys=ctx[b] + per)
            assert torch.equal(one, rows[b * per: (b + 1) * per]), (per, b)
        # the chain as a tree
        parents = [[i - 1 for i in range(per)]] * 3
        assert torch.equal(decode(q[: 3 * per], cache, table, block, ctx, per, d ** -0.5, A.tree_masks(parents, DEV)[0]), rows)


@pytest.mark.parametrize("per", [1, 20])
@pytest.mark.parametrize("dtype,fmt", [(BF16, None), (F32, "int8")])
def test_rows_longer_than_max_keys_are_nan(per, dtype, fmt):
    table, cache, q = setup([100, 700, 300], [per] * 3, 4, 2, 128, dtype, fmt, 16)
    free = decode(q, cache, table, 16, [100, 700, 300], per, 0.1).view(3, per, 4, 128)
    tight = decode(q, cache, table, 16, [100, 700, 300], per, 0.1, max_keys=300 + per).view(3, per, 4, 128)
    assert torch.equal(tight[0], free[0]) and torch.equal(tight[2], free[2])
    assert tight[1].isnan().all()


def test_workspace_of_a_larger_call():
    """A workspace made for the largest step serves every smaller one."""
    d, dtype = 128, BF16
    table, cache, q = setup([3000, 90], [40] * 2, 8, 2, d, dtype, "e4m3", 16)
    big = A.alloc_attention_workspace(torch.empty(4 * 40, 8, d, dtype=dtype, device=DEV), cache["k_cache"], tokens_per_row=40, max_keys=4000)
    for per in (1, 2, 7, 40):
        want = decode(q[: 2 * per], cache, table, 16, [3000, 90], per, 0.1)
        o = torch.empty_like(want)
        A.gdn_attention_decode(q[: 2 * per], o=o, computed=C.i32([3000, 90], DEV), kv_table=table, kv_block=16, scale=0.1, tokens_per_row=per,
                               workspace=big, **cache)
        assert torch.equal(o, want)


@pytest.mark.parametrize("dtype,fmt", [(BF16, None), (BF16, "int8")])
def test_cache_past_32_bits(dtype, fmt):
    """Pages behind 2^32 bytes, and 2^31 elements, of a cache."""
    heads, d, block = 8, 128, 64
    size = 2 if fmt is None else 1
    rows = ((1 << 32) // (heads * d * size) // block + 40) * block
    cache = A.alloc_kv_cache(rows, heads, d, dtype, DEV, fmt)
    last = rows // block
    table = torch.tensor([[last - 1, 3, last - 20], [last - 7, last // 2, 0]], dtype=torch.int32, device=DEV)
    past, new = [130, 70], [50, 100]
    own = C.owned_rows(table, block, [180, 170])
    small = C.filled_cache(own.shape[0], heads, d, dtype, fmt, torch.arange(own.shape[0], device=DEV), DEV, 1)
    for n, t in cache.items():
        if t is not None:
            t.view(torch.uint8)[own] = small[n].view(torch.uint8)
    q = C.queries(150, 16, d, dtype, DEV, 3)
    compact = torch.zeros_like(table)
    # the same keys from a small cache of one page for each request's block
    packed_rows = A.alloc_kv_cache(6 * block, heads, d, dtype, DEV, fmt)
    flat = table.flatten().tolist()
    for i, page in enumerate(flat):
        for n, t in packed_rows.items():
            if t is not None:
                t.view(torch.uint8)[i * block: (i + 1) * block] = cache[n].view(torch.uint8)[page * block: (page + 1) * block]
        compact.view(-1)[i] = i
    assert torch.equal(prefill(q, cache, table, block, past, new, 0.1), prefill(q, packed_rows, compact, block, past, new, 0.1))
    assert torch.equal(decode(q[:4], cache, table, block, past, 2, 0.1), decode(q[:4], packed_rows, compact, block, past, 2, 0.1))


def test_another_stream_and_a_graph():
    """Enqueued on a stream of the caller's, captured once, replayed with other inputs: each replay is the eager call."""
    d, block, per = 128, 16, 4
    past, new = [900, 40], [per, per]
    table, cache, q = setup([901, 41], new, 8, 2, d, BF16, "e4m3", block)
    computed, o = C.i32(past, DEV), torch.empty(2 * per, 8, d, dtype=BF16, device=DEV)
    ws = A.alloc_attention_workspace(q, cache["k_cache"], tokens_per_row=per, max_keys=table.shape[1] * block)
    o2, cu, start = torch.empty_like(o), C.packed(new, DEV), C.i32(past, DEV)

    def step(stream=None):
        A.gdn_attention_decode(q, o=o, computed=computed, kv_table=table, kv_block=block, scale=0.1, tokens_per_row=per, workspace=ws, stream=stream, **cache)
        A.gdn_attention_prefill(q, o=o2, cu_seqlens=cu, start_pos=start, kv_table=table, kv_block=block, scale=0.1, stream=stream, **cache)

    step()
    want = o.clone(), o2.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o.zero_(), o2.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want[0]) and torch.equal(o2, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        q.copy_(C.queries(2 * per, 8, d, BF16, DEV, 50 + i))
        computed.copy_(C.i32([900 - 211 * i, 40 - 13 * i], DEV))
        start.copy_(computed)
        step()
        torch.cuda.synchronize()
        want = o.clone(), o2.clone()
        o.fill_(3.0), o2.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(o2, want[1]), i
