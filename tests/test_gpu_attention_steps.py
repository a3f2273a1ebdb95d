"""The attention layers' operators run together as a serving step runs them: the step's plan, rotary positions,
keys and values into the paged cache, decode rows and prompts over it; prompts in pieces, drafted trees, a
captured step.  Each operator's output is compared with the formula in 64 bits on what it was given."""
import math

import pytest
import torch

from gated_deltanet_rule_amd import attention as A
from gated_deltanet_rule_amd import layer
from tests import attention_cases as C
from tests import attention_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
FORMATS = [(BF16, None), (BF16, "e4m3"), (BF16, "int8"), (F32, None), (F32, "e4m3"), (F32, "int8")]
HQ, HKV, BLOCK = 8, 2, 24


class Engine:
    """One attention layer's cache and tables for requests of at most `longest` tokens each."""

    def __init__(self, requests, longest, d, dtype, fmt, seed=5):
        self.d, self.dtype = d, dtype
        self.table, rows = C.pages([longest] * requests, BLOCK, DEV, seed)
        own = torch.zeros(0, dtype=torch.int64, device=DEV)
        self.cache = C.filled_cache(rows, HKV, d, dtype, fmt, own, DEV, seed)          # NaN everywhere
        self.freq, self.factor = A.rotary_frequencies(d, 10000.0, scaling="ramp", factor=4.0, original_length=256, device=DEV)
        self.scale = d ** -0.5
        self.state_table = torch.zeros(requests, 1, dtype=torch.int32, device=DEV)

    def plan(self, requests, computed, new, decode_rows, tokens):
        out = layer.alloc_step_plan(len(requests), decode_rows, tokens, 0, DEV)
        at = torch.tensor(requests, device=DEV)
        layer.gdn_step_plan(computed, new, self.state_table[at], computed, num_decode_rows=decode_rows, state_block=64, kv_table=self.table[at],
                            kv_block=BLOCK, **out)
        return out, self.table[at]

    def enqueue(self, qkv, plan, table, computed, decode_rows, o, workspace, stream=None):
        """One step over a projection's rows qkv [T, (HQ + 2 HKV) d]."""
        q, k, v = (t.unflatten(1, (-1, self.d)) for t in qkv.split([HQ * self.d, HKV * self.d, HKV * self.d], 1))
        A.gdn_rotary(q, k, plan["token_position"], self.freq, attention_factor=self.factor, stream=stream)
        A.gdn_kv_cache_write(k, v, plan["token_kv_slot"], stream=stream, **self.cache)
        b = decode_rows
        if b:
            A.gdn_attention_decode(q[:b], o=o[:b], computed=computed[:b], kv_table=table[:b], kv_block=BLOCK, scale=self.scale, workspace=workspace,
                                   stream=stream, **self.cache)
        A.gdn_attention_prefill(q[b:], o=o[b:], cu_seqlens=plan["cu_seqlens"], start_pos=plan["start_pos"], kv_table=table[b:], kv_block=BLOCK,
                                scale=self.scale, stream=stream, **self.cache)

    def workspace(self, qkv, decode_rows):
        q = qkv[:, : HQ * self.d].unflatten(1, (HQ, self.d))[:decode_rows]
        return A.alloc_attention_workspace(q, self.cache["k_cache"], tokens_per_row=1, max_keys=self.table.shape[1] * BLOCK) if decode_rows else None

    def step(self, requests, computed, new, decode_rows, seed, check=True):
        tokens = sum(new)
        g = torch.Generator(device=DEV).manual_seed(seed)
        qkv = torch.randn(tokens, (HQ + 2 * HKV) * self.d, generator=g, device=DEV).to(self.dtype)
        given = qkv.clone()
        plan, table = self.plan(requests, C.i32(computed, DEV), C.i32(new, DEV), decode_rows, tokens)
        o = torch.full((tokens, HQ, self.d), 5.0, dtype=self.dtype, device=DEV)
        ws = self.workspace(qkv, decode_rows)
        if ws is not None:
            ws.fill_(0xff)
        self.enqueue(qkv, plan, table, C.i32(computed, DEV), decode_rows, o, ws)
        if check:
            self.compare(given, qkv, plan, table, computed, new, o)
        return o

    def compare(self, given, qkv, plan, table, computed, new, o):
        d, u = self.d, R.HALF_STEP[self.dtype]
        turned = (HQ + HKV) * d
        position = torch.cat([torch.arange(c, c + n, device=DEV) for c, n in zip(computed, new)])
        assert torch.equal(plan["token_position"].long(), position)
        x, y = (t[:, :turned].unflatten(1, (-1, d)) for t in (given, qkv))
        assert torch.equal(given[:, turned:], qkv[:, turned:])
        ref = R.rotary(x, position, self.freq, self.factor, False)
        # output rounding, and eight fp32 roundings of angle, cosine, sine and their products, each of at most |a| + |b|
        pair = x.double().abs()
        both = pair + pair.roll(d // 2, -1)
        R.check("rotary", y, ref, u * ref.abs() + 8 * 2.0 ** -24 * self.factor * both)
        slots = plan["token_kv_slot"]
        got = [torch.full((slots.shape[0], HKV, d), 7.0, dtype=self.dtype, device=DEV) for _ in "kv"]
        A.gdn_kv_cache_read(slots, k_out=got[0], v_out=got[1], **self.cache)
        fmt = {torch.float8_e4m3fn: "e4m3", torch.int8: "int8"}.get(self.cache["k_cache"].dtype)
        for part, back in zip(qkv[:, HQ * d:].unflatten(1, (2, HKV, d)).unbind(1), got):
            if fmt is None:
                assert torch.equal(back, part)
            else:
                code, scale = R.quantise(part, fmt)
                # code times scale: one fp32 product, rounded to the dtype
                assert torch.equal(back, (code.float() * scale[..., None]).to(self.dtype))
        q = qkv[:, : HQ * d].unflatten(1, (HQ, d))
        R.check("attention", o, *R.attention(q, self.cache, table, BLOCK, computed, new, self.scale))


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_steps(d, dtype, fmt):
    """Prompts that come in pieces while others decode, of one token and of many, across page borders."""
    e = Engine(5, 400, d, dtype, fmt)
    e.step([0, 1], [0, 0], [130, 1], 0, 1)
    e.step([0, 1, 2], [130, 1, 0], [1, 1, 200], 2, 2)
    e.step([1, 0, 2, 3, 4], [2, 131, 200, 0, 0], [1, 1, 150, 23, 24], 2, 3)
    e.step([3, 4, 2, 0, 1], [23, 24, 350, 132, 3], [1, 1, 1, 1, 1], 5, 4)


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("d,tokens", [(64, 1100), (128, 150), (128, 1100), (256, 300)])
def test_pieces_of_a_prompt_are_the_prompt(d, tokens, dtype, fmt):
    """Cut anywhere, shared with whatever: the same bits (1100 tokens: more and fewer rows of a workgroup)."""
    whole = Engine(1, tokens, d, dtype, fmt)
    g = torch.Generator(device=DEV).manual_seed(9)
    qkv = torch.randn(tokens, (HQ + 2 * HKV) * d, generator=g, device=DEV).to(dtype)

    def run(cuts):
        out = []
        for a, b in zip(cuts, cuts[1:]):
            part, computed, new = qkv[a:b].clone(), C.i32([a], DEV), C.i32([b - a], DEV)
            plan, table = whole.plan([0], computed, new, 0, b - a)
            o = torch.empty(b - a, HQ, d, dtype=dtype, device=DEV)
            whole.enqueue(part, plan, table, computed, 0, o, None)
            out.append(o)
        return torch.cat(out)

    want = run([0, tokens])
    for cuts in ([0, 1, 2, 70, tokens], [0, 63, 65, 129, tokens - 1, tokens], [0, tokens // 2, tokens]):
        for n in whole.cache:
            if whole.cache[n] is not None:
                whole.cache[n].view(torch.uint8).fill_(0x7f)
        assert torch.equal(run(cuts), want), cuts


@pytest.mark.parametrize("dtype,fmt", FORMATS)
def test_drafted_trees(dtype, fmt):
    """Tokens drafted as a tree behind each context: positions by depth, slots by number, what is not an ancestor unseen."""
    d, per, past = 128, 9, [40, 0, 311]
    e = Engine(3, 330, d, dtype, fmt)
    e.step([0, 2], [0, 0], [40, 311], 0, 1)
    parents = [[-1, 0, 0, 1, 1, 2, 2, 3, 7], [-1] * per, list(range(-1, per - 1))]
    mask, depth = A.tree_masks(parents, DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn(3 * per, h, d, generator=g, device=DEV).to(dtype) for h in (HQ, HKV, HKV))
    computed = C.i32(past, DEV)
    given = q.clone()
    position = computed.repeat_interleave(per) + depth
    A.gdn_rotary(q, k, position, e.freq, attention_factor=e.factor)
    ref = R.rotary(given, position, e.freq, e.factor, False)
    both = given.double().abs() + given.double().abs().roll(d // 2, -1)
    R.check("rotary", q, ref, R.HALF_STEP[dtype] * ref.abs() + 8 * 2.0 ** -24 * e.factor * both)
    number = (computed[:, None] + torch.arange(per, device=DEV)).long()
    slots = (torch.gather(e.table, 1, number // BLOCK).long() * BLOCK + number % BLOCK).flatten()
    A.gdn_kv_cache_write(k, v, slots, **e.cache)
    o = torch.empty_like(q)
    ws = A.alloc_attention_workspace(q, e.cache["k_cache"], tokens_per_row=per, max_keys=320)
    A.gdn_attention_decode(q, o=o, computed=computed, kv_table=e.table, kv_block=BLOCK, scale=e.scale, tokens_per_row=per, tree_mask=mask, max_keys=320,
                           workspace=ws, **e.cache)
    seen = [(mask.view(3, per, 1) >> torch.arange(per, device=DEV))[b] % 2 == 1 for b in range(3)]
    R.check("tree", o, *R.attention(q, e.cache, e.table, BLOCK, past, [per] * 3, e.scale, seen))
    # an accepted path is a chain: its tokens' outputs are those of a row that drafted just them
    chain = [0, 1, 3, 7, 8]
    rows = torch.tensor(chain, device=DEV)
    moved = slots[:len(chain)]
    A.gdn_kv_cache_write(k[rows].contiguous(), v[rows].contiguous(), moved, **e.cache)
    o2 = torch.empty(len(chain), HQ, d, dtype=dtype, device=DEV)
    A.gdn_attention_decode(q[rows].contiguous(), o=o2, computed=computed[:1], kv_table=e.table[:1], kv_block=BLOCK, scale=e.scale, tokens_per_row=len(chain),
                           max_keys=320, workspace=ws, **e.cache)
    R.check("accepted path", o2, *R.attention(q[rows], e.cache, e.table[:1], BLOCK, past[:1], [len(chain)], e.scale))


@pytest.mark.parametrize("dtype,fmt", [(BF16, None), (BF16, "int8"), (F32, "e4m3")])
def test_a_captured_step(dtype, fmt):
    """A whole step captured once and replayed with other lengths and inputs, eager work in between, is the eager step;
    and the same on a stream of the caller's."""
    d, decode_rows, tokens = 128, 2, 2 + 90
    e = Engine(4, 300, d, dtype, fmt)
    e.step([0, 1, 2, 3], [0, 0, 0, 0], [150, 60, 100, 30], 0, 1)
    computed, new = C.i32([150, 60, 100, 30], DEV), C.i32([1, 1, 70, 20], DEV)
    qkv = torch.zeros(tokens, (HQ + 2 * HKV) * d, dtype=dtype, device=DEV)
    o = torch.empty(tokens, HQ, d, dtype=dtype, device=DEV)
    ws = e.workspace(qkv, decode_rows)
    plan = layer.alloc_step_plan(4, decode_rows, tokens, 0, DEV)

    def step(stream=None):
        layer.gdn_step_plan(computed, new, e.state_table, computed, num_decode_rows=decode_rows, state_block=64, kv_table=e.table, kv_block=BLOCK,
                            stream=stream, **plan)
        e.enqueue(qkv, plan, e.table, computed, decode_rows, o, ws, stream)

    def fill(i):
        qkv.copy_(torch.randn(qkv.shape, generator=torch.Generator(device=DEV).manual_seed(20 + i), device=DEV))
        computed.copy_(C.i32([150 - 40 * i, 60 + i, 100 + 3 * i, 30 * (i % 2)], DEV))
        new.copy_(C.i32([1, 1, 70 - i, 20 - 5 * i], DEV))
        o.fill_(3.0)

    fill(0)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    for i in range(4):
        fill(i)
        step()
        want, cached = o.clone(), [t.view(torch.uint8).clone() for t in e.cache.values() if t is not None]
        assert torch.isfinite(want[: 2 + 90 - 6 * i]).all()
        fill(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), i
        assert all(torch.equal(a, t.view(torch.uint8)) for a, t in zip(cached, (t for t in e.cache.values() if t is not None))), i
        fill(i)
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, want), i


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("per,hq,hkv,d", [(1, 8, 2, 128), (2, 6, 2, 64), (9, 16, 1, 256), (40, 4, 1, 128)])
def test_bits_do_not_depend_on_max_keys(per, hq, hkv, d, dtype, fmt):
    """A launch and a workspace sized for more spans (beyond 16 and up to the most there are) give the same bits."""
    past, block = [3000, 700, 11], 16
    keys = [p + per for p in past]
    table, rows = C.pages(keys, block, DEV, 3)
    cache = C.filled_cache(rows, hkv, d, dtype, fmt, C.owned_rows(table, block, keys), DEV, 3)
    wide = torch.cat([table, torch.full((3, 6000), -1, dtype=torch.int32, device=DEV)], 1)
    q = C.queries(3 * per, hq, d, dtype, DEV, 8)
    out = []
    for most in (max(keys), 9000, 30000, 90000):
        ws = A.alloc_attention_workspace(q, cache["k_cache"], tokens_per_row=per, max_keys=most)
        if ws is not None:
            ws.fill_(0xff)
        o = torch.full_like(q, 5.0)
        A.gdn_attention_decode(q, o=o, computed=C.i32(past, DEV), kv_table=wide, kv_block=block, scale=d ** -0.5, tokens_per_row=per, max_keys=most,
                               workspace=ws, **cache)
        out.append(o)
    R.check("decode", out[0], *R.attention(q, cache, table, block, past, [per] * 3, d ** -0.5))
    assert all(torch.equal(o, out[0]) for o in out[1:])


def test_refused_tensors():
    """What the binding refuses before any call: types, shapes, devices, strides, halves of a pair."""
    e = Engine(1, 64, 64, BF16, "int8")
    q, k = (torch.zeros(4, h, 64, dtype=BF16, device=DEV) for h in (HQ, HKV))
    at, slots = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    no_scales = {n: t for n, t in e.cache.items() if "cache" in n}
    cu, past = C.i32([0, 4], DEV), C.i32([0], DEV)
    attend = dict(kv_table=e.table, kv_block=BLOCK, scale=1.0)

    def no(match, f, *a, **kw):
        with pytest.raises((ValueError, A.GdnError), match=match):
            f(*a, **kw)

    no("q or k", A.gdn_rotary, None, None, at, e.freq)
    no("positions", A.gdn_rotary, q, k, at.long(), e.freq)
    no("positions", A.gdn_rotary, q, k, at[:3], e.freq)
    no("inv_freq", A.gdn_rotary, q, k, at, e.freq[None])
    no("k is", A.gdn_rotary, q, k[..., :32], at, e.freq)
    no("k must", A.gdn_rotary, q, k.float(), at, e.freq)
    no("k must", A.gdn_rotary, q, k[:3], at, e.freq)
    no("k_out is given", A.gdn_rotary, q, None, at, e.freq, k_out=k)
    no("q_out is given", A.gdn_rotary, None, k, at, e.freq, q_out=q)
    no("q_out", A.gdn_rotary, q, k, at, e.freq, q_out=q[:, :4])
    no("dense rows", A.gdn_rotary, q.transpose(1, 2).contiguous().transpose(1, 2), k, at, e.freq)
    no("HIP device", A.gdn_rotary, q.cpu(), k, at, e.freq)
    no("is on cpu", A.gdn_rotary, q, k.cpu(), at, e.freq)
    no("rotary_dim", A.gdn_rotary, q, k, at, torch.ones(33, device=DEV))
    no("bfloat16 or float32", A.gdn_kv_cache_write, k.half(), k.half(), slots, **e.cache)
    no("k_scale and v_scale", A.gdn_kv_cache_write, k, k, slots, **no_scales)
    no("slots", A.gdn_kv_cache_write, k, k, slots.int(), **e.cache)
    no("v must", A.gdn_kv_cache_write, k, k[:, :1], slots, **e.cache)
    no("v_cache", A.gdn_kv_cache_write, k, k, slots, **dict(e.cache, v_cache=e.cache["v_cache"][1:]))
    no("k_cache must be", A.gdn_kv_cache_write, k, k, slots, **dict(no_scales, k_cache=no_scales["k_cache"].float()))
    no("has none", A.gdn_kv_cache_write, k, k, slots, **dict(e.cache, k_cache=torch.zeros(8, HKV, 64, dtype=BF16, device=DEV)))
    no("k_out", A.gdn_kv_cache_read, slots, k_out=k[:, :1], v_out=k, **e.cache)
    no("v_out must be contiguous", A.gdn_kv_cache_read, slots, k_out=k, v_out=torch.zeros(4, HKV, 128, dtype=BF16, device=DEV)[..., :64], **e.cache)
    no("o must", A.gdn_attention_prefill, q, o=q[:3], cu_seqlens=cu, start_pos=None, **attend, **e.cache)
    no("q must be", A.gdn_attention_prefill, q[..., :32], o=q, cu_seqlens=cu, start_pos=None, **attend, **e.cache)
    no("start_pos", A.gdn_attention_prefill, q, o=q.clone(), cu_seqlens=cu, start_pos=cu, **attend, **e.cache)
    no("kv_table", A.gdn_attention_prefill, q, o=q.clone(), cu_seqlens=cu, start_pos=None, **dict(attend, kv_table=e.table.long()), **e.cache)
    no("kv_table must have 2 dims", A.gdn_attention_prefill, q, o=q.clone(), cu_seqlens=cu, start_pos=None, **dict(attend, kv_table=e.table[0]), **e.cache)
    no("kv_block", A.gdn_attention_prefill, q, o=q.clone(), cu_seqlens=cu, start_pos=None, **dict(attend, kv_block=0), **e.cache)
    no("num_q_heads", A.gdn_attention_prefill, q[:, :3].contiguous(), o=q[:, :3].contiguous(), cu_seqlens=cu, start_pos=None, **attend, **e.cache)
    no("4 tokens, expected 1 rows of 3", A.gdn_attention_decode, q, o=q.clone(), computed=past, tokens_per_row=3, **attend, **e.cache)
    no("tree_mask", A.gdn_attention_decode, q, o=q.clone(), computed=past, tokens_per_row=4, tree_mask=at, **attend, **e.cache)
    no("scale", A.gdn_attention_decode, q, o=q.clone(), computed=past, tokens_per_row=4, **dict(attend, scale=math.inf), **e.cache)
    wide = torch.full((1, 1 << 12), -1, dtype=torch.int32, device=DEV)
    no("workspace", A.gdn_attention_decode, q, o=q.clone(), computed=past, tokens_per_row=4, max_keys=1 << 16, **dict(attend, kv_table=wide), **e.cache)
    # keys beyond what the table holds (72 here) cannot be there: they need no workspace
    A.gdn_kv_cache_write(k, k, torch.gather(e.table[0].long() * BLOCK, 0, slots) + torch.arange(4, device=DEV), **e.cache)
    o = [torch.ones_like(q) for _ in range(2)]
    for out, most in zip(o, (1 << 20, 0)):
        A.gdn_attention_decode(q, o=out, computed=past, tokens_per_row=4, max_keys=most, **attend, **e.cache)
    assert not o[0].any() and not o[1].any()
    assert not q.any() and not k.any()
