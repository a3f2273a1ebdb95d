"""Keys and values into a paged cache and back, bit for bit against the definition of the codes."""
import math

import pytest
import torch

from gated_deltanet_rule_amd import attention as A
from tests import attention_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def codes(c):
    return c.view(torch.uint8)


def scales(cache):
    return dict(k_scale=cache["k_scale"], v_scale=cache["v_scale"])


def tensors(cache):
    return cache["k_cache"], cache["v_cache"]


def same(a, b):
    return torch.equal(a.nan_to_num(12345.0), b.nan_to_num(12345.0)) and torch.equal(a.isnan(), b.isnan())


def run(x, fmt, rows, slots, pad=0):
    """Writes x = (k, v) and compares all of the cache, then reads it back."""
    tokens, heads, d = x[0].shape
    dtype = x[0].dtype
    cache = A.alloc_kv_cache(rows, heads, d, dtype, DEV, fmt)
    for t in cache.values():
        if t is not None:
            t.view(torch.uint8).fill_(0x35)
    before = {n: None if t is None else t.clone() for n, t in cache.items()}
    wide = torch.cat([x[0].flatten(1), x[1].flatten(1), torch.ones(tokens, pad, dtype=dtype, device=DEV)], 1)
    k, v = wide[:, : heads * d].unflatten(1, (heads, d)), wide[:, heads * d: 2 * heads * d].unflatten(1, (heads, d))
    A.gdn_kv_cache_write(k, v, slots, *tensors(cache), **scales(cache))
    live = (slots >= 0) & (slots < rows)
    out = [torch.full((tokens, heads, d), 9.0, dtype=dtype, device=DEV) for _ in range(2)]
    A.gdn_kv_cache_read(slots, *tensors(cache), *out, **scales(cache))
    for name, values, got in zip("kv", x, out):
        want, kept = before[name + "_cache"], before[name + "_scale"]
        if fmt is None:
            want[slots[live]] = values[live]
            back = values
        else:
            code, scale = R.quantise(values, fmt)
            codes(want)[slots[live]] = codes(code.to(F32).to(want.dtype))[live]
            kept[slots[live]] = scale[live]
            assert same(cache[name + "_scale"], kept)
            back = (code.to(F32) * scale[..., None]).to(dtype)
        assert torch.equal(codes(cache[name + "_cache"]), codes(want))
        assert same(got[live], back[live]) and (got[~live] == 0).all()


@pytest.mark.parametrize("fmt", [None, "e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,heads,d,pad", [(1, 1, 8, 0), (3, 8, 128, 8), (77, 2, 256, 0), (5, 7, 64, 64), (40, 3, 80, 8), (2, 2, 512, 0), (9, 1, 136, 16)])
def test_write_and_read(tokens, heads, d, pad, dtype, fmt):
    g = torch.Generator(device=DEV).manual_seed(tokens + d)
    x = [(torch.randn(tokens, heads, d, generator=g, device=DEV) * 10.0 ** i).to(dtype) for i in range(2)]
    rows = tokens + 5
    slots = torch.randperm(rows, generator=g, device=DEV)[:tokens]
    if tokens > 4:
        slots[1], slots[3], slots[4] = -1, rows, 1 << 40
    run(x, fmt, rows, slots, pad)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_value_between_codes(fmt):
    """Heads that hold every code, every midpoint of two neighbours (ties), and the numbers next to those."""
    if fmt == "int8":
        code = torch.arange(-127, 128, dtype=torch.float64)
    else:
        code = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(F32).double()
        code = code[torch.isfinite(code)].sort().values.unique()
    mid = (code[1:] + code[:-1]) / 2
    v = torch.cat([code, mid]).to(F32)
    v = torch.cat([v, torch.nextafter(v, torch.tensor(1e9)), torch.nextafter(v, torch.tensor(-1e9))]).clamp(-R.TOP[fmt], R.TOP[fmt])
    v = torch.cat([v, v.new_zeros(-v.shape[0] % 127)]).view(-1, 127)
    x = torch.cat([v, v.new_full((v.shape[0], 1), R.TOP[fmt])], 1).view(-1, 1, 128).to(DEV)
    for power in (0, -60, 40):        # the scale is a power of two: quotients are the values above
        run([x * 2.0 ** power, -x * 2.0 ** power], fmt, x.shape[0], torch.arange(x.shape[0], device=DEV))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_special_rows(fmt, dtype):
    """Zeros, the smallest and largest numbers, infinities and NaN: these make a head unreadable, and no other."""
    x = torch.randn(12, 2, 64, device=DEV).to(dtype)
    x[0] = 0
    x[1, 0] = 0
    x[1, 0, 5] = 2.0 ** -120
    x[2] *= torch.finfo(dtype).max / 16
    x[3, 0, 7] = math.inf
    x[4, 1, 63] = -math.inf
    x[5, 0, 0] = math.nan
    x[6] = math.nan
    x[7, 1, 3], x[7, 1, 60] = math.inf, math.nan
    x[8] *= 2.0 ** -110
    run([x, x.flip(0).contiguous()], fmt, 12, torch.arange(12, device=DEV))


def test_no_tokens_and_no_rows():
    cache = A.alloc_kv_cache(0, 2, 64, BF16, DEV, "int8")
    k, slots = torch.randn(3, 2, 64, device=DEV).to(BF16), torch.tensor([0, -1, 5], device=DEV)
    A.gdn_kv_cache_write(k, k, slots, *tensors(cache), **scales(cache))
    out = torch.ones_like(k)
    A.gdn_kv_cache_read(slots, *tensors(cache), out, out.clone(), **scales(cache))
    assert (out == 0).all()
    A.gdn_kv_cache_write(k[:0], k[:0], slots[:0], *tensors(cache), **scales(cache))


def test_offsets_past_32_bits():
    """Rows far behind 2^32 bytes of a cache."""
    rows = (1 << 32) // (8 * 512) + 1000
    cache = A.alloc_kv_cache(rows, 8, 512, BF16, DEV, "e4m3")
    k = torch.randn(4, 8, 512, device=DEV).to(BF16)
    slots = torch.tensor([rows - 1, 5, rows - 900, rows // 2], device=DEV)
    A.gdn_kv_cache_write(k, k, slots, *tensors(cache), **scales(cache))
    out = [torch.empty_like(k) for _ in range(2)]
    A.gdn_kv_cache_read(slots, *tensors(cache), *out, **scales(cache))
    code, scale = R.quantise(k, "e4m3")
    back = (code.to(F32) * scale[..., None]).to(BF16)
    assert torch.equal(out[0], back) and torch.equal(out[1], back)
