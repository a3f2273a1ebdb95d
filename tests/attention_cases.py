"""Inputs of the attention tests: shuffled pages, caches filled through the definition, everything that no
request owns poisoned."""
import itertools
import math

import torch

from gated_deltanet_rule_amd import attention
from tests import attention_reference as R

BF16, F32 = torch.bfloat16, torch.float32


def pages(keys, kv_block, device, seed, extra=3):
    """(table [n, width] int32 of shuffled pages, cache rows) for requests of so many keys; -1 behind a request's pages."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-k // kv_block) for k in keys]
    order = torch.randperm(sum(counts) + extra, generator=g).tolist()
    width, at, rows = max([1] + counts), 0, []
    for c in counts:
        rows.append(order[at: at + c] + [-1] * (width - c))
        at += c
    return torch.tensor(rows, dtype=torch.int32, device=device).view(len(keys), width), len(order) * kv_block


def owned_rows(table, kv_block, keys):
    own = []
    for i, n in enumerate(keys):
        p = torch.arange(n, device=table.device)
        own.append(table[i][p // kv_block].long() * kv_block + p % kv_block)
    return torch.cat(own) if own else torch.zeros(0, dtype=torch.int64, device=table.device)


def filled_cache(rows, heads, d, dtype, fmt, own, device, seed):
    """A cache with normal values in rows `own` and NaN (in integers: a NaN scale) everywhere else."""
    g = torch.Generator(device=device).manual_seed(seed)
    cache = attention.alloc_kv_cache(rows, heads, d, dtype, device, fmt)
    for n in "kv":
        c, s = cache[n + "_cache"], cache[n + "_scale"]
        x = torch.randn(own.shape[0], heads, d, generator=g, device=device).to(dtype)
        if fmt is None:
            c.fill_(math.nan)
            c[own] = x
            continue
        codes, scale = R.quantise(x, fmt)
        c.view(torch.uint8).fill_(0x7f)                       # e4m3's NaN
        c.view(torch.uint8)[own] = codes.to(torch.float32).to(c.dtype).view(torch.uint8)
        s.fill_(math.nan)
        s[own] = scale
    return cache


def packed(new, device):
    return torch.tensor(list(itertools.accumulate(new, initial=0)), dtype=torch.int32, device=device)


def i32(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def queries(tokens, heads, d, dtype, device, seed, pad=0):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.randn(tokens, heads * d + pad, generator=g, device=device).to(dtype)[:, : heads * d].unflatten(1, (heads, d))
