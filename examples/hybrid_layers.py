"""Two recurrent layers of a serving step, run from the requests' lengths and block tables
alone: a gated delta rule layer and a selective state space layer, with their step plan,
short convolutions, norms and caches.

    python examples/hybrid_layers.py

serves the same requests twice, each prompt at once and in pieces beside decode rows, and
shows that the hidden states of every token come out bitwise the same.  (The projections
are computed row by row in fp64, so that they do not depend on the batch either.)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_deltanet_rule_amd import binding, layer  # noqa: E402

DIM, H_K, H_V, D, WIDTH, BLOCK = 256, 2, 4, 64, 4, 128
CHANNELS = [H_K * D, H_K * D, H_V * D]
BF16, F32 = torch.bfloat16, torch.float32


def project(x, weight):
    """x W in fp64, each row by itself, rounded once."""
    return (x.double()[:, :, None] * weight.double()[None]).sum(1).to(x.dtype)


class Caches:
    """State and convolution slots of both layers, and each request's slots: one for every
    BLOCK tokens, one for where it stands."""

    def __init__(self, requests, max_tokens, device):
        self.width = max_tokens // BLOCK + 1
        slots = requests * (self.width + 1)
        self.state = [torch.zeros(slots, H_V, D, D, device=device) for _ in range(2)]
        self.conv = [torch.zeros(slots, WIDTH - 1, sum(CHANNELS), dtype=BF16, device=device) for _ in range(2)]
        self.table = torch.arange(requests * self.width, dtype=torch.int32, device=device).view(requests, self.width)
        self.run = torch.arange(requests * self.width, slots, dtype=torch.int32, device=device)


class Layers:
    def __init__(self, device, seed=0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g) * std).to(device)

        c = sum(CHANNELS)
        self.w = [dict(inp=normal(DIM, c + H_V * D, std=DIM ** -0.5).to(BF16), gates=normal(DIM, 2 * H_V, std=DIM ** -0.5).to(BF16),
                       conv=normal(c, WIDTH, std=0.5), bias=normal(c, std=0.1), norm=1.0 + normal(D, std=0.1),
                       out=normal(H_V * D, DIM, std=(H_V * D) ** -0.5).to(BF16), pre=1.0 + normal(DIM, std=0.1)) for _ in range(2)]
        self.A = -(1.0 + 3.0 * torch.rand(H_V, generator=g)).to(device)
        self.dt_bias, self.skip = normal(H_V) - 3.0, normal(H_V)

    def step(self, hidden, computed, new, decode_rows, caches):
        """One step: rows of `decode_rows` requests with one token each, then the prompts' tokens;
        hidden [tokens, DIM] in, the layers' residual stream out."""
        dev, tokens, requests = hidden.device, hidden.shape[0], len(computed)
        i32 = dict(dtype=torch.int32, device=dev)
        prompts, B = requests - decode_rows, decode_rows
        plan = layer.alloc_step_plan(requests, B, tokens, tokens // BLOCK + prompts, dev, kv=False)
        rows = torch.tensor([*range(requests)], **i32).long() if caches.table.shape[0] != requests else slice(None)
        layer.gdn_step_plan(torch.tensor(computed, **i32), torch.tensor(new, **i32), caches.table[rows].contiguous(), caches.run[rows].contiguous(),
                            num_decode_rows=B, state_block=BLOCK, **plan)
        exports = dict(start_pos=plan["start_pos"], export_grid=BLOCK, export_offsets=plan["export_offsets"], export_slots=plan["export_slots"])
        slots = plan["init_slot"], plan["final_slot"]
        residual = hidden.float()
        x = torch.empty_like(hidden)
        layer.gdn_residual_norm(torch.zeros_like(hidden), residual, residual, x, pre_weight=self.w[0]["pre"])
        for n, w in enumerate(self.w):
            wide, gates = project(x, w["inp"]), project(x.float(), w["gates"])
            outs = [torch.empty(tokens, c, dtype=BF16, device=dev) for c in CHANNELS]
            l2 = (D, D, 0) if n == 0 else (0, 0, 0)
            xc, z = wide[:, : sum(CHANNELS)], wide[:, sum(CHANNELS):].unflatten(1, (H_V, D))
            if B:
                layer.gdn_causal_conv_decode(xc[:B], w["conv"], w["bias"], [o[:B] for o in outs], caches.conv[n], plan["slot_in"], plan["slot_out"],
                                             l2_dims=l2)
            layer.gdn_causal_conv_prefill(xc[B:], w["conv"], w["bias"], [o[B:] for o in outs], caches.conv[n], plan["cu_seqlens"], *slots, l2_dims=l2,
                                          **exports)
            first, second, third = outs[0].view(tokens, H_K, D), outs[1].view(tokens, H_K, D), outs[2].view(tokens, H_V, D)
            y = torch.empty_like(third)
            if n == 0:                        # the gated delta rule: q, k, v
                decay = -torch.nn.functional.softplus(gates[:, :H_V]).contiguous()
                beta = torch.sigmoid(gates[:, H_V:]).contiguous()
                binding.gdn_mixed_step(first, second, third, decay, beta, y, caches.state[0], plan["slot_in"], plan["slot_out"], plan["cu_seqlens"], *slots,
                                       scale=D ** -0.5, workspace=binding.alloc_workspace(H_V, BF16, prompts, tokens - B, dev), **exports)
            else:                             # the state space scan: c, b, x
                dt = gates[:, :H_V].contiguous()
                par = dict(dt_bias=self.dt_bias, D=self.skip)
                if B:
                    layer.gdn_ssm_recurrent_decode(first[:B], second[:B], third[:B], dt[:B], self.A, y[:B], caches.state[1], plan["slot_in"],
                                                   plan["slot_out"], **par)
                layer.gdn_ssm_chunk_prefill(first[B:], second[B:], third[B:], dt[B:], self.A, y[B:], plan["cu_seqlens"], caches.state[1], *slots, **par,
                                            workspace=layer.alloc_ssm_workspace(first[B:], third[B:], prompts), **exports)
            normed = torch.empty_like(y)
            layer.gdn_gated_norm(y, z, w["norm"], normed, gate_first=n == 1)
            out = project(normed.flatten(1), w["out"])
            layer.gdn_residual_norm(out, residual, residual, x if n == 0 else None, pre_weight=self.w[1]["pre"] if n == 0 else None)
        return residual


def serve(device, split, prompts=(200, 70, 333), generated=3):
    """Hidden states of every token of every request; with `split`, prompts come in BLOCK-aligned
    pieces while earlier requests already decode."""
    g = torch.Generator().manual_seed(1)
    streams = [torch.randn(p + generated, DIM, generator=g).to(BF16).to(device) for p in prompts]
    layers, caches = Layers(device), Caches(len(prompts), max(prompts) + generated, device)
    done, states = [0] * len(prompts), [[] for _ in prompts]
    while any(d < len(s) for d, s in zip(done, streams)):
        # a token for the requests that are past their prompt, then the prompts (or a piece of them)
        new = [min(1, len(s) - d) if d >= p else (min(BLOCK - d % BLOCK, p - d) if split else p - d) for d, s, p in zip(done, streams, prompts)]
        order = sorted(range(len(prompts)), key=lambda r: (done[r] < prompts[r], r))
        decode = sum(done[r] >= prompts[r] for r in order)
        view = Caches.__new__(Caches)
        view.state, view.conv, view.table, view.run = caches.state, caches.conv, caches.table[order].contiguous(), caches.run[order].contiguous()
        # a request that has ended keeps a padding row
        rows = torch.cat([streams[r][done[r]: done[r] + new[r]] if new[r] else streams[r][:1] for r in order])
        out = layers.step(rows, [done[r] for r in order], [new[r] for r in order], decode, view)
        at = 0
        for r in order:
            n = max(new[r], 1)
            if new[r]:
                states[r].append(out[at: at + n])
            at += n
            done[r] += new[r]
    return [torch.cat(s) for s in states]


def main():
    if not torch.cuda.is_available():
        raise SystemExit("needs a GPU")
    device = torch.device("cuda", 0)
    whole, pieces = serve(device, split=False), serve(device, split=True)
    for r, (a, b) in enumerate(zip(whole, pieces)):
        same = torch.equal(a, b)
        print("request %d: %d tokens, largest hidden value %.3f, %s" % (r, a.shape[0], a.abs().max().item(), "the same bits" if same else "DIFFERENT"))
        if not same or not torch.isfinite(a).all():
            raise SystemExit(1)


if __name__ == "__main__":
    main()
