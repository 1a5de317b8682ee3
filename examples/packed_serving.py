"""Continuous batching with the packed operators: prompts of different lengths in
chunks, new requests joining while others decode, then one token per request.

A small layer of the kind that the operators serve: one projection gives the gate
z, the convolution's channels (x, B and C side by side) and the steps dt; the
convolution and the scan keep a window and a state per slot; a second projection
closes the layer. Run it on a GPU:

    python examples/packed_serving.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import state_space_model_03_gb300 as ssm  # noqa: E402


class Layer:
    """Random weights; headdim * heads inner channels, one group of B and C."""

    def __init__(self, dim=256, heads=8, headdim=64, dstate=128, width=4, slots=8, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.heads, self.headdim, self.dstate, self.inner = heads, headdim, dstate, heads * headdim
        self.channels = self.inner + 2 * dstate
        # rows of the projection in steps of 8 values: parts of it are 16-byte aligned
        self.w_in = (randn(self.inner + self.channels + heads, dim) / dim ** 0.5).to(dtype)
        self.w_out = (randn(dim, self.inner) / self.inner ** 0.5).to(dtype)
        self.conv_w, self.conv_b = randn(self.channels, width) * 0.5, randn(self.channels) * 0.1
        self.A = -(1 + 15 * torch.rand(heads, generator=g, device="cuda"))
        self.D = torch.ones(heads, device="cuda")
        self.dt_bias = torch.log(torch.expm1(0.001 + 0.099 * torch.rand(heads, generator=g, device="cuda")))
        self.conv_state = torch.zeros(slots, self.channels, width - 1, dtype=dtype, device="cuda")
        self.state = torch.zeros(slots, heads, headdim, dstate, device="cuda")

    def _parts(self, h):
        z, xbc, dt = (h @ self.w_in.t()).split([self.inner, self.channels, self.heads], 1)
        return z.unflatten(1, (self.heads, self.headdim)), xbc, dt

    def _heads(self, xbc):
        x, b, c = xbc.split([self.inner, self.dstate, self.dstate], 1)
        return x.unflatten(1, (self.heads, self.headdim)), b.unsqueeze(1), c.unsqueeze(1)

    def prompt(self, h, tables):
        """h (tokens, dim): the packed tokens of the batch that `tables` describes."""
        z, xbc, dt = self._parts(h)
        xbc = ssm.packed_conv1d_fn(xbc, self.conv_w, tables, bias=self.conv_b, conv_state=self.conv_state, activation="silu")
        x, b, c = self._heads(xbc)
        y = ssm.head_scan_fn(x, dt, self.A, b, c, tables, D=self.D, z=z, dt_bias=self.dt_bias, dt_softplus=True,
                             state=self.state)
        return y.flatten(1) @ self.w_out.t()

    def step(self, h, slots):
        """h (requests, dim): one token per request."""
        z, xbc, dt = self._parts(h)
        xbc = ssm.packed_conv1d_update(xbc, self.conv_state, self.conv_w, bias=self.conv_b, slots=slots, activation="silu")
        x, b, c = self._heads(xbc)
        y = ssm.head_state_update(self.state, x, dt, self.A, b, c, D=self.D, z=z, dt_bias=self.dt_bias, dt_softplus=True,
                                  slots=slots)
        return y.flatten(1) @ self.w_out.t()


def serve(layer, sequences, chunk=100, decode=5):
    """Runs the sequences as a server would: each joins when the one before it is half
    through, brings at most `chunk` prompt tokens a step and decodes its last `decode`
    tokens one by one. Returns their outputs."""
    i32 = dict(dtype=torch.int32, device="cuda")
    done, out = [0] * len(sequences), [[] for _ in sequences]
    slot = torch.full((len(sequences),), -1, **i32)
    free = torch.arange(layer.state.shape[0] - 1, -1, -1, **i32)
    joined = 1
    while any(d < len(s) for d, s in zip(done, sequences)):
        if joined < len(sequences) and 2 * done[joined - 1] >= len(sequences[joined - 1]):
            joined += 1
        # prompts first (and requests that are at their prompt's end wait one round)
        want = [max(0, min(chunk, len(sequences[r]) - decode - done[r])) for r in range(joined)]
        if sum(want):
            lengths, context = torch.tensor(want, **i32), torch.tensor(done[:joined], **i32)
            tokens = sum(want)
            block = ssm.head_scan_block(tokens, joined, layer.heads, layer.headdim)
            tables = ssm.request_tables(lengths, tokens, context=context, slots=slot[:joined], free_slots=free, block=block)
            slot[:joined] = tables.slots
            free = free[int(tables.counts[2]):]
            h = torch.cat([sequences[r][done[r]:done[r] + n] for r, n in enumerate(want)])
            for r, part in enumerate(layer.prompt(h, tables).split(want)):
                out[r].append(part)
                done[r] += want[r]
        ready = [r for r in range(joined) if not want[r] and done[r] < len(sequences[r])]
        if ready:
            h = torch.stack([sequences[r][done[r]] for r in ready])
            for r, row in zip(ready, layer.step(h, slot[ready])):
                out[r].append(row[None])
                done[r] += 1
    return [torch.cat(o) for o in out]


def main():
    g = torch.Generator(device="cuda").manual_seed(1)
    lengths = [310, 47, 129, 600, 6]
    sequences = [torch.randn(n, 256, generator=g, device="cuda").to(torch.bfloat16) for n in lengths]
    served = serve(Layer(), sequences)
    # all at once, each in one piece
    layer = Layer()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    whole = layer.prompt(torch.cat(sequences), ssm.request_tables(n, sum(lengths))).split(lengths)
    worst = max(float((a.float() - b.float()).norm() / b.float().norm()) for a, b in zip(served, whole))
    print(f"{len(lengths)} requests of {lengths} tokens, served in pieces against in one: relative difference {worst:.1e}")
    return worst


if __name__ == "__main__":
    # two bf16 roundings on either side, in other places
    sys.exit(0 if main() < 2e-2 else 1)
