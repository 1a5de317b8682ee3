"""fp64 CPU oracle of the gated recurrence and of the norm with the residual's addition.

TEST INFRASTRUCTURE ONLY: it shares no code with the CUDA library. Token by token
and row by row in numpy, from the definitions in include/ssfwd_layer.h:

    r = sigmoid(gate), i = sigmoid(input_gate) or 1
    L = -rate softplus(decay) r, a = exp(L), h = a h + sqrt(1 - a^2) i x

    s = x + residual (rounded to the residual's type), out = s / sqrt(mean(s^2) + eps) w

The gradients are the chain rule taken in reverse order of the tokens, through a and
sqrt(1 - a^2) one after the other. Pinned in tests/test_oracle_layer.py.
"""
from __future__ import annotations

import numpy as np


def f64(x):
    return None if x is None else np.ascontiguousarray(x.detach().to("cpu").double().numpy())


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def gates(x, gate, decay, input_gate, rate):
    """L, a, sqrt(1 - a^2) and the gated input, from fp64 arrays with the channels last."""
    L = -rate * softplus(decay) * sigmoid(gate)
    u = x if input_gate is None else sigmoid(input_gate) * x
    return L, np.exp(L), np.sqrt(-np.expm1(2 * L)), u


def gated_scan(x, gate, decay, input_gate=None, rate=8.0, initial_state=None):
    """(out, last_state) in fp64 of (batch, seqlen, dim) tensors."""
    x, gate, decay, input_gate, h = (f64(t) for t in (x, gate, decay, input_gate, initial_state))
    _, a, root, u = gates(x, gate, decay, input_gate, rate)
    h = np.zeros_like(x[:, 0]) if h is None else h.copy()
    out = np.empty_like(x)
    for t in range(x.shape[1]):
        h = a[:, t] * h + root[:, t] * u[:, t]
        out[:, t] = h
    return out, h


def gated_scan_bwd(dout, dlast, x, gate, decay, input_gate=None, rate=8.0, initial_state=None):
    """Gradients of sum(dout out) + sum(dlast last_state), by input name."""
    first = f64(initial_state)
    out, _ = gated_scan(x, gate, decay, input_gate, rate, initial_state)
    x, gate, decay, input_gate, dout, dlast = (f64(t) for t in (x, gate, decay, input_gate, dout, dlast))
    L, a, root, u = gates(x, gate, decay, input_gate, rate)
    r = sigmoid(gate)
    i = np.ones_like(x) if input_gate is None else sigmoid(input_gate)
    back = np.zeros_like(x[:, 0]) if dlast is None else dlast.copy()
    first = np.zeros_like(x[:, 0]) if first is None else first
    g = np.empty_like(x)
    for t in reversed(range(x.shape[1])):
        g[:, t] = dout[:, t] + back
        back = a[:, t] * g[:, t]
    before = np.concatenate([first[:, None], out[:, :-1]], 1)
    # h = a before + root u, root = sqrt(1 - a^2)
    with np.errstate(divide="ignore", invalid="ignore"):
        dL = g * (a * before) + np.where(root > 0, -g * u * a * a / root, 0.0)
    dgate = dL * L * (1 - r)
    # where L is 0, so is what it contributes: its gradient is finite as L goes to 0
    dgate = np.where(L == 0, 0.0, dgate)
    with np.errstate(divide="ignore", invalid="ignore"):
        ddecay = np.where(softplus(decay) > 0, (dL * L).sum((0, 1)) * sigmoid(decay) / softplus(decay), 0.0)
    return {"x": g * root * i, "gate": dgate, "decay": ddecay,
            "input_gate": None if input_gate is None else g * root * x * i * (1 - i), "initial_state": back}


def packed_gated_scan(x, gate, decay, lengths, input_gate=None, rate=8.0, state=None, slots=None, context=None):
    """(out, state) in fp64 of packed requests; the state given is not changed."""
    n = [int(v) for v in lengths]
    slots = list(range(len(n))) if slots is None else [int(v) for v in slots]
    context = [0] * len(n) if context is None else [int(v) for v in context]
    new = None if state is None else f64(state).copy()
    out = np.zeros(tuple(x.shape))
    at = 0
    for length, slot, had in zip(n, slots, context):
        if length == 0:
            continue
        part = slice(at, at + length)
        kept = new is not None and 0 <= slot < new.shape[0]
        import torch
        start = torch.from_numpy(new[slot].copy())[None] if kept and had > 0 else None
        o, last = gated_scan(x[None, part], gate[None, part], decay, None if input_gate is None else input_gate[None, part], rate, start)
        out[part] = o[0]
        if kept:
            new[slot] = last[0]
        at += length
    return out, new


def residual_sum(x, residual):
    """s as it is kept, in fp64."""
    if residual is None:
        return f64(x)
    return f64((x.detach().double() + residual.detach().double()).to(residual.dtype))


def rms_norm(x, weight, residual=None, eps=1e-5):
    """(out, s) in fp64."""
    s, w = residual_sum(x, residual), f64(weight)
    return s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * w, s


def rms_norm_bwd(dout, dsum, x, weight, residual=None, eps=1e-5):
    """Gradients of sum(dout out) + sum(dsum s): of s (x's and the residual's), and of the weight."""
    s, w, d = residual_sum(x, residual), f64(weight), f64(dout)
    rms = np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    ds = d * w / rms - s * (d * w * s).mean(-1, keepdims=True) / rms**3
    if dsum is not None:
        ds = ds + f64(dsum)
    return ds, (d * s / rms).reshape(-1, s.shape[-1]).sum(0)


def scales(v, group, power_of_two):
    """(..., groups) scales of fp64 values v: the group's largest over 448, 2^-126 at least."""
    dim = v.shape[-1]
    group = group or dim
    most = np.stack([np.abs(v[..., k:k + group]).max(-1) for k in range(0, dim, group)], -1)
    scale = np.maximum(most / 448.0, 2.0**-126)
    return np.exp2(np.ceil(np.log2(scale))) if power_of_two else scale
