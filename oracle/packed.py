"""Oracle of the packed operators, token by token in fp64 numpy.

Written from the formulas in include/ssfwd_packed.h; shares no code with the
CUDA path. Inputs are torch tensors (any device), read as their stored values.
"""
from __future__ import annotations

import numpy as np


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _ints(t):
    return None if t is None else [int(v) for v in t.cpu()]


def silu(v):
    return v / (1.0 + np.exp(-v))


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def request_tables(lengths, tokens, context=None, slots=None, free_slots=None, block=512):
    """dict of offsets, token_request, token_position, blocks, slots, carried, counts."""
    lengths, context, slots, free = _ints(lengths), _ints(context), _ints(slots), _ints(free_slots) or []
    errors, offsets, taken, got = 0, [0], 0, []
    req, pos, blocks = [-1] * tokens, [0] * tokens, []
    for r, n in enumerate(lengths):
        if n < 0:
            errors, n = errors | 2, 0
        if offsets[-1] + n > tokens:
            errors, n = errors | 1, tokens - offsets[-1]
        for i in range(n):
            req[offsets[-1] + i] = r
            pos[offsets[-1] + i] = (context[r] if context else 0) + i
        blocks += [[r, offsets[-1] + k, min(block, n - k), k // block] for k in range(0, n, block)]
        offsets.append(offsets[-1] + n)
        slot = r if slots is None else slots[r]
        if slot < 0:
            if taken < len(free):
                slot, taken = free[taken], taken + 1
            else:
                slot, errors = -1, errors | 4
        got.append(slot)
    carried = [i for i, b in enumerate(blocks) if b[1] + b[2] < offsets[b[0] + 1]]
    rows = blocks + [[-1, 0, 0, 0]] * (tokens // block + min(len(lengths), tokens) - len(blocks))
    return {"offsets": np.array(offsets), "token_request": np.array(req, dtype=int), "token_position": np.array(pos, dtype=int),
            "blocks": np.array(rows, dtype=int).reshape(-1, 4), "slots": np.array(got),
            "carried": np.array(carried + [-1] * (tokens // block - len(carried)), dtype=int),
            "counts": np.array([offsets[-1], len(blocks), taken, errors])}


def _runs(lengths, slots, context):
    """(first, end, slot, goes on) of every request that has tokens."""
    at = 0
    for r, n in enumerate(lengths):
        if n > 0:
            yield at, at + n, (r if slots is None else slots[r]), bool(context and context[r] > 0)
        at += n


def packed_conv1d(x, weight, lengths, bias=None, conv_state=None, slots=None, context=None, silu_act=False):
    """(out, conv_state after)."""
    x, w, b, st = _np(x), _np(weight), _np(bias), _np(conv_state)
    st = None if st is None else st.copy()
    h = w.shape[1] - 1
    out = np.zeros_like(x)
    for f, e, slot, on in _runs(_ints(lengths), _ints(slots), _ints(context)):
        keep = st is not None and slot >= 0
        old = st[slot].T if keep and on else np.zeros((h, x.shape[1]))
        line = np.concatenate([old, x[f:e]])
        for t in range(e - f):
            v = (0 if b is None else b) + (line[t:t + h + 1] * w.T).sum(0)
            out[f + t] = silu(v) if silu_act else v
        if keep:
            st[slot] = line[len(line) - h:].T
    return out, st


def head_scan(x, dt, A, B, C, lengths, D=None, z=None, dt_bias=None, dt_softplus=False, state=None, slots=None, context=None):
    """(out, state after)."""
    x, dt, A, B, C, D, z, bias, st = (_np(t) for t in (x, dt, A, B, C, D, z, dt_bias, state))
    rep = x.shape[1] // B.shape[1]
    dt = dt + (0 if bias is None else bias)
    if dt_softplus:
        dt = softplus(dt)
    st = None if st is None else st.copy()
    out = np.zeros_like(x)
    for f, e, slot, on in _runs(_ints(lengths), _ints(slots), _ints(context)):
        keep = st is not None and slot >= 0
        s = st[slot].copy() if keep and on else np.zeros(x.shape[1:] + B.shape[2:])
        for t in range(f, e):
            b, c = np.repeat(B[t], rep, 0), np.repeat(C[t], rep, 0)
            s = np.exp(dt[t] * A)[:, None, None] * s + (dt[t][:, None] * x[t])[:, :, None] * b[:, None, :]
            out[t] = np.einsum("hpn,hn->hp", s, c)
            if D is not None:
                out[t] += D[:, None] * x[t]
        if keep:
            st[slot] = s
    if z is not None:
        out = out * silu(z)
    return out, st
