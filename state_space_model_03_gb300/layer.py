"""The operators of a gated recurrent layer beside its projections: Python binding
of include/ssfwd_layer.h.

A layer adds its input to the residual stream and norms the sum (``rms_norm_fn``,
or ``rms_norm_quant_fn`` for a projection in 8 bits), projects it to x and two
gates, and runs a linear recurrence per channel whose decay and input the gates
set: ``gated_scan_fn`` on dense batches, ``packed_gated_scan_fn`` on packed
requests (``request_tables``) and ``gated_state_update`` on one token per request.
Rows have their channels last, as projections leave them.

As in packed.py this is argument marshalling only, on the current stream, and there
is no CPU fallback. ``gated_scan_fn`` and ``rms_norm_fn`` are differentiable (once);
the others are forward only and refuse inputs that require a gradient. A training step
is captured into a CUDA graph as with any of torch's operators: with no eager graph of
the same leaves alive, whose gradients torch accumulates on that graph's stream.
"""
from __future__ import annotations

import torch

from . import api
from .packed import _cuda, _load_extension

_bind_module = None


def _load_bind():
    global _bind_module
    names = ("ss_gated_scan", "ss_gated_scan_bwd", "ss_gated_scan_bwd_workspace_size", "ss_packed_gated_scan",
             "ss_gated_state_update", "ss_rms_norm", "ss_rms_norm_bwd", "ss_rms_norm_bwd_workspace_size",
             "ss_rms_norm_quant", "ss_gated_scan_workspace_size", "ss_packed_gated_scan_workspace_size", "ss_status_string")
    _bind_module = _load_extension("_layer_bind", names)
    return _bind_module


def _bind():
    return _bind_module or _load_bind()


def gated_scan_fn(x, gate, decay, input_gate=None, rate=8.0, initial_state=None, return_last_state=False):
    """Gated linear recurrence on CUDA tensors, differentiable in every tensor.

    x, gate, input_gate: (batch, seqlen, dim), one dtype (fp32/fp16/bf16), any
    strides (a last stride other than 1 is copied); decay: (dim,) fp32; rate: a
    positive number; initial_state: (batch, dim) fp32 (None: zero). Per channel
    and token, with r = sigmoid(gate), i = sigmoid(input_gate) (1 without it):
    a = exp(-rate softplus(decay) r), h = a h + sqrt(1 - a^2) i x, out = h; h is
    held in fp32. The factor sqrt(1 - a^2) is every token's, the first one's too. Returns
    out (x's dtype), or (out, last_state) with last_state (batch, dim) fp32. At least one
    token.
    """
    _cuda(x, "gated_scan_fn")
    return _bind().gated_scan(x, gate, decay, input_gate, rate, initial_state, return_last_state)


def packed_gated_scan_fn(x, gate, decay, tables, input_gate=None, rate=8.0, state=None):
    """``gated_scan_fn``'s recurrence over packed requests.

    x, gate, input_gate: (tokens, dim), rows of any stride; tables:
    ``request_tables`` of the batch (of any block); state: (slots, dim) fp32, read
    where context is above 0 and replaced in place. Returns out (tokens, dim), zeros
    past the last token. Forward only.
    """
    _cuda(x, "packed_gated_scan_fn")
    return _bind().packed_gated_scan(x, gate, decay, tables._plan, input_gate, rate, state)


def gated_state_update(state, x, gate, decay, input_gate=None, rate=8.0, slots=None):
    """One token per request: x, gate, input_gate (requests, dim); row r goes with
    state[slots[r]] (slots None: r), updated in place; a row with slot -1 gets zeros.
    Two rows must not share a slot. Up to 65535 requests. Returns out (requests, dim).
    Forward only.
    """
    _cuda(x, "gated_state_update")
    return _bind().gated_state_update(state, x, gate, decay, input_gate, rate, slots)


def rms_norm_fn(x, weight, residual=None, eps=1e-5, prenorm=False, residual_in_fp32=False):
    """Root-mean-square norm with the residual's addition, differentiable.

    x: (..., dim) fp32/fp16/bf16; weight: (dim,) fp32 or x's dtype; residual: x's
    shape, x's dtype or fp32. s = x + residual, rounded to the residual's dtype (x
    itself without one); out = s / sqrt(mean(s^2) + eps) * weight, in x's dtype: the
    norm takes s as it is kept. Returns out, or with prenorm (out, s). residual_in_fp32:
    s is kept in fp32 (a residual in x's dtype, or none, starts such a stream). dim up
    to 32768.
    """
    _cuda(x, "rms_norm_fn")
    if residual is not None and residual_in_fp32:
        residual = residual.float()
    out, total = _bind().rms_norm(x, weight, residual, eps, prenorm)
    return (out, _kept(x, total, residual_in_fp32)) if prenorm else out


def _kept(x, total, in_fp32):
    # without a residual the stream starts with x
    return total if total is not None else x.float() if in_fp32 else x


def rms_norm_quant_fn(x, weight, residual=None, eps=1e-5, prenorm=False, residual_in_fp32=False, group_size=None,
                      scale_dtype=torch.float32):
    """``rms_norm_fn`` with an output in 8 bits: (out, scale), or with prenorm (out,
    scale, s). out: (..., dim) float8_e4m3fn; scale: (..., groups) with a scale for the
    row (group_size None) or for each group_size (32, 64 or 128) of its channels, so that
    the norm is about out * scale. scale_dtype float32: the group's largest value over
    448 (2^-126 at least); float8_e8m0fnu: the least power of two not below that. A group
    with a NaN or an infinity is NaN, scale and all. Scales lie row by row: a product that
    wants them in tiles needs them reordered. Forward only.
    """
    _cuda(x, "rms_norm_quant_fn")
    if scale_dtype not in (torch.float32, torch.float8_e8m0fnu):
        raise TypeError("scale_dtype must be float32 or float8_e8m0fnu")
    if residual is not None and residual_in_fp32:
        residual = residual.float()
    out, scale, total = _bind().rms_norm_quant(x, weight, residual, eps, prenorm, 0 if group_size is None else group_size,
                                               scale_dtype == torch.float8_e8m0fnu)
    return (out, scale, _kept(x, total, residual_in_fp32)) if prenorm else (out, scale)
