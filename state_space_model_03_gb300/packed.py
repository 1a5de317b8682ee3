"""Packed requests: Python binding of include/ssfwd_packed.h.

A batch of requests of different lengths, their tokens one after another in
(tokens, channels) tensors without padding, each request with a slot in a cache
of states. ``request_tables`` builds the batch's tables on the GPU;
``packed_conv1d_fn`` and ``head_scan_fn`` run prompts, ``packed_conv1d_update``
and ``head_state_update`` one token per request.

As in api.py this is argument marshalling only, on the current stream, and there
is no CPU fallback. The checks and the call are in csrc/packed_bind.cpp. The
operators are forward only: inputs that require a gradient or carry a tangent are
refused, and a cache that is updated in place counts as changed for autograd.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import api
from .api import _DT, _activation

_BIND_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "_packed_bind.so")
_bind_module = None


def _load_bind():
    global _bind_module
    lib = api.load_library()
    if not os.path.exists(_BIND_PATH):
        raise RuntimeError(f"_packed_bind.so is not built ({_BIND_PATH}); build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    loader = importlib.machinery.ExtensionFileLoader("_packed_bind", _BIND_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_packed_bind", loader))
    loader.exec_module(module)
    names = ("ss_request_tables", "ss_packed_conv1d", "ss_packed_conv1d_update", "ss_head_scan",
             "ss_head_scan_workspace_size", "ss_head_state_update", "ss_status_string")
    module.init(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names), api.SSError)
    lib.ss_head_scan_block.argtypes = [ctypes.c_int64] * 4 + [ctypes.c_int32] * 2
    lib.ss_head_scan_block.restype = ctypes.c_int64
    _bind_module = module
    return module


def _bind():
    return _bind_module or _load_bind()


def _cuda(t, what):
    if not t.is_cuda:
        raise RuntimeError(f"{what} needs CUDA tensors (there is no CPU path)")


class RequestTables:
    """Tables of one packed batch (int32, on the GPU), as ``request_tables``
    makes them: ``offsets`` (requests + 1), ``token_request`` and
    ``token_position`` (tokens), ``blocks`` (max_blocks, 4), ``slots``
    (requests), ``counts`` (4: tokens, blocks, slots taken, errors) and
    ``carried`` (rows of blocks that another block of their request follows)."""

    __slots__ = ("tokens", "block", "max_blocks", "offsets", "token_request", "token_position", "blocks", "slots",
                 "counts", "context", "carried", "_plan")

    def check(self):
        """Raise if the lengths did not fit the batch (reads counts: synchronises)."""
        errors = int(self.counts[3])
        said = [w for bit, w in ((1, "the lengths exceed num_tokens"), (2, "a length is negative"),
                                 (4, "free_slots has too few slots")) if errors & bit]
        if said:
            raise ValueError("request_tables: " + "; ".join(said))
        return self


def request_tables(lengths, num_tokens, context=None, slots=None, free_slots=None, block=512):
    """Tables of a packed batch from its request lengths, built on the GPU.

    lengths: (requests,) int32 new tokens per request, 0 allowed, at least one
    request. num_tokens: rows of the packed tensors; rows past the last
    request's are padding. context: (requests,) int32 tokens that each request
    has had before; where it is above 0 the operators go on from the request's
    slot (None: all start from zero). slots: (requests,) int32 slot of each
    request, -1 for one that has none yet and takes the next of free_slots
    (None: request r has slot r); no two requests with tokens may share one.
    block: tokens per unit of work of ``head_scan_fn`` (see
    ``head_scan_block``). Lengths that do not fit are cut and reported in
    counts[3] (``RequestTables.check``). The context is kept, not copied.
    """
    _cuda(lengths, "request_tables")
    t = RequestTables()
    t.tokens, t.block = num_tokens, block
    (t.offsets, t.token_request, t.token_position, t.blocks, t.slots, t.counts, t._plan, t.max_blocks,
     t.context, t.carried) = _bind().request_tables(lengths, num_tokens, context, slots, free_slots, block)
    return t


def head_scan_block(num_tokens, num_requests, heads, headdim, dtype=torch.bfloat16):
    """The block for ``request_tables`` that suits ``head_scan_fn`` at these sizes."""
    _bind()
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return int(api.load_library().ss_head_scan_block(num_tokens, num_requests, heads, headdim, _DT[dtype], sms))


def packed_conv1d_fn(x, weight, tables, bias=None, conv_state=None, activation=None):
    """Causal depthwise conv1d of packed requests on CUDA tensors.

    x: (tokens, dim), rows of any stride; weight: (dim, width) fp32, width 2 to
    4; tables: ``request_tables`` of the batch; bias: (dim,) fp32; conv_state:
    (slots, dim, width - 1) in x's dtype, the last inputs of each slot's
    request, oldest first: read where context is above 0 and replaced in place;
    activation: None, 'silu' or 'swish'. Returns out (tokens, dim), zeros past
    the last token. Forward only.
    """
    _cuda(x, "packed_conv1d_fn")
    return _bind().packed_conv1d(x, weight, tables._plan, bias, conv_state, _activation(activation))


def packed_conv1d_update(x, conv_state, weight, bias=None, slots=None, activation=None):
    """One token per request: x (requests, dim); row r goes with window
    conv_state[slots[r]] (slots None: r), updated in place; a row with slot -1
    gets zeros. Two rows must not share a slot. Returns out (requests, dim).
    """
    _cuda(x, "packed_conv1d_update")
    return _bind().packed_conv1d_update(x, conv_state, weight, bias, slots, _activation(activation))


def head_scan_fn(x, dt, A, B, C, tables, D=None, z=None, dt_bias=None, dt_softplus=False, state=None):
    """Selective scan with one decay per head over packed requests.

    x, z: (tokens, heads, headdim); dt: (tokens, heads) in x's dtype or fp32;
    A, D, dt_bias: (heads,) fp32; B, C: (tokens, groups, dstate), head h of
    group h // (heads // groups); tables: ``request_tables`` of the batch; state:
    (slots, heads, headdim, dstate) fp32, read where context is above 0 and
    replaced in place. Per token: S = exp(dt A) S + dt x B^T, out = (S C + D x)
    silu(z). Returns out (tokens, heads, headdim), zeros past the last token.
    headdim and dstate up to 256. Forward only.
    """
    _cuda(x, "head_scan_fn")
    return _bind().head_scan(x, dt, A, B, C, tables._plan, D, z, dt_bias, dt_softplus, state)


def head_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False, slots=None):
    """One token per request: x, z (requests, heads, headdim), dt (requests,
    heads), B, C (requests, groups, dstate); row r goes with state[slots[r]]
    (slots None: r), updated in place; a row with slot -1 gets zeros. Two rows
    must not share a slot. Returns out (requests, heads, headdim).
    """
    _cuda(x, "head_state_update")
    return _bind().head_state_update(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, slots)
