"""Packed requests: Python binding of include/ssfwd_packed.h.

A batch of requests of different lengths, their tokens one after another in
(tokens, channels) tensors without padding, each request with a slot in a cache
of states. ``request_tables`` builds the batch's tables on the GPU;
``packed_conv1d_fn`` and ``head_scan_fn`` run prompts, ``packed_conv1d_update``
and ``head_state_update`` one token per request.

As in api.py this is argument marshalling only, on the current stream, and there
is no CPU fallback. The parameter blocks are packed with ``struct`` rather than
filled field by field: the one-token operators take a few microseconds on the
GPU, which the host has to keep up with.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import api
from .api import SS_ABI_VERSION, _DT, _activation, _check

_NEG_STATE = "state must be float32 (slots, heads, headdim, dstate) with its last two dimensions contiguous"

_TABLES = struct.Struct("=2i5q10Q")
_CONV = struct.Struct("=4i3q5Q3q4q6Q")
_CONV_STEP = struct.Struct("=4i4q6Q3q")
_SCAN = struct.Struct("=4i5q10Q14qQq4q6Q")
_STEP = struct.Struct("=4i6q11Q14q")

_packed_lib = None


def _lib():
    global _packed_lib
    if _packed_lib is None:
        lib = api.load_library()
        vp = ctypes.c_void_p
        for name in ("ss_request_tables", "ss_packed_conv1d", "ss_packed_conv1d_update", "ss_head_scan",
                     "ss_head_state_update"):
            f = getattr(lib, name)
            f.argtypes, f.restype = [ctypes.c_char_p, vp], ctypes.c_int
            v = getattr(lib, name + "_validate")
            v.argtypes, v.restype = [ctypes.c_char_p], ctypes.c_int
        lib.ss_head_scan_workspace_size.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_int64)]
        lib.ss_head_scan_workspace_size.restype = ctypes.c_int
        lib.ss_head_scan_block.argtypes = [ctypes.c_int64] * 4 + [ctypes.c_int32] * 2
        lib.ss_head_scan_block.restype = ctypes.c_int64
        _packed_lib = lib
    return _packed_lib


def _call(fn, block, device):
    """fn(block, current stream) with `device` current."""
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        _check(fn(block, stream))
    else:
        with torch.cuda.device(device):
            _check(fn(block, stream))


def _int32(name, t, shape, device):
    if t.dtype != torch.int32 or tuple(t.shape) != shape:
        raise TypeError(f"{name} must be int32 {shape}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t if t.is_contiguous() else t.contiguous()


def _on(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}")


def _no_grad(*tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise NotImplementedError("the packed operators are forward only")


class RequestTables:
    """Tables of one packed batch (int32, on the GPU), as ``request_tables``
    makes them: ``offsets`` (requests + 1), ``token_request`` and
    ``token_position`` (tokens), ``blocks`` (max_blocks, 4), ``slots``
    (requests) and ``counts`` (4: tokens, blocks, slots taken, errors)."""

    __slots__ = ("requests", "tokens", "block", "max_blocks", "device", "offsets", "token_request",
                 "token_position", "blocks", "slots", "counts", "context", "_packed")

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

    lengths: (requests,) int32 new tokens per request, 0 allowed. num_tokens:
    rows of the packed tensors; rows past the last request's are padding.
    context: (requests,) int32 tokens that each request has had before; where it
    is above 0 the operators go on from the request's slot (None: all start from
    zero). slots: (requests,) int32 slot of each request, -1 for one that has
    none yet and takes the next of free_slots (None: request r has slot r).
    block: tokens per unit of work of ``head_scan_fn`` (see
    ``head_scan_block``). Lengths that do not fit are cut and reported in
    counts[3] (``RequestTables.check``). The context is kept, not copied.
    """
    if not lengths.is_cuda:
        raise RuntimeError("request_tables needs CUDA tensors (there is no CPU path)")
    lib = _lib()
    dev = lengths.device
    if lengths.dim() != 1:
        raise TypeError("lengths must be int32 (requests,)")
    n, tokens, block = lengths.shape[0], int(num_tokens), int(block)
    lengths = _int32("lengths", lengths, (n,), dev)
    if context is not None:
        context = _int32("context", context, (n,), dev)
    if slots is not None:
        slots = _int32("slots", slots, (n,), dev)
    free = 0
    if free_slots is not None:
        if slots is None:
            raise ValueError("free_slots goes with slots")
        free = free_slots.numel()
        free_slots = _int32("free_slots", free_slots, (free,), dev)
    if tokens < 0 or block < 1:
        raise ValueError("num_tokens must be >= 0 and block >= 1")
    most = tokens // block + min(n, tokens)
    # one buffer for all, each table on 16 bytes
    sizes = [-(-k // 4) * 4 for k in (n + 1, tokens, tokens, 4 * most, n)] + [4]
    buf = torch.empty(sum(sizes), dtype=torch.int32, device=dev)
    at = buf.data_ptr()
    ptr = []
    for k in sizes:
        ptr.append(at)
        at += 4 * k
    t = RequestTables()
    t.requests, t.tokens, t.block, t.max_blocks, t.device, t.context = n, tokens, block, most, dev, context
    ctx = 0 if context is None else context.data_ptr()
    _call(lib.ss_request_tables, _TABLES.pack(
        SS_ABI_VERSION, 0, n, tokens, block, most, free, lengths.data_ptr(), ctx,
        0 if slots is None else slots.data_ptr(), 0 if free_slots is None else free_slots.data_ptr(), *ptr), dev)
    off, req, pos, blk, slt, t.counts = buf.split(sizes)
    t.offsets, t.token_request, t.token_position, t.slots = off[:n + 1], req[:tokens], pos[:tokens], slt[:n]
    t.blocks = blk.view(-1, 4)
    t._packed = (n, tokens, block, most, ptr[0], ptr[1], ptr[3], ptr[4], ptr[5], ctx)
    return t


def head_scan_block(num_tokens, num_requests, heads, headdim, dtype=torch.bfloat16):
    """The block for ``request_tables`` that suits ``head_scan_fn`` at these sizes."""
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return int(_lib().ss_head_scan_block(num_tokens, num_requests, heads, headdim, _DT[dtype], sms))


def _conv_operands(x, weight, bias, conv_state):
    if x.dim() != 2 or x.dtype not in _DT:
        raise TypeError("x must be (tokens, dim) fp32/fp16/bf16")
    dim = x.shape[1]
    if weight.dim() != 2 or weight.shape[0] != dim or weight.dtype != torch.float32:
        raise TypeError("weight must be float32 (dim, width)")
    width = weight.shape[1]
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (dim,)):
        raise TypeError("bias must be float32 (dim,)")
    if conv_state is not None:
        if conv_state.dtype != x.dtype or conv_state.dim() != 3 or tuple(conv_state.shape[1:]) != (dim, width - 1):
            raise TypeError("conv_state must be x's dtype (slots, dim, width - 1)")
        if width > 1 and conv_state.numel() and (conv_state.stride(2) != 1 or conv_state.stride(1) != width - 1):
            raise ValueError("conv_state must be contiguous but for its slot stride (it is updated in place)")
    _on(x.device, weight=weight, bias=bias, conv_state=conv_state)
    _no_grad(x, weight, bias, conv_state)
    if x.stride(1) != 1:
        x = x.contiguous()
    return x, weight.contiguous(), None if bias is None else bias.contiguous(), dim, width


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def packed_conv1d_fn(x, weight, tables, bias=None, conv_state=None, activation=None):
    """Causal depthwise conv1d of packed requests on CUDA tensors.

    x: (tokens, dim), rows of any stride; weight: (dim, width) fp32, width 2 to
    4; tables: ``request_tables`` of the batch; bias: (dim,) fp32; conv_state:
    (slots, dim, width - 1) in x's dtype, the last inputs of each slot's
    request, oldest first: read where context is above 0 and replaced in place;
    activation: None, 'silu' or 'swish'. Returns out (tokens, dim), zeros past
    the last token. Forward only.
    """
    if not x.is_cuda:
        raise RuntimeError("packed_conv1d_fn needs CUDA tensors (there is no CPU path)")
    act = _activation(activation)
    x, weight, bias, dim, width = _conv_operands(x, weight, bias, conv_state)
    if tables.tokens != x.shape[0] or tables.device != x.device:
        raise ValueError("tables are of another batch: x must have num_tokens rows, on their device")
    out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    slots = 0 if conv_state is None else conv_state.shape[0]
    _call(_lib().ss_packed_conv1d, _CONV.pack(
        SS_ABI_VERSION, _DT[x.dtype], act, 0, dim, width, slots, x.data_ptr(), weight.data_ptr(), _ptr(bias),
        _ptr(conv_state), out.data_ptr(), x.stride(0), dim, 0 if conv_state is None else conv_state.stride(0),
        *tables._packed), x.device)
    return out


def packed_conv1d_update(x, conv_state, weight, bias=None, slots=None, activation=None):
    """One token per request: x (requests, dim); row r goes with window
    conv_state[slots[r]] (slots None: r), updated in place; a row with slot -1
    gets zeros. Two rows must not share a slot. Returns out (requests, dim).
    """
    if not x.is_cuda:
        raise RuntimeError("packed_conv1d_update needs CUDA tensors (there is no CPU path)")
    act = _activation(activation)
    x, weight, bias, dim, width = _conv_operands(x, weight, bias, conv_state)
    n = x.shape[0]
    if slots is not None:
        slots = _int32("slots", slots, (n,), x.device)
    out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _call(_lib().ss_packed_conv1d_update, _CONV_STEP.pack(
        SS_ABI_VERSION, _DT[x.dtype], act, 0, n, dim, width, conv_state.shape[0], x.data_ptr(), weight.data_ptr(),
        _ptr(bias), _ptr(slots), conv_state.data_ptr(), out.data_ptr(), x.stride(0), dim, conv_state.stride(0)), x.device)
    return out


def _rows(t):
    return t if t is None or t.stride(-1) == 1 else t.contiguous()


def _head_operands(x, dt, A, B, C, D, z, dt_bias, state):
    if x.dim() != 3 or x.dtype not in _DT:
        raise TypeError("x must be (tokens, heads, headdim) fp32/fp16/bf16")
    rows, heads, headdim = x.shape
    if tuple(dt.shape) != (rows, heads) or dt.dtype not in (x.dtype, torch.float32):
        raise TypeError("dt must be (tokens, heads) in x's dtype or float32")
    if B.dim() != 3 or B.shape[0] != rows or B.dtype != x.dtype or C.shape != B.shape or C.dtype != x.dtype:
        raise TypeError("B and C must be (tokens, groups, dstate) in x's dtype")
    if z is not None and (z.shape != x.shape or z.dtype != x.dtype):
        raise TypeError("z must match x in shape and dtype")
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias)):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (heads,)):
            raise TypeError(f"{name} must be float32 (heads,)")
    groups, dstate = B.shape[1:]
    if state is not None:
        if state.dtype != torch.float32 or state.dim() != 4 or tuple(state.shape[1:]) != (heads, headdim, dstate):
            raise TypeError(_NEG_STATE)
        if state.numel() and (state.stride(3) != 1 or (headdim > 1 and state.stride(2) != dstate)):
            raise ValueError(_NEG_STATE + " (it is updated in place)")
    _on(x.device, dt=dt, A=A, B=B, C=C, D=D, z=z, dt_bias=dt_bias, state=state)
    _no_grad(x, dt, A, B, C, D, z, dt_bias, state)
    return (_rows(x), dt, A.contiguous(), _rows(B), _rows(C), None if D is None else D.contiguous(), _rows(z),
            None if dt_bias is None else dt_bias.contiguous(), heads, headdim, groups, dstate)


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
    if not x.is_cuda:
        raise RuntimeError("head_scan_fn needs CUDA tensors (there is no CPU path)")
    lib = _lib()
    x, dt, A, B, C, D, z, dt_bias, heads, headdim, groups, dstate = _head_operands(x, dt, A, B, C, D, z, dt_bias, state)
    dev = x.device
    if tables.tokens != x.shape[0] or tables.device != dev:
        raise ValueError("tables are of another batch: x must have num_tokens rows, on their device")
    out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    ws, ws_bytes = None, 0
    if tables.tokens > tables.block:
        ws_bytes = 4 * tables.max_blocks * heads * (headdim * dstate + 1)
        ws = torch.empty(ws_bytes // 4, dtype=torch.float32, device=dev)
    slots, ss = (0, (0, 0)) if state is None else (state.shape[0], state.stride()[:2])
    _call(lib.ss_head_scan, _SCAN.pack(
        SS_ABI_VERSION, _DT[x.dtype], _DT[dt.dtype], int(bool(dt_softplus)), heads, headdim, dstate, groups, slots,
        x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(z), A.data_ptr(), _ptr(D), _ptr(dt_bias),
        _ptr(state), out.data_ptr(), *x.stride()[:2], *dt.stride(), *B.stride()[:2], *C.stride()[:2],
        *((0, 0) if z is None else z.stride()[:2]), *out.stride()[:2], *ss, _ptr(ws), ws_bytes, *tables._packed), dev)
    return out


def head_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False, slots=None):
    """One token per request: x, z (requests, heads, headdim), dt (requests,
    heads), B, C (requests, groups, dstate); row r goes with state[slots[r]]
    (slots None: r), updated in place; a row with slot -1 gets zeros. Two rows
    must not share a slot. Returns out (requests, heads, headdim).
    """
    if not x.is_cuda:
        raise RuntimeError("head_state_update needs CUDA tensors (there is no CPU path)")
    lib = _lib()
    x, dt, A, B, C, D, z, dt_bias, heads, headdim, groups, dstate = _head_operands(x, dt, A, B, C, D, z, dt_bias, state)
    n, dev = x.shape[0], x.device
    if slots is not None:
        slots = _int32("slots", slots, (n,), dev)
    out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    _call(lib.ss_head_state_update, _STEP.pack(
        SS_ABI_VERSION, _DT[x.dtype], _DT[dt.dtype], int(bool(dt_softplus)), n, heads, headdim, dstate, groups,
        state.shape[0], x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(z), A.data_ptr(), _ptr(D),
        _ptr(dt_bias), _ptr(slots), state.data_ptr(), out.data_ptr(), *x.stride()[:2], *dt.stride(), *B.stride()[:2],
        *C.stride()[:2], *((0, 0) if z is None else z.stride()[:2]), *out.stride()[:2], *state.stride()[:2]), dev)
    return out
