"""The layer operators through the C ABI on tensors that the test lays out itself (the
Python functions make their own outputs). The structures are read from the headers."""
import ctypes
import os
import re

import torch

from state_space_model_03_gb300 import api

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _structs():
    text = "".join(open(os.path.join(INCLUDE, h)).read() for h in ("ssfwd_packed.h", "ssfwd_layer.h"))
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    plain = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float}
    made = {}
    for body, name in re.findall(r"typedef struct \w+ \{(.*?)\} (\w+);", text, re.S):
        fields = []
        for kind, names in re.findall(r"^\s*(?:const )?(\w+) ([^;]*);", body, re.M):
            for field in (n.strip() for n in names.split(",")):
                at, count = re.match(r"\*?(\w+)(?:\[(\d+)\])?$", field).groups()
                t = ctypes.c_void_p if field.startswith("*") else plain.get(kind) or made[kind]
                fields.append((at, t * int(count) if count else t))
        made[name] = type(name, (ctypes.Structure,), {"_fields_": fields})
    return made


STRUCTS = _structs()


def params(op, dtype, **values):
    """ss_<op>_params with what is given; a tensor gives its field the address, and the strides of its rows."""
    p = STRUCTS[f"ss_{op}_params"]()
    p.abi_version, p.dtype = api.load_library().ss_abi_version(), DTYPES[dtype]
    for k, v in values.items():
        if not torch.is_tensor(v):
            setattr(p, k, v)
            continue
        setattr(p, k, v.data_ptr())
        if hasattr(p, k + "_stride"):
            if isinstance(getattr(p, k + "_stride"), int):
                setattr(p, k + "_stride", v.stride(0))
            else:
                getattr(p, k + "_stride")[:] = v.stride()[:2]
    return p


def packed_tables(tables):
    """A RequestTables as the C ABI takes it."""
    t = STRUCTS["ss_packed_tables"](tables.slots.numel(), tables.tokens, tables.block, tables.max_blocks)
    for c, name in (("offsets", "offsets"), ("token_request", "token_request"), ("blocks", "blocks"), ("carried", "carried"),
                    ("slot_map", "slots"), ("counts", "counts"), ("context", "context")):
        v = getattr(tables, name)
        setattr(t, c, None if v is None else v.data_ptr())
    return t


def run(op, p, workspace=None):
    """The call on the current stream with a workspace of the size that it asks for (in `workspace`: a function that
    makes one of so many bytes); the status."""
    lib, held = api.load_library(), None
    if hasattr(p, "workspace"):
        need = ctypes.c_int64(-1)
        status = getattr(lib, f"ss_{op}_workspace_size")(ctypes.byref(p), ctypes.byref(need))
        if status:
            return status
        if need.value:
            held = (workspace or (lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")))(need.value)
            p.workspace, p.workspace_bytes = held.data_ptr(), need.value
    call = getattr(lib, f"ss_{op}")
    call.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    return call(ctypes.byref(p), torch.cuda.current_stream().cuda_stream)
