"""The layer operators' C ABI and binding checks on the CPU (no CUDA call is made)."""
import os
import re
import shutil
import subprocess

import pytest
import torch

from state_space_model_03_gb300 import api, layer
from state_space_model_03_gb300 import build as ssbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssfwd_layer.h")


@pytest.fixture(scope="module")
def lib():
    ssbuild.build()
    return api.load_library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ss_[a-z_0-9]+)\s*\(", text))
    ops = {"ss_gated_scan", "ss_gated_scan_bwd", "ss_packed_gated_scan", "ss_gated_state_update", "ss_rms_norm", "ss_rms_norm_bwd",
           "ss_rms_norm_quant"}
    assert names == ops | {n + "_validate" for n in ops} | {n + "_workspace_size" for n in ("ss_gated_scan", "ss_packed_gated_scan", "ss_gated_scan_bwd", "ss_rms_norm_bwd")}
    for n in names:
        assert hasattr(lib, n), n


# (name, changes to a valid problem, wanted status)
SCAN = [
    ("good", "", 0),
    ("version", "p.abi_version = 0;", 10),
    ("dtype", "p.dtype = 9;", 3),
    ("rate0", "p.rate = 0;", 7),
    ("rate_nan", "p.rate = 0.0f / (p.rate - p.rate);", 7),
    ("dim0", "p.dim = 0;", 2),
    ("no_tokens", "p.seqlen = 0;", 2),
    ("no_batch", "p.batch = 0; p.x = 0;", 0),
    ("long", "p.seqlen = INT64_MAX / 4;", 7),
    ("many", "p.batch = (int64_t)1 << 23;", 7),
    ("null_x", "p.x = 0;", 1),
    ("null_gate", "p.gate = 0;", 1),
    ("null_decay", "p.decay = 0;", 1),
    ("null_out", "p.out = 0;", 1),
    ("no_input_gate", "p.input_gate = 0;", 0),
    ("negative", "p.gate_stride[1] = -1;", 4),
    ("out_rows_meet", "p.out_stride[1] = 64;", 4),
    ("out_sequences_meet", "p.out_stride[0] = 100;", 4),
    ("out_tokens_first", "p.out_stride[0] = 96; p.out_stride[1] = 288;", 0),
    ("x_broadcast", "p.x_stride[0] = 0;", 0),
    ("align_x", "p.x = (const void *)((uintptr_t)p.x + 1);", 5),
    ("align_state", "p.last_state = (float *)((uintptr_t)p.last_state + 2);", 5),
    ("alias_x", "p.out = (void *)(uintptr_t)p.x;", 6),
    ("alias_kept", "p.kept = p.last_state;", 6),
    ("alias_init", "p.initial_state = p.last_state;", 6),
    ("alias_decay", "p.decay = p.out;", 6),
    # parts of one row
    ("out_beside_x", "p.x_stride[0] = p.out_stride[0] = 20000; p.x_stride[1] = p.out_stride[1] = 200; p.out = (void *)((uintptr_t)p.x + 192);", 0),
    ("out_over_x", "p.x_stride[0] = p.out_stride[0] = 20000; p.x_stride[1] = p.out_stride[1] = 200; p.out = (void *)((uintptr_t)p.x + 190);", 6),
]
BWD = [
    ("good", "", 0),
    ("null_dout", "p.dout = 0;", 1),
    ("null_kept", "p.kept = 0;", 1),
    ("gate_of_none", "p.input_gate = 0;", 1),
    ("only_ddecay", "p.dx = p.dgate = p.dinput_gate = 0; p.dinitial_state = 0;", 0),
    ("no_workspace", "p.workspace = 0;", 11),
    ("small_workspace", "p.workspace_bytes = 4;", 11),
    ("no_ddecay", "p.ddecay = 0; p.workspace = 0; p.workspace_bytes = 0;", 0),
    ("align_workspace", "p.workspace = (void *)((uintptr_t)p.workspace + 4);", 5),
    ("alias", "p.dx = p.dgate;", 6),
    ("alias_in", "p.dx = (void *)(uintptr_t)p.dout;", 6),
    ("alias_flat", "p.dinitial_state = p.ddecay;", 6),
    ("rows_meet", "p.dgate_stride[1] = 1;", 4),
]
PACKED = [
    ("good", "", 0),
    ("rate", "p.rate = -1;", 7),
    ("null_table", "p.tables.token_request = 0;", 1),
    ("max_blocks", "p.tables.max_blocks = 1;", 2),
    ("no_state", "p.state = 0; p.slots = 0;", 0),
    ("slots", "p.slots = -1;", 2),
    ("slots_meet", "p.state_stride = 8;", 4),
    ("alias", "p.out = (void *)(uintptr_t)p.gate;", 6),
    ("alias_state", "p.state = p.out;", 6),
    ("no_tokens", "p.tables.tokens = 0; p.tables.max_blocks = 0; p.x = 0;", 0),
    ("rows_of_one", "p.x_stride = p.out_stride = 300; p.out = (void *)((uintptr_t)p.x + 192);", 0),
]
STEP = [
    ("good", "", 0),
    ("no_state", "p.state = 0;", 1),
    ("slots", "p.slot_map = 0; p.slots = 2;", 2),
    ("many", "p.requests = 65536;", 7),
    ("empty", "p.requests = 0; p.x = 0;", 0),
    ("alias_map", "p.slot_map = (const int32_t *)p.out;", 6),
]
NORM = [
    ("good", "", 0),
    ("dtype", "p.dtype = 4;", 3),
    ("residual_dtype", "p.residual_dtype = SS_F16;", 3),
    ("ignored_dtype", "p.residual = 0; p.sum = 0; p.residual_dtype = SS_F16;", 0),
    ("weight_dtype", "p.weight_dtype = SS_F16;", 3),
    ("dim0", "p.dim = 0;", 2),
    ("wide", "p.dim = SS_NORM_MAX_DIM + 1;", 7),
    ("rows", "p.rows = (int64_t)1 << 31;", 7),
    ("eps", "p.eps = -1;", 7),
    ("eps0", "p.eps = 0;", 0),
    ("null", "p.weight = 0;", 1),
    ("sum_of_none", "p.residual = 0;", 1),
    ("in_place", "p.sum = (void *)(uintptr_t)p.residual;", 0),
    ("alias", "p.out = (void *)(uintptr_t)p.x;", 6),
    ("alias_sum", "p.sum = p.out;", 6),
    ("alias_rstd", "p.rstd = (float *)p.sum;", 6),
    ("no_rows", "p.rows = 0; p.x = 0;", 0),
]
NORM_BWD = [
    ("good", "", 0),
    ("null", "p.rstd = 0;", 1),
    ("no_workspace", "p.workspace = 0;", 11),
    ("small_workspace", "p.workspace_bytes = 16;", 11),
    ("no_dweight", "p.dweight = 0; p.workspace = 0;", 0),
    ("alias", "p.dresidual = (void *)(uintptr_t)p.dsum;", 6),
    ("alias_dweight", "p.dweight = p.dx;", 6),
]
QUANT = [
    ("good", "", 0),
    ("row", "p.group = 0;", 0),
    ("group", "p.group = 16;", 7),
    ("scale_type", "p.scale_type = 2;", 7),
    ("null_scale", "p.scale = 0;", 1),
    ("align_scale", "p.scale = (void *)((uintptr_t)p.scale + 2);", 5),
    ("bytes", "p.scale_type = SS_SCALE_E8M0; p.scale = (void *)((uintptr_t)p.scale + 2);", 0),
    ("alias_scale", "p.scale = p.out;", 6),
]

HEAD = r"""
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include "ssfwd_layer.h"
static uintptr_t next_at = 1u << 20;
static void *buf(void) { next_at += 1u << 24; return (void *)next_at; }
#define ROWS(f, a, b) p.f[0] = a; p.f[1] = b
static ss_gated_scan_params scan(void) {
  ss_gated_scan_params p;
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_BF16; p.rate = 8; p.batch = 3; p.seqlen = 100; p.dim = 96;
  p.x = buf(); p.gate = buf(); p.input_gate = buf(); p.decay = buf(); p.initial_state = buf(); p.out = buf(); p.last_state = buf(); p.kept = buf();
  ROWS(x_stride, 9600, 96); ROWS(gate_stride, 9600, 96); ROWS(input_gate_stride, 9600, 96); ROWS(out_stride, 9600, 96);
  return p;
}
static ss_gated_scan_bwd_params bwd(void) {
  ss_gated_scan_bwd_params p;
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_F32; p.rate = 8; p.batch = 3; p.seqlen = 100; p.dim = 96;
  p.x = buf(); p.gate = buf(); p.input_gate = buf(); p.dout = buf(); p.decay = buf(); p.kept = buf(); p.dlast = buf();
  p.dx = buf(); p.dgate = buf(); p.dinput_gate = buf(); p.ddecay = buf(); p.dinitial_state = buf(); p.workspace = buf();
  ROWS(x_stride, 9600, 96); ROWS(gate_stride, 9600, 96); ROWS(input_gate_stride, 9600, 96); ROWS(dout_stride, 9600, 96);
  ROWS(dx_stride, 9600, 96); ROWS(dgate_stride, 9600, 96); ROWS(dinput_gate_stride, 9600, 96);
  p.workspace_bytes = 1 << 20;
  return p;
}
static ss_packed_gated_scan_params packed(void) {
  ss_packed_gated_scan_params p;
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_BF16; p.rate = 8; p.dim = 96; p.slots = 4;
  p.x = buf(); p.gate = buf(); p.input_gate = buf(); p.decay = buf(); p.state = buf(); p.out = buf();
  p.x_stride = p.gate_stride = p.input_gate_stride = p.out_stride = p.state_stride = 96;
  p.tables.requests = 3; p.tables.tokens = 256; p.tables.block = 128; p.tables.max_blocks = 5;
  p.tables.offsets = buf(); p.tables.token_request = buf(); p.tables.blocks = buf(); p.tables.carried = buf(); p.tables.slot_map = buf();
  p.tables.counts = buf();
  return p;
}
static ss_gated_state_update_params step(void) {
  ss_gated_state_update_params p;
  ss_packed_gated_scan_params s = packed();
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_F16; p.rate = 8; p.requests = 3; p.dim = 96; p.slots = 4;
  p.x = s.x; p.gate = s.gate; p.input_gate = s.input_gate; p.decay = s.decay; p.state = s.state; p.out = s.out; p.slot_map = buf();
  p.x_stride = p.gate_stride = p.input_gate_stride = p.out_stride = p.state_stride = 96;
  return p;
}
static ss_rms_norm_params norm(void) {
  ss_rms_norm_params p;
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_BF16; p.residual_dtype = SS_F32; p.weight_dtype = SS_F32; p.eps = 1e-5f; p.rows = 9; p.dim = 96;
  p.x = buf(); p.residual = buf(); p.weight = buf(); p.out = buf(); p.sum = buf(); p.rstd = buf();
  p.x_stride = p.residual_stride = p.out_stride = p.sum_stride = 96;
  return p;
}
static ss_rms_norm_bwd_params norm_bwd(void) {
  ss_rms_norm_bwd_params p;
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_BF16; p.residual_dtype = SS_F32; p.weight_dtype = SS_BF16; p.rows = 9; p.dim = 96;
  p.dout = buf(); p.dsum = buf(); p.sum = buf(); p.weight = buf(); p.rstd = buf(); p.dx = buf(); p.dresidual = buf(); p.dweight = buf();
  p.workspace = buf(); p.workspace_bytes = 1 << 20;
  p.dout_stride = p.dsum_stride = p.sum_stride = p.dx_stride = p.dresidual_stride = 96;
  return p;
}
static ss_rms_norm_quant_params quant(void) {
  ss_rms_norm_quant_params p;
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_BF16; p.residual_dtype = SS_BF16; p.weight_dtype = SS_F32; p.eps = 1e-5f; p.rows = 9; p.dim = 96;
  p.group = 32; p.x = buf(); p.residual = buf(); p.weight = buf(); p.out = buf(); p.scale = buf(); p.sum = buf();
  p.x_stride = p.residual_stride = p.out_stride = p.sum_stride = 96;
  return p;
}
int main(void) {
  int64_t bytes = -1;
  printf("null %d %d %d %d %d %d %d\n", ss_gated_scan_validate(0), ss_gated_scan_bwd_validate(0), ss_packed_gated_scan_validate(0),
         ss_gated_state_update_validate(0), ss_rms_norm_validate(0), ss_rms_norm_bwd_validate(0), ss_rms_norm_quant_validate(0));
  { ss_gated_scan_bwd_params p = bwd(); p.workspace = 0; const int st = ss_gated_scan_bwd_workspace_size(&p, &bytes);
    printf("ws_scan %d %d\n", st, bytes >= 4 * 3 * 96); }
  { ss_rms_norm_bwd_params p = norm_bwd(); p.workspace = 0; const int st = ss_rms_norm_bwd_workspace_size(&p, &bytes);
    printf("ws_norm %d %d\n", st, bytes >= 4 * 96); }
"""
KINDS = [("scan", "ss_gated_scan", SCAN), ("bwd", "ss_gated_scan_bwd", BWD), ("packed", "ss_packed_gated_scan", PACKED),
         ("step", "ss_gated_state_update", STEP), ("norm", "ss_rms_norm", NORM), ("norm_bwd", "ss_rms_norm_bwd", NORM_BWD),
         ("quant", "ss_rms_norm_quant", QUANT)]


def test_c_program_against_the_library(lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    body = ""
    for kind, fn, cases in KINDS:
        for name, change, _ in cases:
            body += f'  {{ {fn}_params p = {kind}(); {change} printf("{kind}.{name} %d\\n", {fn}_validate(&p)); }}\n'
    libdir = os.path.dirname(api.library_path())
    src, exe = tmp_path / "consumer.c", tmp_path / "consumer"
    src.write_text(HEAD + body + "  return 0;\n}\n")
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    "-L", libdir, "-lssfwd", "-Wl,-rpath," + libdir], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    got = dict(line.split(" ", 1) for line in r.stdout.strip().splitlines())
    assert got["null"] == "1 1 1 1 1 1 1"
    assert got["ws_scan"] == got["ws_norm"] == "0 1"
    wrong = [(kind, name, got[f"{kind}.{name}"], status) for kind, _, cases in KINDS for name, _, status in cases if got[f"{kind}.{name}"] != str(status)]
    assert not wrong


def test_operators_need_cuda_tensors():
    x, d = torch.zeros(1, 2, 8), torch.zeros(8)
    for call in (lambda: layer.gated_scan_fn(x, x, d), lambda: layer.packed_gated_scan_fn(x[0], x[0], d, None),
                 lambda: layer.gated_state_update(torch.zeros(2, 8), x[0], x[0], d), lambda: layer.rms_norm_fn(x, d),
                 lambda: layer.rms_norm_quant_fn(x, d)):
        with pytest.raises(RuntimeError, match="CUDA"):
            call()


def test_binding_checks_before_any_cuda_call(lib):
    b = layer._bind()
    x, d, st = torch.zeros(1, 2, 8), torch.zeros(8), torch.zeros(2, 8)
    with pytest.raises(TypeError, match="arguments"):
        b.gated_scan(x)
    with pytest.raises(TypeError, match="fp32/fp16/bf16"):
        b.gated_scan(x.double(), x, d, None, 8.0, None, False)
    with pytest.raises(TypeError, match="fp32/fp16/bf16"):
        b.gated_scan(x[0], x[0], d, None, 8.0, None, False)
    with pytest.raises(TypeError, match="gate"):
        b.gated_scan(x, x.half(), d, None, 8.0, None, False)
    with pytest.raises(TypeError, match="input_gate"):
        b.gated_scan(x, x, d, x[:, :1], 8.0, None, False)
    with pytest.raises(TypeError, match="decay"):
        b.gated_scan(x, x, d[:7], None, 8.0, None, False)
    with pytest.raises(TypeError, match="initial_state"):
        b.gated_scan(x, x, d, None, 8.0, st, False)
    with pytest.raises(TypeError):
        b.gated_scan(x, x, d, None, "fast", None, False)
    with pytest.raises(TypeError, match="state"):
        b.gated_state_update(st.half(), x[0], x[0], d, None, 8.0, None)
    with pytest.raises(ValueError, match="in place"):
        b.gated_state_update(torch.zeros(8, 2).t(), x[0], x[0], d, None, 8.0, None)
    with pytest.raises(TypeError, match="slots"):
        b.gated_state_update(st, x[0], x[0], d, None, 8.0, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(NotImplementedError):
        b.gated_state_update(st.clone().requires_grad_(), x[0], x[0], d, None, 8.0, None)
    with pytest.raises(TypeError, match="RequestTables"):
        b.packed_gated_scan(x[0], x[0], d, b"", None, 8.0, None)
    with pytest.raises(TypeError, match="weight"):
        b.rms_norm(x, d[:7], None, 1e-5, False)
    with pytest.raises(TypeError, match="weight"):
        b.rms_norm(x, d.half(), None, 1e-5, False)
    with pytest.raises(TypeError, match="residual"):
        b.rms_norm(x, d, x.half(), 1e-5, False)
    with pytest.raises(ValueError, match="channel"):
        b.rms_norm(x[..., :0], d[:0], None, 1e-5, False)
    with pytest.raises(ValueError, match="group_size"):
        b.rms_norm_quant(x, d, None, 1e-5, False, 48, False)
    with pytest.raises(TypeError, match="scale_dtype"):
        layer.rms_norm_quant_fn(_OnGpu(), None, scale_dtype=torch.float16)


class _OnGpu:
    is_cuda = True  # a stand-in: the scale's type is looked at after the device
