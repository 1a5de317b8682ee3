"""The packed operators' C ABI and binding checks on the CPU (no CUDA call is made).

A C99 program compiles include/ssfwd_packed.h with warnings as errors and asks the
validation entry points; the Python binding's checks that come before any CUDA
call run on CPU tensors.
"""
import os
import re
import shutil
import subprocess

import pytest
import torch

from state_space_model_03_gb300 import api, packed
from state_space_model_03_gb300 import build as ssbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssfwd_packed.h")


@pytest.fixture(scope="module")
def lib():
    ssbuild.build()
    return api.load_library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ss_[a-z_0-9]+)\s*\(", text))
    ops = {"ss_request_tables", "ss_packed_conv1d", "ss_packed_conv1d_update", "ss_head_scan", "ss_head_state_update"}
    assert names == ops | {n + "_validate" for n in ops} | {"ss_head_scan_workspace_size", "ss_head_scan_block"}
    for n in names:
        assert hasattr(lib, n), n


# (name, changes to a valid problem, wanted status)
SCAN = [
    ("good", "", 0),
    ("version", "p.abi_version = 0;", 10),
    ("dtype", "p.dtype = 9;", 3),
    ("dt_dtype", "p.dt_dtype = SS_F16;", 3),
    ("groups", "p.ngroups = 3;", 2),
    ("headdim0", "p.headdim = 0;", 2),
    ("headdim257", "p.headdim = 257;", 7),
    ("dstate257", "p.dstate = 257;", 7),
    ("heads8193", "p.heads = 8193;", 7),
    ("null_x", "p.x = 0;", 1),
    ("null_out", "p.out = 0;", 1),
    ("null_table", "p.tables.blocks = 0;", 1),
    ("null_carried", "p.tables.carried = 0;", 1),
    ("max_blocks", "p.tables.max_blocks = 1;", 2),
    ("requests", "p.tables.requests = SS_MAX_REQUESTS + 1;", 7),
    ("negative", "p.B_stride[0] = -1;", 4),
    ("out_rows_meet", "p.out_stride[0] = 64;", 4),
    ("state_slots_meet", "p.state_stride[0] = 64;", 4),
    ("align_x", "p.x = (const void *)((uintptr_t)p.x + 1);", 5),
    ("align_table", "p.tables.blocks = (const int32_t *)((uintptr_t)p.tables.blocks + 4);", 5),
    ("alias_x", "p.out = (void *)(uintptr_t)p.x;", 6),
    ("alias_state", "p.state = (float *)(uintptr_t)p.x;", 6),
    ("no_workspace", "p.workspace = 0;", 11),
    ("small_workspace", "p.workspace_bytes -= 4;", 11),
    ("one_block", "p.tables.block = 512; p.tables.max_blocks = 3; p.workspace = 0; p.workspace_bytes = 0;", 0),
    ("no_tokens", "p.tables.tokens = 0; p.tables.max_blocks = 0; p.x = 0; p.workspace = 0;", 0),
    # parts of one row: out beside x, and out over the end of x
    ("out_beside_x", "p.x_stride[0] = p.out_stride[0] = 512; p.out = (void *)((uintptr_t)p.x + 256);", 0),
    ("out_over_x", "p.x_stride[0] = p.out_stride[0] = 512; p.out = (void *)((uintptr_t)p.x + 128);", 6),
]
CONV = [
    ("good", "", 0),
    ("width1", "p.width = 1;", 7),
    ("width5", "p.width = 5;", 7),
    ("dim_large", "p.dim = (1 << 20) + 8;", 7),
    ("act", "p.activation = 7;", 7),
    ("dim", "p.dim = 0;", 2),
    ("null_w", "p.weight = 0;", 1),
    ("rows_meet", "p.out_stride = 8;", 4),
    ("windows_meet", "p.state_stride = 8;", 4),
    ("alias", "p.out = (void *)(uintptr_t)p.x;", 6),
    ("alias_state", "p.conv_state = p.out;", 6),
    ("no_state", "p.conv_state = 0;", 0),
]
TABLES = [
    ("good", "", 0),
    ("no_requests", "p.requests = 0; p.max_blocks = 2;", 2),
    ("block0", "p.block = 0;", 2),
    ("null_lengths", "p.lengths = 0;", 1),
    ("null_map", "p.token_request = 0;", 1),
    ("alias", "p.offsets = (int32_t *)(uintptr_t)p.lengths;", 6),
    ("alias_out", "p.token_request = p.token_position;", 6),
    ("align", "p.blocks = (int32_t *)((uintptr_t)p.blocks + 8);", 5),
    ("no_tokens", "p.tokens = 0; p.max_blocks = 0; p.token_request = p.token_position = p.blocks = 0;", 0),
]
STEP = [
    ("good", "", 0),
    ("no_state", "p.state = 0;", 1),
    ("slots", "p.slot_map = 0; p.slots = 2;", 2),
    ("many", "p.requests = 65536;", 7),
    ("empty", "p.requests = 0; p.x = 0;", 0),
]


def _program():
    head = r"""
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include "ssfwd_packed.h"
static uintptr_t next_at = 1u << 20;
static void *buf(void) { next_at += 1u << 24; return (void *)next_at; }
static ss_packed_tables tables(void) {
  ss_packed_tables t;
  memset(&t, 0, sizeof(t));
  t.requests = 3; t.tokens = 256; t.block = 128; t.max_blocks = 5;
  t.offsets = buf(); t.token_request = buf(); t.blocks = buf(); t.carried = buf(); t.slot_map = buf(); t.counts = buf();
  return t;
}
static ss_head_scan_params scan(void) {
  ss_head_scan_params p;
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_BF16; p.dt_dtype = SS_F32;
  p.heads = 2; p.headdim = 64; p.dstate = 32; p.ngroups = 1; p.slots = 4;
  p.x = buf(); p.dt = buf(); p.B = buf(); p.C = buf(); p.A = buf(); p.state = buf(); p.out = buf(); p.workspace = buf();
  p.x_stride[0] = p.out_stride[0] = 128; p.x_stride[1] = p.out_stride[1] = 64;
  p.dt_stride[0] = 2; p.dt_stride[1] = 1;
  p.B_stride[0] = p.C_stride[0] = 32;
  p.state_stride[0] = 4096; p.state_stride[1] = 2048;
  p.tables = tables();
  p.workspace_bytes = 5 * 2 * (2048 + 1) * 4;
  return p;
}
static ss_packed_conv1d_params conv(void) {
  ss_packed_conv1d_params p;
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_F16;
  p.dim = 24; p.width = 4; p.slots = 4;
  p.x = buf(); p.weight = buf(); p.conv_state = buf(); p.out = buf();
  p.x_stride = p.out_stride = 24; p.state_stride = 72;
  p.tables = tables();
  return p;
}
static ss_request_tables_params tab(void) {
  ss_request_tables_params p;
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.requests = 3; p.tokens = 256; p.block = 128; p.max_blocks = 5;
  p.lengths = buf(); p.offsets = buf(); p.token_request = buf(); p.token_position = buf(); p.blocks = buf(); p.carried = buf(); p.slot_map = buf();
  p.counts = buf();
  return p;
}
static ss_head_state_update_params step(void) {
  ss_head_state_update_params p;
  ss_head_scan_params s = scan();
  memset(&p, 0, sizeof(p));
  p.abi_version = SS_ABI_VERSION; p.dtype = SS_BF16; p.dt_dtype = SS_F32; p.requests = 3;
  p.heads = 2; p.headdim = 64; p.dstate = 32; p.ngroups = 1; p.slots = 4;
  p.x = s.x; p.dt = s.dt; p.B = s.B; p.C = s.C; p.A = s.A; p.state = s.state; p.out = s.out; p.slot_map = buf();
  memcpy(p.x_stride, s.x_stride, sizeof(s.x_stride)); memcpy(p.out_stride, s.out_stride, sizeof(s.out_stride));
  memcpy(p.dt_stride, s.dt_stride, sizeof(s.dt_stride)); memcpy(p.B_stride, s.B_stride, sizeof(s.B_stride));
  memcpy(p.C_stride, s.C_stride, sizeof(s.C_stride)); memcpy(p.state_stride, s.state_stride, sizeof(s.state_stride));
  return p;
}
int main(void) {
  int64_t bytes = -1;
  printf("null %d %d %d %d %d\n", ss_request_tables_validate(0), ss_packed_conv1d_validate(0), ss_packed_conv1d_update_validate(0),
         ss_head_scan_validate(0), ss_head_state_update_validate(0));
"""
    body = ""
    for kind, maker, fn, cases in (("scan", "ss_head_scan_params p = scan()", "ss_head_scan_validate", SCAN),
                                   ("conv", "ss_packed_conv1d_params p = conv()", "ss_packed_conv1d_validate", CONV),
                                   ("tables", "ss_request_tables_params p = tab()", "ss_request_tables_validate", TABLES),
                                   ("step", "ss_head_state_update_params p = step()", "ss_head_state_update_validate", STEP)):
        for name, change, _ in cases:
            body += f'  {{ {maker}; {change} printf("{kind}.{name} %d\\n", {fn}(&p)); }}\n'
    return head + body + r"""
  { ss_head_scan_params p = scan(); p.workspace = 0;
    { const int st = ss_head_scan_workspace_size(&p, &bytes); printf("ws %d %d\n", st, (int)bytes); } }
  return 0;
}
"""


def test_c_program_against_the_library(lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    libdir = os.path.dirname(api.library_path())
    src, exe = tmp_path / "consumer.c", tmp_path / "consumer"
    src.write_text(_program())
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    "-L", libdir, "-lssfwd", "-Wl,-rpath," + libdir], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    got = dict(line.split(" ", 1) for line in r.stdout.strip().splitlines())
    assert got["null"] == "1 1 1 1 1"
    assert got["ws"] == f"0 {5 * 2 * (2048 + 1) * 4}"
    for kind, cases in (("scan", SCAN), ("conv", CONV), ("tables", TABLES), ("step", STEP)):
        for name, _, status in cases:
            assert got[f"{kind}.{name}"] == str(status), (kind, name, got[f"{kind}.{name}"])


def test_block_rule(lib):
    packed._bind()
    block = lambda *a: lib.ss_head_scan_block(*a, 152)  # noqa: E731
    for tokens in (1, 100, 2048, 65536, 1 << 20):
        for requests in (1, 7, 64):
            for heads in (1, 24, 80):
                for dtype in (api.SS_F32, api.SS_BF16):
                    b = block(tokens, requests, heads, 64, dtype)
                    assert 1 <= b < 1 << 20
                    assert b % (16 if dtype == api.SS_F32 else 128) == 0
    # few heads and one long request: cut; many CTAs without cutting: whole requests
    assert block(65536, 1, 8, 64, api.SS_BF16) < 65536 // 8
    assert block(64 * 2048, 64, 80, 64, api.SS_BF16) >= 2048
    assert block(0, 0, 0, 0, api.SS_BF16) >= 1


def test_operators_need_cuda_tensors():
    t = torch.zeros(2, 2, 8)
    with pytest.raises(RuntimeError, match="CUDA"):
        packed.request_tables(torch.ones(2, dtype=torch.int32), 2)
    with pytest.raises(RuntimeError, match="CUDA"):
        packed.packed_conv1d_fn(torch.zeros(2, 4), torch.zeros(4, 3), None)
    with pytest.raises(RuntimeError, match="CUDA"):
        packed.head_scan_fn(t, t[:, :, 0], torch.zeros(2), t, t, None)
    with pytest.raises(RuntimeError, match="CUDA"):
        packed.head_state_update(torch.zeros(2, 2, 8, 8), t, t[:, :, 0], torch.zeros(2), t, t)


def test_binding_checks_before_any_cuda_call(lib):
    b = packed._bind()
    x, w, st = torch.zeros(2, 4), torch.zeros(4, 3), torch.zeros(2, 4, 2)
    with pytest.raises(TypeError, match="arguments"):
        b.packed_conv1d(x)
    with pytest.raises(TypeError, match="fp32/fp16/bf16"):
        b.packed_conv1d_update(x.double(), st, w, None, None, 0)
    with pytest.raises(TypeError, match="weight"):
        b.packed_conv1d_update(x, st, w.half(), None, None, 0)
    with pytest.raises(TypeError, match="conv_state"):
        b.packed_conv1d_update(x, st[:, :, :1], w, None, None, 0)
    with pytest.raises(ValueError, match="in place"):
        b.packed_conv1d_update(x, torch.zeros(2, 2, 4).transpose(1, 2), w, None, None, 0)
    with pytest.raises(NotImplementedError):
        b.packed_conv1d_update(x.clone().requires_grad_(), st, w, None, None, 0)
    with pytest.raises(TypeError, match="RequestTables"):
        b.packed_conv1d(x, w, b"", None, None, 0)
    h = torch.zeros(2, 2, 8)
    with pytest.raises(TypeError, match="dt"):
        b.head_state_update(torch.zeros(2, 2, 8, 8), h, h[:, :, 0].half(), torch.zeros(2), h, h, None, None, None, False, None)
    with pytest.raises(TypeError, match="slots"):
        b.head_state_update(torch.zeros(2, 2, 8, 8), h, h[:, :, 0], torch.zeros(2), h, h, None, None, None, False,
                            torch.zeros(3, dtype=torch.int32))
