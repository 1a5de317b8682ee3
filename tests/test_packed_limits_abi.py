"""Limits of the packed operators that are checked on the host (no CUDA call is made)."""
import os
import shutil
import subprocess

import pytest
import torch
import torch.autograd.forward_ad as fwad

from state_space_model_03_gb300 import api, packed
from state_space_model_03_gb300 import build as ssbuild
from test_packed_abi import ROOT, _program


@pytest.fixture(scope="module")
def lib():
    ssbuild.build()
    return api.load_library()


# A scan whose blocks are many and short, with heads of `headdim` values: x, dt, B and C
# are broadcast, so that only out has a large span.
MANY = """
  p.heads = %d; p.headdim = %d; p.dstate = %d; p.ngroups = 1; p.dtype = %s; p.state = 0;
  p.tables.tokens = %d; p.tables.block = %d; p.tables.max_blocks = %d / %d + 3;
  p.x_stride[0] = p.x_stride[1] = %d; p.dt_stride[0] = p.dt_stride[1] = p.B_stride[0] = p.C_stride[0] = 0;
  p.out = (void *)((uintptr_t)1 << 46); p.out_stride[1] = %d; p.out_stride[0] = (int64_t)%d * %d;
  p.workspace = (void *)((uintptr_t)1 << 45); p.workspace_bytes = INT64_MAX;
"""


def _many(heads, headdim, dstate, dtype, tokens, block, x_stride=0):
    return MANY % (heads, headdim, dstate, dtype, tokens, block, tokens, block, x_stride, headdim, heads, headdim)


GRIDS = [
    # name, problem, status
    ("small", _many(8, 64, 32, "SS_F32", 1 << 12, 16), 0),
    ("carry", _many(8192, 1, 1, "SS_F32", 1 << 18, 1), 7),           # 2^31 CTAs of the carry
    ("carry_fits", _many(8192, 1, 1, "SS_F32", (1 << 18) - 1, 1), 0),
    ("carry_of_pieces", _many(8192, 256, 256, "SS_F32", 1 << 12, 1), 7),
    ("tensor_cores", _many(8192, 128, 128, "SS_BF16", 1 << 18, 1), 7),
    ("tensor_cores_one_block", _many(8192, 128, 128, "SS_BF16", 1 << 18, 1 << 18), 0),
]


def test_grids_are_checked_before_anything_is_enqueued(lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    text = _program()
    body = "int main(void) {\n  int64_t bytes;\n  { ss_packed_conv1d_params c = conv(); ss_request_tables_params t = tab();" \
        " ss_head_state_update_params s = step(); (void)c; (void)t; (void)s; }\n"
    for name, change, _ in GRIDS:
        body += f'  {{ ss_head_scan_params p = scan(); {change} printf("{name} %d %d\\n", ss_head_scan_validate(&p),' \
            " ss_head_scan_workspace_size(&p, &bytes)); }\n"
    src, exe = tmp_path / "grids.c", tmp_path / "grids"
    src.write_text(text[:text.index("int main(void)")] + body + "  return 0;\n}\n")
    libdir = os.path.dirname(api.library_path())
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    "-L", libdir, "-lssfwd", "-Wl,-rpath," + libdir], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    got = dict(line.split(" ", 1) for line in r.stdout.strip().splitlines())
    for name, _, status in GRIDS:
        assert got[name] == f"{status} {status}", (name, got[name])


class _Undecided:
    def __bool__(self):
        raise ValueError("neither")


def test_flags_that_are_neither_true_nor_false(lib):
    b = packed._bind()
    h = torch.zeros(2, 2, 8)
    with pytest.raises(ValueError, match="neither"):
        b.head_state_update(torch.zeros(2, 2, 8, 8), h, h[:, :, 0], torch.zeros(2), h, h, None, None, None, _Undecided(), None)
    with pytest.raises(ValueError, match="neither"):
        b.head_scan(h, h[:, :, 0], torch.zeros(2), h, h, b"", None, None, None, _Undecided(), None)


def test_forward_mode_tangents_are_refused(lib):
    b = packed._bind()
    h, x, w = torch.zeros(2, 2, 8), torch.zeros(2, 4), torch.zeros(4, 3)
    with fwad.dual_level():
        with pytest.raises(NotImplementedError):
            b.head_state_update(torch.zeros(2, 2, 8, 8), fwad.make_dual(h, torch.ones_like(h)), h[:, :, 0], torch.zeros(2), h, h,
                                None, None, None, False, None)
        with pytest.raises(NotImplementedError):
            b.packed_conv1d_update(fwad.make_dual(x, torch.ones_like(x)), torch.zeros(2, 4, 2), w, None, None, 0)
