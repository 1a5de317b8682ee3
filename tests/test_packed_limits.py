"""Packed operators on the GPU at the edges of what their types hold, against the
fp64 oracle (oracle/packed.py). Tolerances of norms are those of test_packed.py;
those of single elements are derived where they stand.
"""
import numpy as np
import pytest
import torch

import state_space_model_03_gb300 as ssm
from oracle import packed as oracle
from test_packed import TYPES, _i32, _run_scan, _scan_problem

pytestmark = pytest.mark.gpu

HALF = [torch.bfloat16, torch.float16]


# ---- large inputs and steps in requests of several blocks ----

@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("block", [128, 256, 384, 4096])
@pytest.mark.parametrize("headdim,dstate", [(64, 64), (128, 128)])
def test_large_inputs_do_not_depend_on_the_block(dtype, block, headdim, dstate):
    """|x| from 4100 to 60000 at the tokens with the largest steps, which end blocks: states of a
    few thousand and outputs of some hundred, far below 65504, whatever the block."""
    n = 700
    p, t, st = _scan_problem([n], 2, 1, headdim, dstate, dtype, z=False, dt32=True, seed=21, fused=False)
    p |= {"dt_bias": None, "dt_softplus": False, "D": None}
    p["dt"] = p["dt"].abs() * 0.005
    at = torch.arange(127, n, 128, device="cuda")
    p["dt"][at] = 0.0987
    size = torch.linspace(4100, 60000, headdim, device="cuda") * (1 - 2 * (torch.arange(headdim, device="cuda") % 2))
    p["x"][at] = size.to(dtype)
    p["B"] *= 0.25
    p["C"] *= 0.01
    t["context"].fill_(1)
    _run_scan(p, t, st, [n], block)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [128, 4096])
def test_growing_states(dtype, block):
    """A > 0: the weights of a block's first tokens are the largest."""
    n = 260
    p, t, st = _scan_problem([n], 2, 1, 64, 64, dtype, z=False, dt32=True, seed=22, fused=False)
    p |= {"dt_bias": None, "dt_softplus": False, "D": None}
    p["A"] = torch.tensor([1.5, 0.3], device="cuda")
    p["dt"] = p["dt"].abs() * 0.02
    p["x"] *= 100
    p["C"] *= 0.02
    t["context"].fill_(1)
    _run_scan(p, t, st, [n], block)


# ---- steps that leave nothing of what was before ----

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [128, 4096])
@pytest.mark.parametrize("A", [-3e38, -float("inf")])
def test_steps_that_end_everything(dtype, block, A):
    """dt A past the largest number: a decay of 0, as token by token, not a difference of infinities."""
    n = 300
    p, t, st = _scan_problem([n], 2, 1, 64, 64, dtype, z=False, dt32=True, seed=23)
    p |= {"dt_bias": None, "dt_softplus": False}
    p["A"] = torch.tensor([A, -2.0], device="cuda")
    p["dt"] = 1 + p["dt"].abs()
    t["context"].fill_(1)
    _run_scan(p, t, st, [n], block)


@pytest.mark.parametrize("block", [128, 4096])
@pytest.mark.parametrize("step", [1e3, 1e6])
def test_ordinary_steps_after_huge_ones(block, step):
    """One huge step in each 32 tokens (with nothing to add) leaves the decays of those after it exact
    to bf16: the rounding of a prefix that holds it would be as large as the steps themselves."""
    n = 300
    p, t, st = _scan_problem([n], 2, 1, 64, 64, torch.bfloat16, z=False, dt32=True, seed=24, fused=False)
    p |= {"dt_bias": None, "dt_softplus": False, "D": None}
    p["dt"] = p["dt"].abs() * 0.05
    at = torch.arange(3, n, 32, device="cuda")
    p["dt"][at] = step
    p["x"][at] = 0
    p["B"][at] = 0
    t["context"].fill_(1)
    _run_scan(p, t, st, [n], block)


# ---- silu, element by element ----

# Half a unit of the last place is at most 2^-8, 2^-11 and 2^-24 of the value (in fp16 at least 2^-25).
# silu in fp32 adds the rounding of its exponent (58 in log2 at z = -40, to 2^-24 of it and of log2 e),
# of ex2 and of rcp (2^-22 each): below 5e-6.
ELEMENT = {torch.bfloat16: 2.0 ** -8 + 5e-6, torch.float16: 2.0 ** -11 + 5e-6, torch.float32: 5e-6}


def _gates(dtype):
    z = torch.linspace(-12.0 if dtype == torch.float16 else -40.0, 10.0, 2048).to(dtype)
    return z.cuda(), oracle.silu(z.double().numpy())


def _elements(got, want, dtype):
    off = np.abs(got.double().cpu().numpy() - want)
    bound = ELEMENT[dtype] * np.abs(want) + (2.0 ** -25 if dtype == torch.float16 else 0)
    worst = int(np.argmax(off - bound))
    assert (off <= bound).all(), (worst, got.flatten()[worst].item(), want.flat[worst])


@pytest.mark.parametrize("dtype", TYPES)
def test_silu_of_the_convolutions(dtype):
    z, want = _gates(dtype)
    x, w = z.view(64, 32), torch.tensor([0.0, 1.0], device="cuda").repeat(32, 1)
    tables = ssm.request_tables(_i32([64]), 64)
    _elements(ssm.packed_conv1d_fn(x, w, tables, activation="silu"), want.reshape(64, 32), dtype)
    st = torch.zeros(64, 32, 1, dtype=dtype, device="cuda")
    _elements(ssm.packed_conv1d_update(x, st, w, activation="silu"), want.reshape(64, 32), dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_silu_of_the_gate(dtype):
    """x = D = 1 and B = 0 leave silu(z); the prompt's and the step's agree to their rounding."""
    z, want = _gates(dtype)
    z, want = z.view(32, 1, 64), want.reshape(32, 1, 64)
    x, bc = torch.ones_like(z), torch.zeros(32, 1, 64, dtype=dtype, device="cuda")
    dt, A, D = torch.zeros(32, 1, dtype=dtype, device="cuda"), -torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
    _elements(ssm.head_scan_fn(x, dt, A, bc, bc, ssm.request_tables(_i32([32]), 32), D=D, z=z), want, dtype)
    st = torch.zeros(32, 1, 64, 64, device="cuda")
    _elements(ssm.head_state_update(st, x, dt, A, bc, bc, D=D, z=z), want, dtype)


# ---- number of requests ----

TABLES_IN_A_FRESH_PROCESS = """
import torch
import state_space_model_03_gb300 as ssm
from oracle import packed as oracle
for n in (4084, 4085, 4090, 4095, 4096, 16384):
    lengths = torch.arange(n, dtype=torch.int32, device="cuda") % 3
    t = ssm.request_tables(lengths, n, block=2)
    want = oracle.request_tables(lengths, n, block=2)
    for k, v in want.items():
        assert (getattr(t, k).cpu().numpy() == v).all(), (n, k)
print("tables ok")
"""


def test_tables_of_any_number_of_requests_in_a_fresh_process():
    """Numbers whose tables just pass the shared memory that needs no request, before any larger call."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", TABLES_IN_A_FRESH_PROCESS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "tables ok" in r.stdout, r.stderr[-2000:]


# ---- caches under autograd ----

def test_caches_count_their_versions():
    """A cache that autograd saved is known to have changed; one made in inference mode still works."""
    p, t, st = _scan_problem([1] * 3, 2, 1, 16, 16, torch.float32, seed=25)
    tables = ssm.request_tables(_i32([1, 1, 1]), 3, context=_i32([1, 1, 1]))
    x, w = torch.randn(3, 8, device="cuda"), torch.randn(8, 4, device="cuda")
    win = torch.zeros(3, 8, 3, device="cuda")
    calls = [(st, lambda s: ssm.head_scan_fn(**p, tables=tables, state=s)),
             (st, lambda s: ssm.head_state_update(s, **p)),
             (win, lambda s: ssm.packed_conv1d_fn(x, w, tables, conv_state=s)),
             (win, lambda s: ssm.packed_conv1d_update(x, s, w))]
    for cache, call in calls:
        before = cache._version
        call(cache)
        assert cache._version > before
        factor = torch.ones((), device="cuda", requires_grad=True)
        y = (cache * factor).sum()
        call(cache)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        with torch.inference_mode():
            frozen = cache.clone()
        call(frozen)


# ---- blocks of many chunks, and other forms in several blocks ----

@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("block", [384, 512, 640, 1100])
@pytest.mark.parametrize("headdim,dstate", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_blocks_of_many_chunks(dtype, block, headdim, dstate):
    """Summaries of 3 to 9 chunks, the last of them partial, in requests of several blocks."""
    lengths = [3 * block + 37, 5, 2 * block, block + 1]
    p, t, st = _scan_problem(lengths, 3, 1, headdim, dstate, dtype, z=block == 512, pad=2, seed=block, A_max=2.0)
    p["dt_bias"] = p["dt_bias"] - 2  # states that last for hundreds of tokens
    t["context"].fill_(1)
    _run_scan(p, t, st, lengths, block)


@pytest.mark.parametrize("dtype", HALF)
def test_the_blocks_that_the_rule_gives(dtype):
    """One long request of a few heads, cut as head_scan_block says."""
    n = 9001
    block = ssm.head_scan_block(n, 1, 4, 64, dtype=dtype)
    assert 128 < block < n
    p, t, st = _scan_problem([n], 4, 2, 64, 64, dtype, z=False, seed=26, A_max=2.0)
    p["dt_bias"] = p["dt_bias"] - 2
    t["context"].fill_(1)
    _run_scan(p, t, st, [n], block)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("block", [16, 50, 128])
@pytest.mark.parametrize("headdim,dstate", [(200, 24), (33, 256)])
def test_large_heads_and_states_in_several_blocks(dtype, block, headdim, dstate):
    """The token-by-token form for 16-bit operands."""
    lengths = [70, 0, 1, 129, 3 * block + 5]
    p, t, st = _scan_problem(lengths, 2, 1, headdim, dstate, dtype, pad=3, seed=block)
    t["context"].fill_(1)
    _run_scan(p, t, st, lengths, block)
