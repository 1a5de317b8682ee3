"""Waits of the gated recurrence that run out, on the GPU, without a hang or a fault.

SSFWD_TEST_STALL=<k>: the copies of every CTA's round k are asked of their barrier and never
made, as if lost. SSFWD_TEST_STALL_MAPS=<k>: what the CTAs of a cluster send one another in round k.
Waits then give up after 1024 tries of at most 1 us. The kernels set the error word,
ask nothing more of a barrier that waits, run on and return; the context stays usable.
"""
import time

import pytest
import torch

import state_space_model_03_gb300 as ssm
from state_space_model_03_gb300 import api
from test_layer import _gen, _i32, _packed_problem, _rand, _scan_problem

pytestmark = pytest.mark.gpu

COPY, MAPS = "SSFWD_TEST_STALL", "SSFWD_TEST_STALL_MAPS"
# eight tiles a CTA; four rounds of clusters of 8; segments of four tiles
ALONE, CLUSTERS, SEGMENTS = (48, 450, 256), (1, 1600, 1304), (1, 24600, 64)


def _stalled(monkeypatch, name, k, call):
    """The error word after the call, which returns."""
    api.device_error(clear=True)
    monkeypatch.setenv(name, str(k))
    start = time.time()
    call()
    torch.cuda.synchronize()
    monkeypatch.delenv(name)
    assert time.time() - start < 30
    return api.device_error(clear=True)


CASES = [(COPY, k, shape, 1) for shape in (ALONE, CLUSTERS, SEGMENTS) for k in (0, 1, 2)] + [(MAPS, k, CLUSTERS, 3) for k in (0, 1, 2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name,k,shape,code", CASES)
def test_dense(dtype, name, k, shape, code, monkeypatch):
    p = _scan_problem(shape, dtype, seed=k)
    dout = _rand(_gen(1), *shape, dtype=dtype)
    leaves = {n: v.requires_grad_() for n, v in p.items()}

    def forward():
        return ssm.gated_scan_fn(**leaves)

    out = forward()
    want = [out.detach(), *torch.autograd.grad(out, list(leaves.values()), dout, retain_graph=True)]
    assert _stalled(monkeypatch, name, k, forward) == code
    assert _stalled(monkeypatch, name, k, lambda: torch.autograd.grad(out, list(leaves.values()), dout, retain_graph=True)) == code
    again = forward()
    got = [again.detach(), *torch.autograd.grad(again, list(leaves.values()), dout)]
    torch.cuda.synchronize()
    assert api.device_error() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name,k,dim,code", [(COPY, 0, 1304, 1), (COPY, 2, 1304, 1), (COPY, 1, 64, 1), (MAPS, 1, 1304, 3)])
def test_packed(name, k, dim, code, monkeypatch):
    lengths = [900, 0, 1, 507, 128, 63, 129, 3, 64, 64] if dim == 1304 else [20000, 1, 4000]
    p, t, st = _packed_problem(lengths, dim, torch.bfloat16, seed=k)
    tables = ssm.request_tables(_i32(lengths), sum(lengths), **t)
    keep = st.clone()
    want = ssm.packed_gated_scan_fn(**p, tables=tables, state=st)
    after = st.clone()
    st.copy_(keep)
    assert _stalled(monkeypatch, name, k, lambda: ssm.packed_gated_scan_fn(**p, tables=tables, state=st)) == code
    st.copy_(keep)
    assert torch.equal(ssm.packed_gated_scan_fn(**p, tables=tables, state=st), want) and torch.equal(st, after)
    assert api.device_error() == 0
