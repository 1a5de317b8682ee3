"""The layer operators where a CTA goes on for many rounds, against the fp64 oracle.

Clusters have 8 CTAs at most, fewer where more than 95 (16 bits) or 57 (fp32) units of
32 channels of a sequence share 152 SMs, and none from 381 (229) on; below 40 units long
sequences go in segments. A CTA's places for the maps of its cluster are two, so the third round
is the first that writes one again. The norm's CTAs start again at the first row that no other
has once there are more rows than 16 warps by 152 SMs (short rows) or 2048 threads an SM (a
CTA a row) hold. Tolerances are test_layer.py's.
"""
import numpy as np
import pytest
import torch

import state_space_model_03_gb300 as ssm
from oracle import layer as oracle
from test_layer import (GTOL, STATE_TOL, TOL, TYPES, _close, _gen, _norm_problem, _packed_problem, _rand, _run_packed, _scan_problem)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [
    # 41 units in clusters of 8, four rounds: rows by TMA, in pairs, in single values
    (1, 1600, 1304), (1, 1590, 1302), (1, 1601, 1301),
    # 120 units in clusters of 6 (fp32: 3), four rounds (seven), the last with an empty tile
    (3, 1300, 1280),
    # 300 units in pairs of CTAs, three rounds (fp32: by themselves, six tiles each)
    (10, 330, 960),
    # 384 units by themselves, eight tiles each
    (48, 450, 256),
])
def test_scan_and_gradients(dtype, shape):
    p = _scan_problem(shape, dtype, ig=shape[0] != 3, seed=sum(shape))
    g = _gen(7)
    h0, dout, dlast = _rand(g, shape[0], shape[2]), _rand(g, *shape, dtype=dtype), _rand(g, shape[0], shape[2])
    leaves = {k: v.clone().requires_grad_() for k, v in (p | {"initial_state": h0}).items()}
    out, last = ssm.gated_scan_fn(**leaves, return_last_state=True)
    got = dict(zip(leaves, torch.autograd.grad((out, last), list(leaves.values()), (dout, dlast))))
    want, wlast = oracle.gated_scan(**p, initial_state=h0)
    _close(out, want, TOL[dtype], "out")
    _close(last, wlast, STATE_TOL, "last")
    ref = oracle.gated_scan_bwd(dout, dlast, **p, initial_state=h0)
    for k, v in got.items():
        _close(v, ref[k], GTOL[v.dtype], k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [1304, 1302, 1301])
@pytest.mark.parametrize("lengths,pad", [
    # 30 tiles, four rounds: requests within a tile, of several rounds, that end where a tile or a round does
    ([900, 0, 1, 507, 128, 63, 129, 3, 64, 64], 37),
    ([1800], 0),
    ([1] * 300 + [800, 1, 500], 0),
])
def test_packed_in_clusters(dtype, dim, lengths, pad):
    p, t, st = _packed_problem(lengths, dim, dtype, dim != 1302, pad, seed=dim)
    _run_packed(p, t, st, lengths, dtype)


# short rows, a warp each; a CTA each, with the weight kept and without; single values of both
ROWS = [(20500, 40), (20100, 133), (10500, 520), (4100, 2560), (5000, 769), (1600, 10248)]


@pytest.mark.parametrize("dtype,residual", [(torch.bfloat16, "fp32"), (torch.float16, "none"), (torch.float32, "same")])
@pytest.mark.parametrize("shape", ROWS)
def test_norm_and_gradients(dtype, residual, shape):
    p = _norm_problem(shape, dtype, residual, seed=shape[0])
    g = _gen(8)
    dout = _rand(g, *shape, dtype=dtype)
    dsum = None if p["residual"] is None else _rand(g, *shape, dtype=p["residual"].dtype)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items() if v is not None}
    got = ssm.rms_norm_fn(**leaves, prenorm=dsum is not None)
    grads = dict(zip(leaves, torch.autograd.grad(got, list(leaves.values()), dout if dsum is None else (dout, dsum))))
    out, kept = (got, p["x"]) if dsum is None else got
    want, s = oracle.rms_norm(**p)
    _close(out, want, TOL[dtype], "out")
    _close(kept, s, torch.finfo(kept.dtype).eps / 2, "sum")
    assert torch.equal(ssm.rms_norm_fn(**p), out)
    ds, dw = oracle.rms_norm_bwd(dout, dsum, torch.zeros_like(p["x"]), p["weight"], kept.detach())
    _close(grads["x"], ds, GTOL[dtype], "x")
    if dsum is not None:
        _close(grads["residual"], ds, GTOL[dsum.dtype], "residual")
    _close(grads["weight"], dw, GTOL[torch.float32], "weight")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", ROWS)
@pytest.mark.parametrize("group", [None, 32, 128])
@pytest.mark.parametrize("e8m0", [False, True])
def test_quant(dtype, shape, group, e8m0):
    """As test_layer.py's: scales off by 3e-6, values by half a step of e4m3."""
    p = _norm_problem(shape, dtype, "same", seed=shape[1])
    v, s = oracle.rms_norm(**p)
    q, scale, kept = ssm.rms_norm_quant_fn(**p, prenorm=True, group_size=group, scale_dtype=torch.float8_e8m0fnu if e8m0 else torch.float32)
    _close(kept, s, torch.finfo(dtype).eps / 2)
    q, scale = q.float().double().cpu().numpy(), scale.float().double().cpu().numpy()
    exact = oracle.scales(v, group, False)
    if e8m0:
        assert (np.exp2(np.round(np.log2(scale))) == scale).all()
        assert (scale >= exact * (1 - 3e-6)).all() and (scale < 2 * exact * (1 + 3e-6)).all()
    else:
        np.testing.assert_allclose(scale, exact, rtol=3e-6)
    wide = np.repeat(scale, group or shape[-1], -1)[..., :shape[-1]]
    off = np.abs(q * wide - v)
    assert (off <= np.maximum(2.0**-4 * np.abs(v), 2.0**-10 * wide) * (1 + 1e-5) + 3e-6 * np.abs(v)).all()
