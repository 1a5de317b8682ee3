"""Guard regions around the outputs of the layer operators (test_guard.py's, for
include/ssfwd_layer.h): every output stands in a poisoned buffer with padding after its
rows, as the inputs do, the workspace with a margin on both sides. After the call the view
holds what the oracle has, and every byte outside it the poison. Sizes are ragged: parts of runs, tiles,
channel tiles and groups, rows by TMA, in pairs and in single values, clusters and
segments, warps and CTAs for a row of the norm. Tolerances are test_layer.py's.
"""
import numpy as np
import pytest
import torch

import layer_abi
import state_space_model_03_gb300 as ssm
from oracle import layer as oracle
from test_guard import Guarded
from test_layer import GTOL, STATE_TOL, TOL, TYPES, _close, _gen, _i32, _norm_problem, _packed_problem, _rand, _scan_problem

pytestmark = pytest.mark.gpu


class Buffers:
    """Guarded outputs, inputs and workspaces, with their names."""

    def __init__(self, pad):
        self.pad, self.held = pad, []

    def rows(self, name, shape, dtype):
        return self._hold(name, Guarded(shape, dtype, self.pad))

    def given(self, tensors):
        """Inputs by name, in rows like the outputs'."""
        return {k: v if v is None or v.dim() < 2 else self.rows(k, tuple(v.shape), v.dtype).copy_(v) for k, v in tensors.items()}

    def flat(self, name, shape, dtype=torch.float32):
        return self._hold(name, Guarded(shape, dtype))

    def workspace(self, n):
        return self.flat("workspace", (n,), torch.uint8)

    def _hold(self, name, guarded):
        self.held.append((name, guarded))
        return guarded.view

    def check(self):
        for name, g in self.held:
            assert g.untouched(), name


# (batch, tokens, dim), padding of rows: to 16 bytes, to pairs, to odd places
SCANS = [((2, 100, 37), 3), ((2, 100, 40), 8), ((3, 9, 34), 2), ((1, 1, 1), 1), ((2, 1200, 37), 3), ((1, 1187, 34), 2), ((1, 1153, 40), 0),
         ((2, 1100, 1303), 1), ((2, 1100, 1304), 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,pad", SCANS)
def test_scan(dtype, shape, pad):
    b, n, d = shape
    p = _scan_problem(shape, dtype, ig=n % 2 == 0, seed=n + d)
    g = _gen(1)
    h0, dout, dlast = _rand(g, b, d), _rand(g, *shape, dtype=dtype), _rand(g, b, d)
    o = Buffers(pad)
    sizes = dict(rate=8.0, batch=b, seqlen=n, dim=d) | o.given(p)
    out, last, kept = o.rows("out", shape, dtype), o.flat("last", (b, d)), o.flat("kept", (b, -(-n // 64), d))
    a = layer_abi.params("gated_scan", dtype, **sizes, initial_state=h0, out=out, last_state=last, kept=kept)
    assert layer_abi.run("gated_scan", a, o.workspace) == 0
    want, wlast = oracle.gated_scan(**p, initial_state=h0)
    _close(out, want, TOL[dtype], "out")
    _close(last, wlast, STATE_TOL, "last")
    _close(kept, np.concatenate([oracle.f64(h0)[:, None], want[:, 63:n - 1:64]], 1), STATE_TOL, "kept")
    grads = {k: o.rows(k, shape, dtype) for k in ("dx", "dgate", "dinput_gate") if k[1:] in p}
    grads |= {"ddecay": o.flat("ddecay", (d,)), "dinitial_state": o.flat("dinitial_state", (b, d))}
    a = layer_abi.params("gated_scan_bwd", dtype, **sizes, **o.given({"dout": dout}), dlast=dlast, kept=kept, **grads)
    assert layer_abi.run("gated_scan_bwd", a, o.workspace) == 0
    ref = oracle.gated_scan_bwd(dout, dlast, **p, initial_state=h0)
    for k, v in grads.items():
        _close(v, ref[k[1:]], GTOL[v.dtype], k)
    o.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,tail,dim,pad", [([3, 0, 70, 1, 33], 5, 37, 3), ([600, 1, 700], 9, 40, 8), ([600, 1, 700], 0, 33, 1), ([1500], 7, 1303, 1)])
def test_packed_and_steps(dtype, lengths, tail, dim, pad):
    p, t, st = _packed_problem(lengths, dim, dtype, dim != 33, tail, seed=dim)
    n, r = sum(lengths) + tail, len(lengths)
    o = Buffers(pad)
    state = o.rows("state", tuple(st.shape), torch.float32).copy_(st)
    out = o.rows("out", (n, dim), dtype)
    tables = ssm.request_tables(_i32(lengths), n, **t)
    a = layer_abi.params("packed_gated_scan", dtype, rate=8.0, dim=dim, slots=st.shape[0], **o.given(p), state=state, out=out)
    a.tables = layer_abi.packed_tables(tables)
    assert layer_abi.run("packed_gated_scan", a, o.workspace) == 0
    want, wst = oracle.packed_gated_scan(**p, lengths=lengths, state=st, **t)
    _close(out, want, TOL[dtype], "out")
    _close(state, wst, STATE_TOL, "state")
    one = o.rows("one", (r, dim), dtype)
    q = {k: v if k == "decay" else v[:r].contiguous() for k, v in p.items()}
    a = layer_abi.params("gated_state_update", dtype, rate=8.0, requests=r, dim=dim, slots=st.shape[0], **o.given(q), state=state, slot_map=t["slots"], out=one)
    before = state.cpu()
    assert layer_abi.run("gated_state_update", a) == 0
    want, wst = oracle.packed_gated_scan(**q, lengths=[1] * r, state=before, slots=t["slots"], context=[1] * r)
    _close(one, want, TOL[dtype], "one")
    _close(state, wst, STATE_TOL, "state after a step")
    o.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", ["none", "same", "fp32"])
@pytest.mark.parametrize("shape,pad", [((3, 1), 1), ((70, 37), 3), ((70, 40), 8), ((9, 769), 1), ((640, 264), 8), ((5, 1032), 16), ((2, 8199), 1), ((2, 8200), 8)])
def test_norm(dtype, residual, shape, pad):
    rows, d = shape
    p = _norm_problem(shape, dtype, residual, seed=d)
    kept = dtype if p["residual"] is None else p["residual"].dtype
    g = _gen(2)
    dout, dsum = _rand(g, *shape, dtype=dtype), _rand(g, *shape, dtype=kept)
    o = Buffers(pad)
    q = o.given(p)
    more = {} if p["residual"] is None else {"residual": q["residual"], "sum": o.rows("sum", shape, kept)}
    sizes = dict(residual_dtype=layer_abi.DTYPES[kept], weight_dtype=0, rows=rows, dim=d)
    out, rstd = o.rows("out", shape, dtype), o.flat("rstd", (rows,))
    a = layer_abi.params("rms_norm", dtype, **sizes, eps=1e-5, x=q["x"], weight=p["weight"], **more, out=out, rstd=rstd)
    assert layer_abi.run("rms_norm", a) == 0
    want, s = oracle.rms_norm(**p)
    _close(out, want, TOL[dtype], "out")
    _close(rstd, 1 / np.sqrt((s * s).mean(-1) + 1e-5), STATE_TOL, "rstd")
    if more:
        _close(more["sum"], s, torch.finfo(kept).eps / 2, "sum")
    total = more.get("sum", q["x"])
    grads = {"dx": o.rows("dx", shape, dtype), "dresidual": o.rows("dresidual", shape, kept), "dweight": o.flat("dweight", (d,))}
    a = layer_abi.params("rms_norm_bwd", dtype, **sizes, **o.given({"dout": dout, "dsum": dsum}), sum=total, weight=p["weight"], rstd=rstd, **grads)
    assert layer_abi.run("rms_norm_bwd", a, o.workspace) == 0
    ds, dw = oracle.rms_norm_bwd(dout, dsum, torch.zeros_like(p["x"]), p["weight"], total)
    # one channel: the terms cancel to eps, each off by 2^-21 of itself (test_layer.py)
    slack = 2.0**-21 * np.linalg.norm(oracle.f64(dout) * oracle.f64(p["weight"]) / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-5))
    _close(grads["dx"], ds, GTOL[dtype], "dx", slack)
    _close(grads["dresidual"], ds, GTOL[kept], "dresidual", slack)
    _close(grads["dweight"], dw, GTOL[torch.float32], "dweight")
    o.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("shape,pad", [((3, 1), 1), ((70, 37), 3), ((70, 40), 8), ((9, 769), 1), ((640, 264), 8), ((5, 1032), 16), ((2, 8199), 1), ((2, 8200), 8)])
def test_quant(dtype, group, e8m0, shape, pad):
    """As test_layer.py's: scales off by 3e-6, values by half a step of e4m3."""
    rows, d = shape
    p = _norm_problem(shape, dtype, "same", seed=d)
    o = Buffers(pad)
    out, total = o.rows("out", shape, torch.uint8), o.rows("sum", shape, dtype)
    scale = o.flat("scale", (rows, -(-d // (group or d))), torch.uint8 if e8m0 else torch.float32)
    kind = layer_abi.DTYPES[dtype]
    a = layer_abi.params("rms_norm_quant", dtype, residual_dtype=kind, weight_dtype=0, eps=1e-5, scale_type=int(e8m0), rows=rows, dim=d, group=group,
                         **o.given(p), out=out, scale=scale, sum=total)
    assert layer_abi.run("rms_norm_quant", a) == 0
    v, s = oracle.rms_norm(**p)
    _close(total, s, torch.finfo(dtype).eps / 2, "sum")
    scale = (scale.view(torch.float8_e8m0fnu) if e8m0 else scale).float().double().cpu().numpy()
    exact = oracle.scales(v, group, False)
    if e8m0:
        assert (scale >= exact * (1 - 3e-6)).all() and (scale < 2 * exact * (1 + 3e-6)).all()
    else:
        np.testing.assert_allclose(scale, exact, rtol=3e-6)
    wide = np.repeat(scale, group or d, -1)[..., :d]
    off = np.abs(out.contiguous().view(torch.float8_e4m3fn).float().double().cpu().numpy() * wide - v)
    assert (off <= np.maximum(2.0**-4 * np.abs(v), 2.0**-10 * wide) * (1 + 1e-5) + 3e-6 * np.abs(v)).all()
    o.check()
