"""The layer operators at the ends of sequences, rows and types, against the fp64 oracle.
Tolerances are test_layer.py's."""
import numpy as np
import pytest
import torch

import layer_abi
import state_space_model_03_gb300 as ssm
from oracle import layer as oracle
from test_layer import GTOL, STATE_TOL, TOL, TYPES, _close, _gen, _i32, _norm_problem, _packed_problem, _rand, _scan_problem

pytestmark = pytest.mark.gpu


# ---- the last token ----

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("n,d", [
    # a part of a run of 8 tokens, a tile, one token more, a cluster of a CTA a tile, one with tiles past the end, segments
    (1, 8), (5, 8), (8, 33), (64, 40), (65, 40), (300, 70), (1100, 1304), (1090, 1301), (1200, 48), (1216, 33),
])
def test_last_state_is_what_the_last_token_leaves(dtype, bad, n, d):
    """Infinite there too: no token comes after it, whatever is left of its tile and of its cluster's."""
    p = _scan_problem((2, n, d), dtype, seed=n + d)
    clean, clean_last = ssm.gated_scan_fn(**p, return_last_state=True)
    at = (1, n - 1, d // 2)
    p["x"][at] = bad
    out, last = ssm.gated_scan_fn(**p, return_last_state=True)
    want = torch.tensor(bad, device="cuda")
    torch.testing.assert_close(out[at].float(), want, equal_nan=True)
    torch.testing.assert_close(last[1, d // 2], want, equal_nan=True)
    out[at] = clean[at]
    last[1, d // 2] = clean_last[1, d // 2]
    assert torch.equal(out, clean) and torch.equal(last, clean_last)


@pytest.mark.parametrize("n", [700, 1300])  # clusters; segments
def test_gradients_beside_nan(n):
    """Channels with a NaN or an infinity in a sequence leave the gradients of the other channels and sequences alone."""
    shape = (3, n, 70)
    p = _scan_problem(shape, torch.bfloat16, seed=n)
    dout = _rand(_gen(4), *shape, dtype=torch.bfloat16)

    def grads(p):
        leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
        return dict(zip(leaves, torch.autograd.grad(ssm.gated_scan_fn(**leaves), list(leaves.values()), dout)))

    clean = grads(p)
    p["x"][0, :, 7] = float("nan")
    p["gate"][1, 100:, 8] = float("nan")
    p["x"][2, 50, 9] = float("inf")
    got = grads(p)
    same = torch.ones(shape, dtype=torch.bool, device="cuda")
    same[0, :, 7] = same[1, :, 8] = same[2, :, 9] = False
    for k in ("x", "gate", "input_gate"):
        assert torch.equal(got[k][same], clean[k][same]), k
    others = [c for c in range(70) if c not in (7, 8, 9)]
    assert torch.equal(got["decay"][others], clean["decay"][others])


# ---- odd widths in rows of 16 bytes ----

def _padded(t, step):
    """t in rows `step` apart that end with the buffer, NaN between them."""
    *outer, n, d = t.shape
    rows = int(np.prod(outer)) * n
    flat = torch.full(((rows - 1) * step + d,), float("nan"), dtype=t.dtype, device="cuda")
    strides = (n * step, step, 1)[-t.dim():]
    return flat.as_strided(t.shape, strides).copy_(t)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", [(1200, 333), (1153, 33), (1100, 1)])
def test_odd_widths_in_rows_of_16_bytes(dtype, n, d):
    """Rows that start on 16 bytes, of an odd number of channels, in segments: nothing beyond a row's last channel counts
    or is written."""
    step = (d + 8) // 8 * 8
    p = _scan_problem((2, n, d), dtype, seed=n)
    dout = _rand(_gen(3), 2, n, d, dtype=dtype)
    q = {k: v if k == "decay" else _padded(v, step) for k, v in p.items()}
    outs = {k: _padded(torch.zeros_like(p["x"]), step) for k in ("out", "dx", "dgate", "dinput_gate")}
    f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    last, kept, ddecay, dinit = f32(2, d), f32(2, -(-n // 64), d), f32(d), f32(2, d)
    sizes = dict(rate=8.0, batch=2, seqlen=n, dim=d)
    assert layer_abi.run("gated_scan", layer_abi.params("gated_scan", dtype, **sizes, **q, out=outs["out"], last_state=last, kept=kept)) == 0
    want, wlast = oracle.gated_scan(**p)
    _close(outs["out"], want, TOL[dtype], "out")
    _close(last, wlast, STATE_TOL, "last")
    grads = {k: outs[k] for k in ("dx", "dgate", "dinput_gate")} | {"ddecay": ddecay, "dinitial_state": dinit}
    args = sizes | q | {"dout": _padded(dout, step), "kept": kept}
    assert layer_abi.run("gated_scan_bwd", layer_abi.params("gated_scan_bwd", dtype, **args, **grads)) == 0
    ref = oracle.gated_scan_bwd(dout, None, **p)
    for k, v in grads.items():
        _close(v, ref[k[1:]], GTOL[v.dtype], k)
    for v in outs.values():
        flat = torch.empty(0, dtype=dtype, device="cuda").set_(v.untyped_storage())
        assert int(torch.isnan(flat).sum()) == (2 * n - 1) * (step - d)
    # the decay's gradient alone, from Python: nothing is written in rows
    leaf = p["decay"].clone().requires_grad_()
    got, = torch.autograd.grad(ssm.gated_scan_fn(**(q | {"decay": leaf})), leaf, args["dout"])
    _close(got, ref["decay"], GTOL[got.dtype])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [333, 33])
def test_packed_odd_widths_in_rows_of_16_bytes(dtype, dim):
    lengths = [500, 3, 700, 64, 200]
    n, step = sum(lengths), (dim + 8) // 8 * 8
    p, t, st = _packed_problem(lengths, dim, dtype, seed=dim)
    want, wst = oracle.packed_gated_scan(**p, lengths=lengths, state=st, **t)
    tables = ssm.request_tables(_i32(lengths), n, **t)
    q = {k: v if k == "decay" else _padded(v, step) for k, v in p.items()}
    out = _padded(torch.zeros_like(p["x"]), step)
    a = layer_abi.params("packed_gated_scan", dtype, rate=8.0, dim=dim, slots=st.shape[0], **q, state=st, out=out)
    a.tables = layer_abi.packed_tables(tables)
    assert layer_abi.run("packed_gated_scan", a) == 0
    _close(out, want, TOL[dtype], "out")
    _close(st, wst, STATE_TOL, "state")


# ---- packed segments ----

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("times", [1, 8])  # segments of one tile, of two
def test_packed_neighbours_do_not_leak_over_segments(dtype, bad, times):
    """test_layer.py's, over segments: a bad request that crosses their ends, good ones that start in the segment that it
    ends in and go on into the next, one that starts where a segment does, and bad padding of whole segments."""
    lengths = [times * v for v in (50, 300, 150, 12, 128, 60, 600)]
    total, pad = sum(lengths), times * 300
    p, t, st = _packed_problem(lengths, 70, dtype, pad=pad, seed=21, spare=1)
    t["context"] = _i32([3, 0, 5, 0, 4, 0, 0])
    tables = ssm.request_tables(_i32(lengths), total + pad, **t)
    st2 = st.clone()
    clean = ssm.packed_gated_scan_fn(**p, tables=tables, state=st2)
    want, wst = oracle.packed_gated_scan(**p, lengths=lengths, state=st, **t)
    _close(clean, want, TOL[dtype])
    _close(st2, wst, STATE_TOL)
    slots, starts = t["slots"].tolist(), np.concatenate([[0], np.cumsum(lengths)])
    rows = torch.ones(total + pad, dtype=torch.bool, device="cuda")
    for r in (1, 5):
        rows[starts[r]:starts[r + 1]] = False
    for k in ("x", "gate", "input_gate"):
        p[k][~rows] = bad
        p[k][total:] = bad
    for r in (1, 3, 5, 6):
        st[slots[r]] = bad  # not read: without context
    got = ssm.packed_gated_scan_fn(**p, tables=tables, state=st)
    assert torch.equal(got[rows], clean[rows])
    for r in (0, 2, 3, 4, 6):
        assert torch.equal(st[slots[r]], st2[slots[r]])


# ---- graphs at once ----

def test_graphs_replayed_at_once():
    """Two graphs of a training step and two of a packed batch, all in segments with workspaces, on a stream each, again
    and again: every one has its own."""
    lengths, n = [1500, 0, 3500], 5000

    def problem(i):
        if i < 2:
            p = _scan_problem((1, n, 64), torch.bfloat16, seed=70 + i)
            leaves = {k: v.requires_grad_() for k, v in p.items()}
            dout = _rand(_gen(72 + i), 1, n, 64, dtype=torch.bfloat16)

            def train():
                out = ssm.gated_scan_fn(**leaves)
                return [out.detach(), *torch.autograd.grad(out, list(leaves.values()), dout)]
            return train
        p, t, st = _packed_problem(lengths, 64, torch.bfloat16, seed=70 + i, spare=0)
        t["context"] = _i32([0, 0, 0])  # so that a replay does not go on from the one before
        tables = ssm.request_tables(_i32(lengths), n, **t)
        return lambda: [ssm.packed_gated_scan_fn(**p, tables=tables, state=st), st.clone()]

    work = [problem(i) for i in range(4)]
    want = [[v.clone() for v in w()] for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    graphs, held = [], []
    for w, s in zip(work, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            held.append(w())
        graphs.append(graph)
    for _ in range(4):
        for outs in held:
            for v in outs:
                v.zero_()
        torch.cuda.synchronize()
        for _ in range(25):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for outs, wanted in zip(held, want):
            for a, b in zip(outs, wanted):
                assert torch.equal(a, b)


# ---- scales ----

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("group", [None, 32, 64, 128])
@pytest.mark.parametrize("dim", [256, 261, 1024])
@pytest.mark.parametrize("big", [3e38, float("inf"), -float("inf")])
def test_a_group_with_an_infinity_is_nan(dtype, e8m0, group, dim, big):
    """Where the infinity comes of the weight: the row's other groups hold what they held."""
    x = _rand(_gen(80), 3, dim, dtype=dtype).abs() + 2
    w = torch.ones(dim, device="cuda")
    x[:, 40] = 1000.0  # some 10 times the rest's root mean square: 3e38 of it is past fp32
    kind = torch.float8_e8m0fnu if e8m0 else torch.float32
    clean = ssm.rms_norm_quant_fn(x, w, group_size=group, scale_dtype=kind)
    w[40] = big
    q, scale = ssm.rms_norm_quant_fn(x, w, group_size=group, scale_dtype=kind)
    size = group or dim
    bad = slice(40 // size * size, (40 // size + 1) * size)
    assert torch.isnan(q.float()[:, bad]).all() and torch.isnan(scale.float()[:, 40 // size]).all()
    keep, groups = torch.ones(dim, dtype=torch.bool, device="cuda"), torch.ones(scale.shape[1], dtype=torch.bool, device="cuda")
    keep[bad] = False
    groups[40 // size] = False
    assert torch.equal(q.float()[:, keep], clean[0].float()[:, keep])
    assert torch.equal(scale.float()[:, groups], clean[1].float()[:, groups])


@pytest.mark.parametrize("group", [None, 32, 128])
@pytest.mark.parametrize("shape", [(700, 264), (37, 769), (700, 2560)])
def test_fp32_scales_are_rounded_once(group, shape):
    """The largest value over 448 to the nearest fp32, from the values that the norm gives in fp32."""
    p = _norm_problem(shape, torch.float32, "same", seed=81)
    v = ssm.rms_norm_fn(**p)
    _, scale = ssm.rms_norm_quant_fn(**p, group_size=group)
    size = group or shape[1]
    most = torch.stack([part.abs().amax(1) for part in v.split(size, 1)], 1)
    assert torch.equal(scale, (most.double() / 448.0).float())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_row_whose_squares_pass_fp32_is_zeros(dtype):
    """What the header says of it; the rows beside it are as without it."""
    x = _rand(_gen(82), 3, 320, dtype=dtype)
    w = torch.ones(320, device="cuda")
    clean, q0 = ssm.rms_norm_fn(x, w), ssm.rms_norm_quant_fn(x, w, group_size=32)
    x[1, 5] = 2e19  # its square is 4e38
    out, q = ssm.rms_norm_fn(x, w), ssm.rms_norm_quant_fn(x, w, group_size=32)
    for got, want in ((out, clean), (q[0].float(), q0[0].float()), (q[1], q0[1])):
        assert torch.equal(got[::2], want[::2])
    assert not out[1].any() and not q[0].float()[1].any() and (q[1][1] == 2.0**-126).all()


# ---- rows of rank 3 ----

@pytest.mark.parametrize("dtype", TYPES)
def test_norm_of_parts_of_wider_rows_copies_nothing(dtype):
    """Parts of a projection's rows in rank 3, forward and backward: what is allocated is what is returned."""
    b, n, d = 3, 700, 640
    g = _gen(90)
    wide, dwide = _rand(g, b, n, 3 * d, dtype=dtype), _rand(g, b, n, 3 * d, dtype=dtype)
    x, res, _ = wide.split(d, 2)
    dout, dsum, _ = dwide.split(d, 2)
    w = (_rand(g, d, std=0.1) + 1).requires_grad_()
    one, spare = b * n * d * x.element_size(), 2 << 20  # spare: statistics, parts of the weight's gradient

    def peak(call):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        got = call()
        return got, torch.cuda.max_memory_allocated() - before

    with torch.no_grad():
        got, most = peak(lambda: ssm.rms_norm_fn(x, w, residual=res, prenorm=True))
        assert most <= 2 * one + spare
        want = ssm.rms_norm_fn(x.contiguous(), w, residual=res.contiguous(), prenorm=True)
        assert all(torch.equal(a, c) for a, c in zip(got, want))
        q, most = peak(lambda: ssm.rms_norm_quant_fn(x, w, residual=res, prenorm=True, group_size=32))
        assert most <= one + b * n * d * 2 + spare
        want = ssm.rms_norm_quant_fn(x.contiguous(), w, residual=res.contiguous(), prenorm=True, group_size=32)
        assert all(torch.equal(a.float(), c.float()) for a, c in zip(q, want))
    leaves = [x.detach().requires_grad_(), w, res.detach().requires_grad_()]
    outs = ssm.rms_norm_fn(leaves[0], w, residual=leaves[2], prenorm=True)
    spare += 608 * d * 4
    got, most = peak(lambda: torch.autograd.grad(outs, leaves, (dout, dsum)))
    assert most <= one + spare  # one tensor for both inputs
    ds, dw = oracle.rms_norm_bwd(dout, dsum, torch.zeros_like(x), w, outs[1].detach())
    _close(got[0], ds, GTOL[dtype])
    _close(got[1], dw, GTOL[torch.float32])
    _close(got[2], ds, GTOL[dtype])
    # a last stride of another kind is copied
    t = _rand(g, b, d, n, dtype=dtype).transpose(1, 2)
    want, _ = oracle.rms_norm(t, w)
    _close(ssm.rms_norm_fn(t, w), want, TOL[dtype])
