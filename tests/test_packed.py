"""Packed requests on the GPU against the fp64 oracle (oracle/packed.py).

Tolerances are norms of the difference over norms of the result, from the
arithmetic: an output rounded once to 16 bits is off by at most half a unit
(2^-9 bf16, 2^-12 fp16), 1/sqrt(3) of that in the mean; the tensor-core scan
rounds two of its operands to the same type, which adds about as much again, so
twice the unit bounds it: 4e-3 and 5e-4. fp32 outputs and states are sums of a
few hundred products in fp32, each with a decay whose exponent (up to some tens)
is rounded to 2^-24: 2e-5 leaves a factor of about ten.
"""
import numpy as np
import pytest
import torch

import state_space_model_03_gb300 as ssm
from oracle import packed as oracle
from state_space_model_03_gb300 import api

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2e-5, torch.float16: 5e-4, torch.bfloat16: 4e-3}
STATE_TOL = 2e-5
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _close(got, want, tol, what=""):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    assert np.isfinite(got).all(), what
    norm = np.linalg.norm(want)
    off = np.linalg.norm(got - want)
    assert off <= tol * max(norm, 1e-30), f"{what}: {off / max(norm, 1e-30):.3e} > {tol:.1e}"


# ---- tables ----

TABLE_CASES = [
    # lengths, tokens, block
    ([5], 5, 4),
    ([0], 3, 7),
    ([1], 1, 1),
    ([3, 0, 0, 9, 1], 13, 4),
    ([3, 0, 0, 9, 1], 21, 4),            # padding at the end
    ([0, 0, 4, 0], 4, 128),
    ([128, 256, 1, 127], 512, 128),      # lengths on the block
    (list(range(600)), 600 * 599 // 2, 33),
    ([2] * 5000, 10001, 1),              # more requests than threads
]


@pytest.mark.parametrize("lengths,tokens,block", TABLE_CASES)
@pytest.mark.parametrize("mode", ["plain", "slots", "free"])
def test_tables(lengths, tokens, block, mode):
    n = len(lengths)
    rng = np.random.default_rng(n + tokens)
    kw = {}
    if mode != "plain":
        slots = rng.permutation(n + 2)[:n]
        if mode == "free":
            slots = np.where(rng.random(n) < 0.5, -1, slots)
            kw["free_slots"] = _i32((n + 2 + rng.permutation(n)).tolist())
        kw |= {"slots": _i32(slots.tolist()), "context": _i32(rng.integers(0, 100, n).tolist())}
    t = ssm.request_tables(_i32(lengths), tokens, block=block, **kw).check()
    want = oracle.request_tables(_i32(lengths), tokens, block=block, **kw)
    for k, v in want.items():
        got = getattr(t, k)
        assert got.dtype == torch.int32
        np.testing.assert_array_equal(got.cpu().numpy(), v, err_msg=k)


@pytest.mark.parametrize("lengths,tokens,free,errors", [
    ([4, 5, 6], 10, 3, 1),
    ([4, -5, 6], 10, 3, 2),
    ([1, 1, 1], 3, 2, 4),
    ([2**31 - 1, 2**31 - 1, 2**31 - 1], 50, 3, 1),   # sums past 32 bits
    ([4, -1, 9], 10, 0, 7),
])
def test_tables_report_what_does_not_fit(lengths, tokens, free, errors):
    kw = {"slots": _i32([-1] * 3), "free_slots": _i32(list(range(10, 10 + free)))}
    t = ssm.request_tables(_i32(lengths), tokens, block=3, **kw)
    want = oracle.request_tables(_i32(lengths), tokens, block=3, **kw)
    assert want["counts"][3] == errors
    for k, v in want.items():
        np.testing.assert_array_equal(getattr(t, k).cpu().numpy(), v, err_msg=k)
    with pytest.raises(ValueError):
        t.check()


# ---- convolution ----

RAGGED = [3, 0, 1, 2, 40, 0, 33, 31, 1, 1, 65]


def _conv_problem(lengths, dim, width, dtype, pad=0, seed=0, strided=False):
    g = _gen(seed)
    n, tokens = len(lengths), sum(lengths) + pad
    x = _rand(g, tokens, dim + (24 if strided else 0), dtype=dtype)
    if strided:
        x = x[:, 8:8 + dim]
    rng = np.random.default_rng(seed)
    return dict(x=x, weight=_rand(g, dim, width, std=0.5), bias=_rand(g, dim, std=0.1),
                conv_state=_rand(g, n + 2, dim, width - 1, dtype=dtype)), \
        dict(slots=_i32(rng.permutation(n + 2)[:n].tolist()), context=_i32((rng.integers(0, 2, n) * 7).tolist()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("dim,strided", [(64, False), (8, False), (31, False), (40, True), (1, False)])
def test_packed_conv(dtype, width, dim, strided):
    p, t = _conv_problem(RAGGED, dim, width, dtype, pad=5, seed=width * 100 + dim, strided=strided)
    want, wst = oracle.packed_conv1d(**p, lengths=_i32(RAGGED), silu_act=True, **t)
    tables = ssm.request_tables(_i32(RAGGED), p["x"].shape[0], block=16, **t)
    st = p.pop("conv_state")
    out = ssm.packed_conv1d_fn(p["x"], p["weight"], tables, bias=p["bias"], conv_state=st, activation="silu")
    _close(out, want, TOL[dtype])
    np.testing.assert_array_equal(st.double().cpu().numpy(), wst)  # windows are copies
    assert not out[sum(RAGGED):].any()


@pytest.mark.parametrize("lengths", [[1], [2, 1], [32, 32], [31, 3, 30], [29, 4, 31], [30, 2, 1, 1, 40], [200]])
def test_packed_conv_at_run_edges(lengths):
    """First tokens near the ends of the threads' runs of 32."""
    p, t = _conv_problem(lengths, 16, 4, torch.float32, seed=sum(lengths))
    t["context"].fill_(3)
    want, wst = oracle.packed_conv1d(**p, lengths=_i32(lengths), **t)
    tables = ssm.request_tables(_i32(lengths), sum(lengths), **t)
    out = ssm.packed_conv1d_fn(p["x"], p["weight"], tables, bias=p["bias"], conv_state=p["conv_state"])
    _close(out, want, TOL[torch.float32])
    np.testing.assert_array_equal(p["conv_state"].double().cpu().numpy(), wst)


def test_packed_conv_without_state_or_slot():
    p, t = _conv_problem([5, 6], 16, 4, torch.float32)
    lengths = _i32([5, 6])
    tables = ssm.request_tables(lengths, 11, context=_i32([4, 4]))
    want, _ = oracle.packed_conv1d(p["x"], p["weight"], lengths)
    _close(ssm.packed_conv1d_fn(p["x"], p["weight"], tables), want, TOL[torch.float32])
    st = p["conv_state"]
    before = st.clone()
    tables = ssm.request_tables(lengths, 11, context=_i32([4, 4]), slots=_i32([-1, st.shape[0]]))  # none, and out of range
    _close(ssm.packed_conv1d_fn(p["x"], p["weight"], tables, conv_state=st), want, TOL[torch.float32])
    assert torch.equal(st, before)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [2, 4])
@pytest.mark.parametrize("n,dim", [(1, 64), (5, 31), (300, 40)])
def test_conv_step(dtype, width, n, dim):
    p, t = _conv_problem([1] * n, dim, width, dtype, seed=n)
    want, wst = oracle.packed_conv1d(**p, lengths=_i32([1] * n), silu_act=True, slots=t["slots"], context=_i32([1] * n))
    out = ssm.packed_conv1d_update(p["x"], p["conv_state"], p["weight"], bias=p["bias"], slots=t["slots"], activation="silu")
    _close(out, want, TOL[dtype])
    np.testing.assert_array_equal(p["conv_state"].double().cpu().numpy(), wst)


# ---- scan ----

def _scan_problem(lengths, heads, groups, headdim, dstate, dtype, z=True, pad=0, seed=0, fused=True, dt32=False, spare=2,
                  A_max=16.0):
    g = _gen(seed)
    n, tokens = len(lengths), sum(lengths) + pad
    hp, gn = heads * headdim, groups * dstate
    if fused:  # x, B and C side by side in one row
        rows = _rand(g, tokens, hp + 2 * gn, dtype=dtype)
        x, B, C = rows[:, :hp], rows[:, hp:hp + gn], rows[:, hp + gn:]
    else:
        x, B, C = (_rand(g, tokens, k, dtype=dtype) for k in (hp, gn, gn))
    first = 0.001 + 0.099 * torch.rand(heads, generator=g)
    p = dict(x=x.view(tokens, heads, headdim), dt=_rand(g, tokens, heads, dtype=torch.float32 if dt32 else dtype),
             A=-(1 + (A_max - 1) * torch.rand(heads, generator=g)).cuda(), B=B.view(tokens, groups, dstate),
             C=C.view(tokens, groups, dstate), D=1 + _rand(g, heads, std=0.1),
             z=_rand(g, tokens, heads, headdim, dtype=dtype) if z else None,
             dt_bias=torch.log(torch.expm1(first)).cuda(), dt_softplus=True)
    rng = np.random.default_rng(seed)
    t = dict(slots=_i32(rng.permutation(n + spare)[:n].tolist()), context=_i32((rng.integers(0, 2, n) * 7).tolist()))
    return p, t, _rand(g, n + spare, heads, headdim, dstate, std=0.5)


def _run_scan(p, t, state, lengths, block):
    want, wst = oracle.head_scan(**p, lengths=_i32(lengths), state=state, **t)
    tables = ssm.request_tables(_i32(lengths), p["x"].shape[0], block=block, **t)
    out = ssm.head_scan_fn(**p, tables=tables, state=state)
    torch.cuda.synchronize()
    assert api.device_error() == 0
    _close(out, want, TOL[p["x"].dtype], "out")
    _close(state, wst, STATE_TOL, "state")
    assert not out[sum(lengths):].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,groups,headdim,dstate", [
    (2, 1, 64, 128), (4, 2, 64, 64), (3, 1, 64, 128), (6, 2, 64, 16), (2, 2, 128, 128), (1, 1, 128, 64), (3, 3, 64, 40),
    (2, 1, 40, 72), (2, 1, 80, 96), (2, 1, 17, 33), (1, 1, 200, 24), (2, 1, 33, 256), (1, 1, 1, 1),
])
def test_scan_shapes(dtype, heads, groups, headdim, dstate):
    lengths = [70, 0, 1, 129, 128, 17]
    p, t, st = _scan_problem(lengths, heads, groups, headdim, dstate, dtype, z=heads != 2, pad=3, seed=headdim + dstate)
    _run_scan(p, t, st, lengths, 4096)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [1, 50, 128, 200, 256])
@pytest.mark.parametrize("headdim,dstate", [(64, 128), (128, 64), (24, 20)])
def test_scan_blocks(dtype, block, headdim, dstate):
    """Requests of several blocks: summaries, their folding, and the start state of a request that goes on."""
    lengths = [1, 300, 0, 51, 128, 257, 20] if block > 1 else [1, 4, 0, 2]
    p, t, st = _scan_problem(lengths, 3, 1, headdim, dstate, dtype, z=False, seed=block)
    t["context"].fill_(1)
    _run_scan(p, t, st, lengths, block)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 385, 640, 1500])
def test_scan_lengths(dtype, n):
    p, t, st = _scan_problem([n], 2, 1, 64, 128, dtype, seed=n)
    _run_scan(p, t, st, [n], 1 << 15)


@pytest.mark.parametrize("dtype", TYPES)
def test_scan_options(dtype):
    lengths = [130, 5]
    p, t, st = _scan_problem(lengths, 2, 1, 64, 64, dtype, z=False, fused=False, dt32=True, seed=3)
    p |= {"D": None, "dt_bias": None}
    p["dt"] = p["dt"].abs() * 0.05
    p["dt_softplus"] = False
    _run_scan(p, t, st, lengths, 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [1e-4, 30.0])
def test_scan_step_sizes(dtype, scale):
    """Steps so small that the state keeps everything, and so large that it keeps one token."""
    lengths = [300]
    p, t, st = _scan_problem(lengths, 2, 1, 64, 128, dtype, z=False, dt32=True, seed=4)
    p |= {"dt_bias": None, "dt_softplus": False}
    p["dt"] = p["dt"].abs() * scale
    t["context"].fill_(1)
    _run_scan(p, t, st, lengths, 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("block", [256, 4096])
@pytest.mark.parametrize("large_first", [True, False])
def test_scan_steps_of_different_size(dtype, block, large_first):
    """Tokens whose steps are next to nothing after ordinary ones, and before: no term overflows or is lost."""
    lengths = [700]
    p, t, st = _scan_problem(lengths, 2, 1, 64, 64, dtype, z=False, dt32=True, seed=11)
    p |= {"dt_bias": None, "dt_softplus": False}
    p["dt"] = p["dt"].abs() * 0.02
    part = slice(200, 700) if large_first else slice(0, 500)
    p["dt"][part] *= 1e-8
    p["x"][100] *= 100
    t["context"].fill_(1)
    _run_scan(p, t, st, lengths, block)


def test_steps_and_prompts_in_a_cuda_graph():
    lengths = [130, 7]
    p, t, st = _scan_problem(lengths, 2, 1, 64, 64, torch.bfloat16, seed=12)
    c, _ = _conv_problem(lengths, 40, 4, torch.bfloat16, seed=12)
    length = _i32(lengths)

    def work():
        tables = ssm.request_tables(length, 137, block=64, **t)
        a = ssm.packed_conv1d_fn(c["x"], c["weight"], tables, bias=c["bias"], conv_state=c["conv_state"])
        b = ssm.head_scan_fn(**p, tables=tables, state=st)
        q = {k: (v[:2] if k in ("x", "dt", "B", "C", "z") else v) for k, v in p.items()}
        d = ssm.head_state_update(st, slots=t["slots"], **q)
        e = ssm.packed_conv1d_update(c["x"][:2], c["conv_state"], c["weight"], slots=t["slots"])
        return a, b, d, e, st, c["conv_state"]

    keep = st.clone(), c["conv_state"].clone()

    def reset():
        st.copy_(keep[0])
        c["conv_state"].copy_(keep[1])

    want = [v.clone() for v in work()]
    reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
def test_caches_and_operands_of_other_strides(dtype):
    """Slots inside a larger cache, dt of another order, operands without unit stride (copied)."""
    lengths = [60, 150, 3]
    p, t, _ = _scan_problem(lengths, 2, 1, 64, 32, dtype, seed=13)
    big = _rand(_gen(14), 7, 5, 64, 32, std=0.5)
    st, rest = big[1:6, 2:4], big.clone()
    p["dt"] = p["dt"].t().contiguous().t()
    p["B"] = p["B"].transpose(1, 2).contiguous().transpose(1, 2)
    p["z"] = p["z"].flip(2).contiguous().flip(2)
    _run_scan(p, t, st, lengths, 64)
    rest[1:6, 2:4] = st
    assert torch.equal(big, rest)  # nothing outside the view
    q = {k: (v[:3] if k in ("x", "dt", "B", "C", "z") else v) for k, v in p.items()}
    want, wst = oracle.head_scan(**q, lengths=_i32([1] * 3), state=st, slots=t["slots"], context=_i32([1] * 3))
    _close(ssm.head_state_update(st, slots=t["slots"], **q), want, TOL[dtype])
    _close(st, wst, STATE_TOL)
    rest[1:6, 2:4] = st
    assert torch.equal(big, rest)
    c, ct = _conv_problem(lengths, 24, 4, dtype, seed=15)
    wide = _rand(_gen(16), 5, 40, 3, dtype=dtype)
    c["conv_state"] = wide[:, 8:32]
    rest = wide.clone()
    want, wst = oracle.packed_conv1d(**c, lengths=_i32(lengths), **ct)
    out = ssm.packed_conv1d_fn(c["x"], c["weight"], ssm.request_tables(_i32(lengths), 213, **ct), bias=c["bias"],
                               conv_state=c["conv_state"])
    _close(out, want, TOL[dtype])
    rest[:, 8:32] = torch.from_numpy(wst).to(dtype).cuda()
    assert torch.equal(wide, rest)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_neighbours_do_not_leak(dtype, bad):
    """A request of NaN or infinities, and padding of them, leaves the other requests' results alone."""
    lengths = [50, 20, 130, 7]
    p, t, st = _scan_problem(lengths, 2, 1, 64, 64, dtype, z=False, pad=30, seed=5, spare=0)
    tables = ssm.request_tables(_i32(lengths), p["x"].shape[0], block=64, **t)
    st2 = st.clone()
    clean = ssm.head_scan_fn(**p, tables=tables, state=st2)
    for k in ("x", "dt", "B", "C"):
        p[k][50:70] = bad
        p[k][207:] = bad
    got = ssm.head_scan_fn(**p, tables=tables, state=st)
    rows = [i for i in range(237) if not 50 <= i < 70]
    assert torch.equal(got[rows], clean[rows])
    slots = t["slots"].tolist()
    for r in (0, 2, 3):
        assert torch.equal(st[slots[r]], st2[slots[r]])


@pytest.mark.parametrize("dtype", TYPES)
def test_scan_without_state_or_slot(dtype):
    lengths = [140, 33]
    p, t, st = _scan_problem(lengths, 2, 1, 64, 64, dtype, seed=6)
    want, _ = oracle.head_scan(**p, lengths=_i32(lengths))
    tables = ssm.request_tables(_i32(lengths), 173, block=64, context=_i32([1, 1]))
    _close(ssm.head_scan_fn(**p, tables=tables), want, TOL[dtype])
    before = st.clone()
    tables = ssm.request_tables(_i32(lengths), 173, block=64, context=_i32([1, 1]), slots=_i32([-1, st.shape[0]]))
    _close(ssm.head_scan_fn(**p, tables=tables, state=st), want, TOL[dtype])
    assert torch.equal(st, before)


def test_scan_large_offsets():
    """A cache whose last slots lie past 2^31 elements."""
    heads, headdim, dstate = 8, 64, 128
    slots = (1 << 31) // (heads * headdim * dstate) + 3
    st = torch.zeros(slots, heads, headdim, dstate, device="cuda")
    lengths = [9, 4]
    p, t, small = _scan_problem(lengths, heads, 1, headdim, dstate, torch.bfloat16, seed=7)
    where = [slots - 1, slots - 2]
    for i, s in enumerate(where):
        st[s] = small[i]
    ctx = _i32([1, 1])
    want, wst = oracle.head_scan(**p, lengths=_i32(lengths), state=small, slots=_i32([0, 1]), context=ctx)
    tables = ssm.request_tables(_i32(lengths), 13, slots=_i32(where), context=ctx)
    _close(ssm.head_scan_fn(**p, tables=tables, state=st), want, TOL[torch.bfloat16])
    for i, s in enumerate(where):
        _close(st[s], wst[i], STATE_TOL)
    q = {k: (v[:2] if k in ("x", "dt", "B", "C", "z") else v) for k, v in p.items()}
    w2, wst2 = oracle.head_scan(**q, lengths=_i32([1, 1]), state=torch.from_numpy(wst), slots=_i32([0, 1]), context=ctx)
    _close(ssm.head_state_update(st, slots=_i32(where), **q), w2, TOL[torch.bfloat16])
    for i, s in enumerate(where):
        _close(st[s], wst2[i], STATE_TOL)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,heads,groups,headdim,dstate", [
    (1, 2, 1, 64, 128), (5, 3, 3, 64, 64), (3, 2, 1, 17, 33), (2, 1, 1, 200, 256), (4, 2, 1, 8, 5), (2, 2, 2, 128, 16), (1, 1, 1, 1, 1),
    (70, 4, 2, 64, 24),
])
def test_scan_step(dtype, n, heads, groups, headdim, dstate):
    p, t, st = _scan_problem([1] * n, heads, groups, headdim, dstate, dtype, z=n != 5, seed=n + headdim)
    want, wst = oracle.head_scan(**p, lengths=_i32([1] * n), state=st, slots=t["slots"], context=_i32([1] * n))
    out = ssm.head_state_update(st, slots=t["slots"], **p)
    _close(out, want, TOL[dtype], "out")
    _close(st, wst, STATE_TOL, "state")


def test_steps_skip_rows_without_a_slot():
    p, t, st = _scan_problem([1] * 4, 2, 1, 64, 64, torch.bfloat16, seed=8)
    slots = _i32([2, -1, 0, st.shape[0]])
    before = st.clone()
    out = ssm.head_state_update(st, slots=slots, **p)
    assert not out[1].any() and not out[3].any()
    for k in (1, 3, 4, 5):
        assert torch.equal(st[k], before[k])
    c, _ = _conv_problem([1] * 4, 32, 4, torch.bfloat16)
    cs = c["conv_state"]
    before = cs.clone()
    out = ssm.packed_conv1d_update(c["x"], cs, c["weight"], slots=slots)
    assert not out[1].any() and not out[3].any()
    for k in (1, 3, 4, 5):
        assert torch.equal(cs[k], before[k])


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_in_pieces_then_steps(dtype):
    """One request in two pieces and then token by token gives what it gives at once."""
    n, cut, steps = 200, 77, 3
    p, _, st = _scan_problem([n], 2, 1, 64, 128, dtype, z=False, seed=9, spare=0)
    whole, wst = oracle.head_scan(**p, lengths=_i32([n]))[0], None
    for a, b, ctx in ((0, cut, 0), (cut, n - steps, cut)):
        q = {k: (v[a:b] if k in ("x", "dt", "B", "C") else v) for k, v in p.items()}
        tables = ssm.request_tables(_i32([b - a]), b - a, context=_i32([ctx]))
        _close(ssm.head_scan_fn(**q, tables=tables, state=st), whole[a:b], TOL[dtype])
    for i in range(n - steps, n):
        q = {k: (v[i:i + 1] if k in ("x", "dt", "B", "C") else v) for k, v in p.items()}
        _close(ssm.head_state_update(st, **q), whole[i:i + 1], TOL[dtype])


def test_runs_are_repeatable_and_on_the_current_stream():
    lengths = [200, 31]
    p, t, st = _scan_problem(lengths, 4, 1, 64, 128, torch.bfloat16, seed=10)
    base = None
    for _ in range(3):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            st2 = st.clone()
            tables = ssm.request_tables(_i32(lengths), 231, block=128, **t)
            out = ssm.head_scan_fn(**p, tables=tables, state=st2)
        s.synchronize()
        if base is None:
            base = (out, st2)
        assert torch.equal(out, base[0]) and torch.equal(st2, base[1])


def test_nothing_is_done_for_no_tokens():
    p, t, st = _scan_problem([4], 2, 1, 64, 64, torch.bfloat16)
    before = st.clone()
    tables = ssm.request_tables(_i32([0]), 0)
    q = {k: (v[:0] if k in ("x", "dt", "B", "C", "z") else v) for k, v in p.items()}
    assert ssm.head_scan_fn(**q, tables=tables, state=st).shape == (0, 2, 64)
    assert torch.equal(st, before)
    assert tables.counts.tolist() == [0, 0, 0, 0]


def test_example_serves_in_pieces():
    import examples.packed_serving as example
    # convolution, scan and projections each round to bf16 (2^-9) on either side, in other places
    assert example.main() < 2e-2


# ---- refusals ----

def _step_args(n=2):
    p, t, st = _scan_problem([1] * n, 2, 1, 64, 64, torch.bfloat16)
    return p, t, st


@pytest.mark.parametrize("change,error", [
    (dict(dt=lambda p: p["dt"].to(torch.float16)), TypeError),
    (dict(B=lambda p: p["B"].float()), TypeError),
    (dict(C=lambda p: p["C"][:, :, :8]), TypeError),
    (dict(z=lambda p: p["z"][:1]), TypeError),
    (dict(A=lambda p: p["A"].double()), TypeError),
    (dict(D=lambda p: p["D"][:1]), TypeError),
    (dict(x=lambda p: p["x"].clone().requires_grad_()), NotImplementedError),
    (dict(x=lambda p: p["x"].cpu()), RuntimeError),
    (dict(A=lambda p: p["A"].cpu()), ValueError),
])
def test_scan_refuses(change, error):
    p, t, st = _step_args()
    q = p | {k: f(p) for k, f in change.items()}
    with pytest.raises(error):
        ssm.head_state_update(st, **q)
    tables = ssm.request_tables(_i32([2]), 2)
    with pytest.raises(error):
        ssm.head_scan_fn(**q, tables=tables)


def test_operators_refuse_what_does_not_belong_together():
    p, t, st = _step_args(3)
    tables = ssm.request_tables(_i32([2]), 2)
    with pytest.raises(ValueError):
        ssm.head_scan_fn(**p, tables=tables)           # tables of another batch
    with pytest.raises(ValueError):
        ssm.head_state_update(st.transpose(2, 3).contiguous().transpose(2, 3), **p)
    with pytest.raises(TypeError):
        ssm.head_state_update(st.bfloat16(), **p)
    with pytest.raises(TypeError):
        ssm.head_state_update(st, slots=_i32([0, 1]), **p)
    with pytest.raises(api.SSError) as e:
        ssm.head_state_update(st[:2], **p)             # three rows, two slots, no map
    assert e.value.status == 2
    with pytest.raises(api.SSError) as e:              # 257 states
        q, _, st2 = _scan_problem([1], 1, 1, 8, 257, torch.float32)
        ssm.head_state_update(st2, **q)
    assert e.value.status == 7
    c, ct = _conv_problem([3], 16, 4, torch.float32)
    with pytest.raises(NotImplementedError):
        ssm.packed_conv1d_update(c["x"], c["conv_state"], c["weight"], activation="gelu")
    with pytest.raises(TypeError):
        ssm.packed_conv1d_update(c["x"], c["conv_state"][:, :, :2], c["weight"])
    with pytest.raises(api.SSError) as e:
        ssm.packed_conv1d_update(c["x"], torch.zeros(3, 16, 4, device="cuda"), torch.zeros(16, 5, device="cuda"))
    assert e.value.status == 7
    with pytest.raises(ValueError):
        ssm.request_tables(_i32([1]), 1, free_slots=_i32([0]))
    with pytest.raises(TypeError):
        ssm.request_tables(torch.ones(2, device="cuda"), 2)
    with pytest.raises(ValueError):
        ssm.request_tables(_i32([1]), 1, block=0)
    with pytest.raises(RuntimeError):
        ssm.request_tables(torch.ones(2, dtype=torch.int32), 2)
