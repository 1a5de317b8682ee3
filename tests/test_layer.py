"""The gated recurrence and the norm on the GPU against the fp64 oracle (oracle/layer.py).

Tolerances are norms of the difference over norms of the result. An output rounded
once to 16 bits is off by at most half a step, finfo(t).eps / 2 relative: 3.9e-3 bf16,
4.9e-4 fp16. Underneath, and for fp32, the recurrence: L is off by up to 2e-6 of itself
(the sigmoid's exponent is rounded at |gate| log2(e), the exponential, reciprocal and
softplus are off by some 3e-7 each), which moves a state by as much as L does, and a and
the state's own rounding by 2^-24 a step, which add up over the 1 / (1 - a) <= 2000
tokens that a state remembers: 2^-24 sqrt(2000) = 3e-6 where they are independent. 2e-5
leaves a factor of about four; gradients are products of two such recurrences: 4e-5.
"""
import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwad

import state_space_model_03_gb300 as ssm
from oracle import layer as oracle

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
STATE_TOL, GRAD_TOL = 2e-5, 4e-5
TOL = {t: torch.finfo(t).eps / 2 + STATE_TOL for t in TYPES}
GTOL = {t: torch.finfo(t).eps / 2 + GRAD_TOL for t in TYPES}


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _close(got, want, tol, what="", slack=0.0):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), what
    norm = np.linalg.norm(want)
    off = np.linalg.norm(got - want)
    assert off <= tol * max(norm, 1e-30) + slack, f"{what}: {off / max(norm, 1e-30):.3e} > {tol:.1e}"


def _decay(g, dim, lo=0.9, hi=0.999, rate=8.0):
    """What the state is multiplied by where the gate is open, drawn from lo to hi."""
    keep = lo + (hi - lo) * torch.rand(dim, generator=g)
    return torch.log(torch.expm1(-torch.log(keep) / rate)).cuda()


def _scan_problem(shape, dtype, ig=True, seed=0, **kw):
    g = _gen(seed)
    p = {k: _rand(g, *shape, dtype=dtype) for k in (("x", "gate", "input_gate") if ig else ("x", "gate"))}
    return p | {"decay": _decay(g, shape[-1], **kw)}


# ---- dense recurrence ----

SHAPES = [
    # one token; one channel; under, at and over a warp's 8 and a tile's 64 tokens; clusters; odd widths
    (1, 1, 1), (2, 1, 64), (1, 7, 3), (3, 8, 66), (2, 63, 130), (1, 64, 128), (1, 65, 32), (2, 127, 200), (1, 128, 33),
    (1, 129, 64), (1, 513, 96), (1, 1500, 10), (2, 1025, 31), (5, 300, 2), (700, 3, 64),
    # enough sequences and channels without clusters; long ones with them, in rows of 16 bytes and not
    (16, 200, 1288), (24, 131, 903), (1, 16384, 24), (3, 9000, 100), (350, 130, 48), (1, 5000, 64), (2, 3333, 40), (1, 2100, 81),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_scan(dtype, shape):
    p = _scan_problem(shape, dtype, ig=sum(shape) % 2 == 0, seed=sum(shape))
    h0 = _rand(_gen(1), shape[0], shape[2]) if shape[1] % 2 else None
    want, wlast = oracle.gated_scan(**p, initial_state=h0)
    out, last = ssm.gated_scan_fn(**p, initial_state=h0, return_last_state=True)
    assert out.dtype == dtype and last.dtype == torch.float32
    _close(out, want, TOL[dtype], "out")
    _close(last, wlast, STATE_TOL, "last")
    assert torch.equal(ssm.gated_scan_fn(**p, initial_state=h0), out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_scan_gradients(dtype, shape):
    p = _scan_problem(shape, dtype, ig=sum(shape) % 2 == 0, seed=1 + sum(shape))
    g = _gen(2)
    h0 = _rand(g, shape[0], shape[2]) if shape[1] % 2 else None
    dout, dlast = _rand(g, *shape, dtype=dtype), _rand(g, shape[0], shape[2])
    leaves = {k: v.clone().requires_grad_() for k, v in (p | ({} if h0 is None else {"initial_state": h0})).items()}
    out, last = ssm.gated_scan_fn(**leaves, return_last_state=True)
    got = dict(zip(leaves, torch.autograd.grad((out, last), list(leaves.values()), (dout, dlast))))
    want = oracle.gated_scan_bwd(dout, dlast, **p, initial_state=h0)
    for k, v in got.items():
        assert v.dtype == leaves[k].dtype
        _close(v, want[k], GTOL[v.dtype], k)


def test_gradients_against_differences():
    """Along a direction, of the fp64 oracle's loss: within what the gradients are off, and 1e-6 of the differences' own."""
    p = _scan_problem((2, 100, 40), torch.float32, seed=3)
    g = _gen(4)
    dout = _rand(g, 2, 100, 40)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    grads = torch.autograd.grad(ssm.gated_scan_fn(**leaves), list(leaves.values()), dout)
    for name, grad in zip(leaves, grads):
        v = torch.randn(grad.shape, generator=g).double()
        loss = []
        for sign in (1, -1):
            q = {k: t.cpu().double() + (sign * 1e-5 * v if k == name else 0) for k, t in p.items()}
            loss.append((oracle.gated_scan(**q)[0] * dout.cpu().double().numpy()).sum())
        slope = float((grad.cpu().double() * v).sum())
        scale = float(grad.double().norm().cpu() * v.norm())
        assert abs((loss[0] - loss[1]) / 2e-5 - slope) <= (GRAD_TOL + 1e-6) * scale, name


@pytest.mark.parametrize("dtype", TYPES)
def test_only_the_wanted_gradients(dtype):
    shape = (2, 150, 24)
    p = _scan_problem(shape, dtype, seed=5)
    dout = _rand(_gen(6), *shape, dtype=dtype)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    want = dict(zip(leaves, torch.autograd.grad(ssm.gated_scan_fn(**leaves), list(leaves.values()), dout)))
    for k in p:
        q = {n: v.clone().requires_grad_() if n == k else v for n, v in p.items()}
        got, = torch.autograd.grad(ssm.gated_scan_fn(**q), [q[k]], dout)
        assert torch.equal(got, want[k]), k
    # the last state alone
    q = {n: v.clone().requires_grad_() for n, v in p.items()}
    _, last = ssm.gated_scan_fn(**q, return_last_state=True)
    dlast = _rand(_gen(7), 2, 24)
    got = torch.autograd.grad(last, list(q.values()), dlast)
    want = oracle.gated_scan_bwd(torch.zeros_like(dout), dlast, **p)
    for k, v in zip(q, got):
        _close(v, want[k], GTOL[v.dtype], k)


@pytest.mark.parametrize("dtype", TYPES)
def test_scan_strides(dtype):
    """Parts of one projection's rows, sequences in the second place, rows at odd places, a last stride of its own."""
    b, n, d = 3, 140, 48
    g = _gen(8)
    decay = _decay(g, d)
    wide = _rand(g, b, n, 3 * d + 1, dtype=dtype)
    second = _rand(g, n, b, 3 * d, dtype=dtype).transpose(0, 1)
    flipped = _rand(g, b, 3 * d, n, dtype=dtype).transpose(1, 2)
    for name, t in (("wide", wide[..., :-1]), ("odd", wide[..., 1:]), ("second", second), ("flipped", flipped)):
        parts = dict(zip(("x", "gate", "input_gate"), t.split(d, 2)))
        want, _ = oracle.gated_scan(**parts, decay=decay)
        _close(ssm.gated_scan_fn(**parts, decay=decay), want, TOL[dtype], name)
        leaves = {k: v.detach().requires_grad_() for k, v in parts.items()}
        dout = _rand(_gen(9), b, d, n, dtype=dtype).transpose(1, 2) if name == "flipped" else _rand(_gen(9), b, n, d, dtype=dtype)
        grads = torch.autograd.grad(ssm.gated_scan_fn(**leaves, decay=decay), list(leaves.values()), dout)
        ref = oracle.gated_scan_bwd(dout, None, **parts, decay=decay)
        for k, v in zip(leaves, grads):
            _close(v, ref[k], GTOL[dtype], f"{name} {k}")
    # one sequence for the whole batch, and a broadcast dout
    x = _rand(g, 1, n, d, dtype=dtype).expand(b, n, d)
    gate = _rand(g, b, n, d, dtype=dtype)
    want, _ = oracle.gated_scan(x, gate, decay)
    _close(ssm.gated_scan_fn(x, gate, decay), want, TOL[dtype])
    leaf = gate.clone().requires_grad_()
    ssm.gated_scan_fn(x, leaf, decay).sum().backward()
    _close(leaf.grad, oracle.gated_scan_bwd(torch.ones_like(gate), None, x, gate, decay)["gate"], GTOL[dtype])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", [(200, 64), (1200, 48)])  # clusters; segments
def test_scan_of_rows_that_share_memory(dtype, n, d):
    """Tokens of one row, windows of one buffer that overlap, a gradient that all tokens share, one tensor as x and gate."""
    b = 2
    g = _gen(11)
    decay = _decay(g, d)
    rest = {k: _rand(g, b, n, d, dtype=dtype) for k in ("gate", "input_gate")}
    buffer = _rand(g, (n + 8) * d + 64, dtype=dtype)
    for name, x in (("one row", buffer[:d].expand(b, n, d)), ("rows", buffer.as_strided((b, n, d), (8 * d, 16, 1))),
                    ("sequences", buffer.as_strided((b, n, d), (8 * d, d, 1))), ("channels", buffer.as_strided((b, n, d), (16, d, 1)))):
        want, _ = oracle.gated_scan(x, decay=decay, **rest)
        _close(ssm.gated_scan_fn(x, decay=decay, **rest), want, TOL[dtype], name)
        gate = rest["gate"].clone().requires_grad_()
        dout = x[:, :1].expand(b, n, d)
        got, = torch.autograd.grad(ssm.gated_scan_fn(x, gate, decay, rest["input_gate"]), [gate], dout)
        _close(got, oracle.gated_scan_bwd(dout, None, x, decay=decay, **rest)["gate"], GTOL[dtype], name)
    x = rest["gate"]
    want, _ = oracle.gated_scan(x, x, decay, x)
    _close(ssm.gated_scan_fn(x, x, decay, x), want, TOL[dtype])


def test_far_offsets():
    """Rows past 2^31 elements, and past 2^31 bytes of a smaller tensor."""
    n, d = 70, 64
    big = torch.empty((1 << 31) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    far = (1 << 31) // n + 64  # the last rows lie past 2^31 elements
    far -= far % 2
    rows = torch.as_strided(big, (1, n, 3 * d), ((n - 1) * far + 3 * d, far, 1))
    rows.copy_(_rand(_gen(10), 1, n, 3 * d, dtype=torch.bfloat16))
    p = dict(zip(("x", "gate", "input_gate"), rows.split(d, 2)), decay=_decay(_gen(11), d))
    want, _ = oracle.gated_scan(**p)
    _close(ssm.gated_scan_fn(**p), want, TOL[torch.bfloat16])
    leaves = {k: v.detach().requires_grad_() for k, v in p.items()}
    dout = _rand(_gen(12), 1, n, d, dtype=torch.bfloat16)
    for (k, ref), v in zip(((k, oracle.gated_scan_bwd(dout, None, **p)[k]) for k in leaves),
                           torch.autograd.grad(ssm.gated_scan_fn(**leaves), list(leaves.values()), dout)):
        _close(v, ref, GTOL[v.dtype], k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rate,lo,hi", [(8.0, -30.0, 20.0), (0.01, -3.0, 3.0), (100.0, -8.0, 8.0)])
def test_decays_and_gates_of_any_size(dtype, rate, lo, hi):
    """From decays that keep everything to ones that keep nothing, gates from shut to open, far beyond where a sigmoid
    rounds to 0 or 1. Elementwise besides: a state is off by TOL of the largest before it in its sequence."""
    g = _gen(13)
    shape = (2, 200, 64)
    p = {"x": _rand(g, *shape, dtype=dtype), "gate": _rand(g, *shape, dtype=dtype, std=30.0), "input_gate": _rand(g, *shape, dtype=dtype, std=30.0),
         "decay": torch.linspace(lo, hi, 64).cuda(), "rate": rate}
    p["gate"][:, ::17] = float("inf")
    p["gate"][:, 5::17] = -float("inf")
    want, wlast = oracle.gated_scan(**p)
    out, last = ssm.gated_scan_fn(**p, return_last_state=True)
    _close(out, want, TOL[dtype])
    _close(last, wlast, STATE_TOL)
    # for gates up to 140 the sigmoid's exponent is rounded to 2^-24 of 200: a factor of 1e-5 in L more
    bound = (TOL[dtype] + 4e-5) * np.maximum.accumulate(np.abs(want), 1) + 1e-7
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()
    dout = _rand(g, *shape, dtype=dtype)
    leaves = {k: v.clone().requires_grad_() if torch.is_tensor(v) else v for k, v in p.items()}
    grads = torch.autograd.grad(ssm.gated_scan_fn(**leaves), [v for v in leaves.values() if torch.is_tensor(v)], dout)
    ref = oracle.gated_scan_bwd(dout, None, **p)
    for k, v in zip((k for k in leaves if k != "rate"), grads):
        assert torch.isfinite(v).all(), k
        if k != "decay":  # its channels differ by many orders of size: below
            _close(v, ref[k], GTOL[dtype] + 4e-5, k)
    off = np.abs(grads[3].double().cpu().numpy() - ref["decay"])
    assert (off <= 1e-3 * np.abs(ref["decay"]).max()).all()


def test_long_memory():
    """65536 tokens of a state that remembers 10^4 of them: errors of a step must not add up."""
    n, d = 65536, 8
    g = _gen(14)
    p = {"x": _rand(g, 1, n, d), "gate": torch.zeros(1, n, d, device="cuda"), "decay": _decay(g, d, 0.9998, 0.9999)}
    want, wlast = oracle.gated_scan(**p)
    out, last = ssm.gated_scan_fn(**p, return_last_state=True)
    _close(out, want, STATE_TOL)
    _close(last, wlast, STATE_TOL)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_sequences_and_channels_do_not_leak(bad):
    p = _scan_problem((3, 200, 70), torch.bfloat16, seed=15)
    clean = ssm.gated_scan_fn(**p)
    q = {k: v.clone() for k, v in p.items()}
    q["x"][1] = bad
    q["x"][0, :, 7] = bad
    q["x"][2, 100:, 9] = bad
    got = ssm.gated_scan_fn(**q)
    same = torch.ones(3, 200, 70, dtype=torch.bool, device="cuda")
    same[1] = same[0, :, 7] = False
    same[2, 100:, 9] = False
    assert torch.equal(got[same], clean[same])
    assert not torch.isfinite(got[~same].float()).any()


def test_in_pieces():
    """A sequence cut in two, the second part from the first one's last state; gradients through the cut."""
    p = _scan_problem((2, 300, 32), torch.float32, seed=16)
    dout = _rand(_gen(17), 2, 300, 32)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    whole = ssm.gated_scan_fn(**leaves)
    want = torch.autograd.grad(whole, list(leaves.values()), dout)
    cut = 101
    part = lambda s: {k: (v if k == "decay" else v[:, s]) for k, v in leaves.items()}  # noqa: E731
    a, state = ssm.gated_scan_fn(**part(slice(0, cut)), return_last_state=True)
    b = ssm.gated_scan_fn(**part(slice(cut, None)), initial_state=state)
    _close(torch.cat([a, b], 1), whole.detach().double().cpu().numpy(), STATE_TOL)
    for k, u, v in zip(leaves, torch.autograd.grad(torch.cat([a, b], 1), list(leaves.values()), dout), want):
        _close(u, v.double().cpu().numpy(), GRAD_TOL, k)


# ---- packed requests ----

RAGGED = [3, 0, 1, 2, 40, 0, 33, 31, 1, 1, 65, 0, 200]


def _packed_problem(lengths, dim, dtype, ig=True, pad=0, seed=0, spare=2):
    n = len(lengths)
    p = _scan_problem((sum(lengths) + pad, dim), dtype, ig, seed)
    rng = np.random.default_rng(seed)
    t = dict(slots=_i32(rng.permutation(n + spare)[:n].tolist()), context=_i32((rng.integers(0, 2, n) * 7).tolist()))
    return p, t, _rand(_gen(seed + 100), n + spare, dim)


def _run_packed(p, t, st, lengths, dtype, block=512):
    want, wst = oracle.packed_gated_scan(**p, lengths=lengths, state=st, **t)
    tables = ssm.request_tables(_i32(lengths), p["x"].shape[0], block=block, **t)
    out = ssm.packed_gated_scan_fn(**p, tables=tables, state=st)
    _close(out, want, TOL[dtype], "out")
    assert not out[sum(lengths):].any()
    _close(st, wst, STATE_TOL, "state")
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,dim,ig,pad", [
    (RAGGED, 96, True, 0), (RAGGED, 33, False, 13), ([1], 1, True, 0), ([0, 0, 5], 64, False, 100), ([1] * 300, 64, True, 0),
    ([700], 130, True, 0), ([64, 128, 64], 64, True, 64), ([8] * 40, 200, False, 1), ([0, 2000, 0, 1], 66, True, 3),
    # segments of many tiles: requests that start in one and end in another, that fill some, that end where one does
    ([5000, 64, 700, 1984, 1, 2047, 3], 40, True, 50), ([1] * 999 + [3000, 1000], 24, False, 0), ([8192, 8192], 33, True, 0),
    (RAGGED * 40, 16, True, 0), ([64] * 100, 96, False, 0),
])
def test_packed(dtype, lengths, dim, ig, pad):
    p, t, st = _packed_problem(lengths, dim, dtype, ig, pad, seed=len(lengths) + dim)
    _run_packed(p, t, st, lengths, dtype)


def test_packed_block_does_not_matter():
    p, t, st = _packed_problem(RAGGED, 64, torch.bfloat16, seed=20)
    outs = []
    for block in (1, 64, 4096):
        s = st.clone()
        outs.append((ssm.packed_gated_scan_fn(**p, tables=ssm.request_tables(_i32(RAGGED), sum(RAGGED), block=block, **t), state=s), s))
    for out, s in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(s, outs[0][1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_packed_neighbours_do_not_leak(dtype, bad):
    """A request of NaN or infinities, padding of them, and such states of other slots leave the others' results alone."""
    lengths = [50, 20, 130, 7]
    p, t, st = _packed_problem(lengths, 70, dtype, pad=30, seed=21, spare=1)
    t["context"] = _i32([3, 0, 0, 4])
    tables = ssm.request_tables(_i32(lengths), 237, **t)
    st2 = st.clone()
    clean = ssm.packed_gated_scan_fn(**p, tables=tables, state=st2)
    slots = t["slots"].tolist()
    for k in ("x", "gate", "input_gate"):
        p[k][50:70] = bad
        p[k][207:] = bad
    st[slots[1]] = st[slots[2]] = bad  # not read: without context
    got = ssm.packed_gated_scan_fn(**p, tables=tables, state=st)
    rows = [i for i in range(237) if not 50 <= i < 70]
    assert torch.equal(got[rows], clean[rows])
    for r in (0, 2, 3):
        assert torch.equal(st[slots[r]], st2[slots[r]])


def test_packed_without_state_or_slot():
    lengths = [140, 33]
    p, _, st = _packed_problem(lengths, 64, torch.float16, seed=22)
    want, _ = oracle.packed_gated_scan(**p, lengths=lengths)
    _close(ssm.packed_gated_scan_fn(**p, tables=ssm.request_tables(_i32(lengths), 173, context=_i32([1, 1]))), want, TOL[torch.float16])
    before = st.clone()
    tables = ssm.request_tables(_i32(lengths), 173, context=_i32([1, 1]), slots=_i32([-1, st.shape[0]]))
    _close(ssm.packed_gated_scan_fn(**p, tables=tables, state=st), want, TOL[torch.float16])
    assert torch.equal(st, before)


def test_lengths_that_do_not_fit():
    """The tables cut them; the rows that are left run as they say."""
    p, _, st = _packed_problem([10], 64, torch.bfloat16, seed=23)
    tables = ssm.request_tables(_i32([4, -3, 9]), 10, slots=_i32([0, 1, 2]))
    want, wst = oracle.packed_gated_scan(**p, lengths=[4, 0, 6], state=st, slots=[0, 1, 2])
    _close(ssm.packed_gated_scan_fn(**p, tables=tables, state=st), want, TOL[torch.bfloat16])
    _close(st, wst, STATE_TOL)


def test_caches_inside_others_and_far_slots():
    """Nothing beside a cache's rows is written; slots past 2^31 elements."""
    lengths, dim = [60, 3], 48
    for far in (False, True):
        p, t, small = _packed_problem(lengths, dim, torch.bfloat16, seed=24, spare=0)
        if far:
            slots = (1 << 31) // 4096 + 9
            big = torch.empty(slots, 4096, device="cuda")
            big[-12:] = 7.0
            st = big[:, 16:16 + dim]
            t["slots"] = _i32([slots - 1, slots - 2])
        else:
            slots = 5
            big = torch.full((slots, 4096), 7.0, device="cuda")
            st = big[:, 16:16 + dim]
            t["slots"] = _i32([4, 1])
        where = t["slots"].tolist()
        for i, s in enumerate(where):
            st[s] = small[i]
        tail = slice(max(0, slots - 12), None)
        rest = big[tail].clone()
        want, wst = oracle.packed_gated_scan(**p, lengths=lengths, state=small, slots=[0, 1], context=t["context"])
        out = ssm.packed_gated_scan_fn(**p, tables=ssm.request_tables(_i32(lengths), 63, **t), state=st)
        _close(out, want, TOL[torch.bfloat16])
        q = {k: (v if k == "decay" else v[:2]) for k, v in p.items()}
        w2, wst2 = oracle.packed_gated_scan(**q, lengths=[1, 1], state=torch.from_numpy(wst), slots=[0, 1], context=[1, 1])
        _close(ssm.gated_state_update(st, slots=t["slots"], **q), w2, TOL[torch.bfloat16])
        for i, s in enumerate(where):
            _close(st[s], wst2[i], STATE_TOL)
            rest[s - (slots if far else 0) + (rest.shape[0] if far else 0), 16:16 + dim] = st[s]
        assert torch.equal(big[tail], rest)
        del big, st


# ---- one token ----

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,dim,ig", [(1, 1, True), (5, 64, False), (3, 33, True), (2, 200, True), (4, 1024, False), (70, 36, True), (513, 8, True)])
def test_step(dtype, n, dim, ig):
    p, t, st = _packed_problem([1] * n, dim, dtype, ig, seed=n + dim)
    want, wst = oracle.packed_gated_scan(**p, lengths=[1] * n, state=st, slots=t["slots"], context=[1] * n)
    out = ssm.gated_state_update(st, slots=t["slots"], **p)
    _close(out, want, TOL[dtype], "out")
    _close(st, wst, STATE_TOL, "state")
    want, wst = oracle.packed_gated_scan(**p, lengths=[1] * n, state=st, context=[1] * n)
    _close(ssm.gated_state_update(st, **p), want, TOL[dtype], "out")
    _close(st, wst, STATE_TOL, "state")


def test_step_skips_rows_without_a_slot():
    p, _, st = _packed_problem([1] * 6, 64, torch.bfloat16, seed=25, spare=0)
    before = st.clone()
    p["x"][1] = float("nan")
    out = ssm.gated_state_update(st, slots=_i32([2, -1, 0, st.shape[0], -7, 5]), **p)
    for k in (1, 3, 4):
        assert not out[k].any() and torch.equal(st[k], before[k])
    assert not torch.equal(st[5], before[5])


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_in_pieces_then_steps_and_dense(dtype):
    """One request in two pieces and then token by token gives what it gives at once, packed or dense."""
    n, cut, steps = 200, 77, 3
    p, _, st = _packed_problem([n], 80, dtype, seed=26, spare=0)
    whole, _ = oracle.packed_gated_scan(**p, lengths=[n])
    _close(ssm.gated_scan_fn(**{k: (v if k == "decay" else v[None]) for k, v in p.items()})[0], whole, TOL[dtype])
    part = lambda a, b: {k: (v if k == "decay" else v[a:b]) for k, v in p.items()}  # noqa: E731
    for a, b, ctx in ((0, cut, 0), (cut, n - steps, cut)):
        tables = ssm.request_tables(_i32([b - a]), b - a, context=_i32([ctx]))
        _close(ssm.packed_gated_scan_fn(**part(a, b), tables=tables, state=st), whole[a:b], TOL[dtype])
    for i in range(n - steps, n):
        _close(ssm.gated_state_update(st, **part(i, i + 1)), whole[i:i + 1], TOL[dtype])


# ---- norm ----

def _norm_problem(shape, dtype, residual, seed=0, wide=False):
    g = _gen(seed)
    kept = {"none": None, "same": dtype, "fp32": torch.float32}[residual]
    return dict(x=_rand(g, *shape, dtype=dtype), weight=_rand(g, shape[-1], std=0.2, dtype=dtype if wide else torch.float32) + 1,
                residual=None if kept is None else _rand(g, *shape, dtype=kept, std=3.0))


# single rows and channels, under and over every way that a row is laid out over threads, odd widths, wide rows
NORM_SHAPES = [(1, 1), (3, 8), (5, 33), (2, 256), (700, 264), (7, 1000), (4, 1024), (3, 1032), (1, 2560), (700, 2560), (2, 3, 640), (3, 769),
               (2, 8200), (2, 8199), (1, 16384), (1, 32768), (2, 32765), (1300, 40)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", ["none", "same", "fp32"])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_norm_and_gradients(dtype, residual, shape):
    p = _norm_problem(shape, dtype, residual, seed=shape[-1], wide=shape[-1] % 16 == 0)
    want, s = oracle.rms_norm(**p)
    out = ssm.rms_norm_fn(**p)
    assert out.dtype == dtype
    _close(out, want, TOL[dtype], "out")
    out2, kept = ssm.rms_norm_fn(**p, prenorm=True)
    assert torch.equal(out2, out)
    if p["residual"] is None:
        assert kept is p["x"]
    else:
        # the sum in fp32 and then in 16 bits may round twice: half a step more of the few that lie half way
        assert kept.dtype == p["residual"].dtype
        _close(kept, s, torch.finfo(kept.dtype).eps / 2)
    g = _gen(31)
    dout = _rand(g, *shape, dtype=dtype)
    dsum = None if p["residual"] is None else _rand(g, *shape, dtype=p["residual"].dtype)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items() if v is not None}
    got = ssm.rms_norm_fn(**leaves, prenorm=dsum is not None)
    grads = dict(zip(leaves, torch.autograd.grad(got, list(leaves.values()), dout if dsum is None else (dout, dsum))))
    # the gradients of the sum as it was kept
    q = p if p["residual"] is None else {"x": torch.zeros_like(p["x"]), "residual": kept, "weight": p["weight"]}
    ds, dw = oracle.rms_norm_bwd(dout, dsum, **q)
    # ds = rstd (w d - n mean(w d n)) is a difference of two terms, each off by some 2^-24 of itself (a product, rstd, the
    # mean's sum and division: below 2^-21 for both). Over few channels they all but cancel (one channel: to eps), so that
    # is no part of the result, but of the terms, whose norms are at most that of rstd w d.
    slack = 2.0**-21 * np.linalg.norm(oracle.f64(dout) * oracle.f64(p["weight"]) / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-5))
    _close(grads["x"], ds, GTOL[dtype], "x", slack)
    if dsum is not None:
        _close(grads["residual"], ds, GTOL[dsum.dtype], "residual", slack)
    _close(grads["weight"], dw, GTOL[p["weight"].dtype], "weight")


def test_norm_gradients_of_parts():
    p = _norm_problem((6, 520), torch.bfloat16, "fp32", seed=32)
    dout, dsum = _rand(_gen(33), 6, 520, dtype=torch.bfloat16), _rand(_gen(34), 6, 520)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    want = dict(zip(leaves, torch.autograd.grad(ssm.rms_norm_fn(**leaves, prenorm=True), list(leaves.values()), (dout, dsum))))
    for k in p:
        q = {n: v.clone().requires_grad_() if n == k else v for n, v in p.items()}
        got, = torch.autograd.grad(ssm.rms_norm_fn(**q, prenorm=True), [q[k]], (dout, dsum))
        assert torch.equal(got, want[k]), k
    # the sum alone, and the output alone
    q = {n: v.clone().requires_grad_() for n, v in p.items()}
    _, s = ssm.rms_norm_fn(**q, prenorm=True)
    got = torch.autograd.grad(s, [q["x"], q["residual"], q["weight"]], dsum, allow_unused=True)
    assert torch.equal(got[1], dsum) and torch.equal(got[0], dsum.to(torch.bfloat16)) and not got[2].any()
    out = ssm.rms_norm_fn(**q)
    got = torch.autograd.grad(out, [q["residual"], q["weight"]], dout)
    ds, dw = oracle.rms_norm_bwd(dout, None, torch.zeros_like(p["x"]), p["weight"], s.detach())
    _close(got[0], ds, GTOL[torch.float32])
    _close(got[1], dw, GTOL[torch.float32])


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_of_broadcast_gradients_and_of_one_tensor_twice(dtype):
    """A gradient that all rows share, one for all of the output, and a tensor that is its own residual."""
    p = _norm_problem((37, 520), dtype, "none", seed=36)
    row = _rand(_gen(37), 520, dtype=dtype)
    for dout in (row.expand(37, 520), row[:1].expand(37, 520)):
        leaves = {k: v.clone().requires_grad_() for k, v in p.items() if v is not None}
        grads = torch.autograd.grad(ssm.rms_norm_fn(**leaves), list(leaves.values()), dout)
        ds, dw = oracle.rms_norm_bwd(dout, None, p["x"], p["weight"])
        _close(grads[0], ds, GTOL[dtype])
        _close(grads[1], dw, GTOL[torch.float32])
    # x + x is exact, and so is the sum of the two gradients, which are the same
    x = p["x"].clone().requires_grad_()
    dout = _rand(_gen(38), 37, 520, dtype=dtype)
    got, = torch.autograd.grad(ssm.rms_norm_fn(x, p["weight"], residual=x), [x], dout)
    ds, _ = oracle.rms_norm_bwd(dout, None, 2 * p["x"].double(), p["weight"])
    _close(got, 2 * ds, GTOL[dtype])


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_strides_and_streams_in_fp32(dtype):
    g = _gen(35)
    wide = _rand(g, 9, 700, dtype=dtype)
    w = _rand(g, 256) + 1
    for x in (wide[:, :256], wide[:, 3:259], wide[::2, 8:264], wide.t()[:256].t(), wide[:3, :256].expand(4, 3, 256), wide[:8, :256].view(2, 4, 256)):
        want, _ = oracle.rms_norm(x, w)
        _close(ssm.rms_norm_fn(x, w), want, TOL[dtype])
    x = wide[:, :256]
    out, s = ssm.rms_norm_fn(x, w, prenorm=True, residual_in_fp32=True)
    assert s.dtype == torch.float32 and torch.equal(s, x.float())
    out, s = ssm.rms_norm_fn(x, w, residual=x, prenorm=True, residual_in_fp32=True)
    assert s.dtype == torch.float32 and torch.equal(s, x.float() * 2)


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_of_rows_that_are_nothing_or_too_much(dtype):
    x = torch.zeros(4, 96, dtype=dtype, device="cuda")
    x[1] = 1e-4
    x[2, 3] = float("inf")
    x[3, 5] = float("nan")
    w = torch.ones(96, device="cuda")
    out = ssm.rms_norm_fn(x, w)
    assert not out[0].any()
    want, _ = oracle.rms_norm(x[1:2], w)
    _close(out[1:2], want, TOL[dtype])
    assert torch.isnan(out[2, 3]) and not out[2, :3].any() and torch.isnan(out[3]).all()
    for group in (None, 32):
        q, scale = ssm.rms_norm_quant_fn(x, w, group_size=group)
        q = q.float()
        assert not q[0].any() and (scale[0] == 2.0**-126).all()
        assert torch.isfinite(q[1]).all()
        bad = slice(None) if group is None else slice(0, 32)
        assert torch.isnan(q[2, bad]).all() and torch.isnan(scale[2, 0])
        assert torch.isnan(q[3]).all() and torch.isnan(scale[3]).all()
        if group:
            assert not q[2, 32:].any()


# ---- norm in 8 bits ----

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", ["none", "same", "fp32"])
@pytest.mark.parametrize("group", [None, 32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1), (3, 32), (5, 33), (700, 264), (7, 1000), (2, 3, 1024), (3, 1032), (2, 2560), (3, 769), (1, 8200), (1, 8199),
                                   (1, 32768)])
@pytest.mark.parametrize("e8m0", [False, True])
def test_quant(dtype, residual, group, shape, e8m0):
    """scale: as fp32 computes it from values that are off by 1e-6; out * scale: within half a step of e4m3 (2^-4 of the
    value, 2^-10 of the scale below its normal numbers) of the norm, whatever the scale."""
    p = _norm_problem(shape, dtype, residual, seed=shape[-1] + 1)
    v, s = oracle.rms_norm(**p)
    more = p["residual"] is not None
    got = ssm.rms_norm_quant_fn(**p, prenorm=more, group_size=group, scale_dtype=torch.float8_e8m0fnu if e8m0 else torch.float32)
    q, scale = got[0], got[1]
    assert q.dtype == torch.float8_e4m3fn and q.shape == shape and scale.shape == shape[:-1] + (-(-shape[-1] // (group or shape[-1])),)
    if more:
        assert got[2].dtype == p["residual"].dtype
        _close(got[2], s, torch.finfo(got[2].dtype).eps / 2)
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


def test_quant_rounds_to_nearest_even_and_holds_its_largest():
    """Values whose quotients are exact: what torch's own conversion gives."""
    x = torch.tensor([[448.0, 17.0, 18.0, 19.0, 21.0, -25.0, 27.0, 0.001953125, 0.0009765625, 0.00146484375, -448.0, 416.0, 432.0, 3.25, -3.75, 5.0] * 2],
                     device="cuda")
    rms = float(x.double().square().mean().sqrt())
    w = torch.full((32,), rms, device="cuda")
    for group in (None, 32):
        q, scale = ssm.rms_norm_quant_fn(x, w, eps=0.0, group_size=group, scale_dtype=torch.float8_e8m0fnu)
        # rms / rms may be off in the last bit: the largest then has the next power of two
        s = float(scale.float()[0, 0])
        assert s in (1.0, 2.0)
        v = ssm.rms_norm_fn(x, w, eps=0.0)
        assert torch.equal(q.float(), (v / s).clamp(-448, 448).to(torch.float8_e4m3fn).float())


# ---- together ----

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_layer_serves_in_pieces(dtype):
    """Norm in 8 bits, a projection, the packed convolution and the recurrence: prompts at once, in pieces, and token by
    token give the same (the same rows go through the same arithmetic but for the recurrence's order of sums)."""
    dim, width, rate = 64, 4, 8.0
    g = _gen(40)
    lengths = [37, 130, 1, 64]
    total = sum(lengths)
    x, res = _rand(g, total, dim, dtype=dtype), _rand(g, total, dim)
    weight, proj = _rand(g, dim, std=0.1) + 1, _rand(g, dim, 3 * dim, std=dim**-0.5)
    conv_w, decay = _rand(g, dim, width, std=0.5), _decay(g, dim)

    def layer(x, res, windows, states, tables=None, slots=None):
        q, scale, s = ssm.rms_norm_quant_fn(x, weight, residual=res, prenorm=True, group_size=32)
        rows = (q.float().view(-1, dim // 32, 32) * scale[..., None]).view(-1, dim)
        u, gate, igate = (rows.double() @ proj.double()).to(dtype).split(dim, 1)
        if tables is not None:
            u = ssm.packed_conv1d_fn(u, conv_w, tables, conv_state=windows, activation="silu")
            return ssm.packed_gated_scan_fn(u, gate, decay, tables, input_gate=igate, rate=rate, state=states), s
        u = ssm.packed_conv1d_update(u, windows, conv_w, slots=slots, activation="silu")
        return ssm.gated_state_update(states, u, gate, decay, input_gate=igate, rate=rate, slots=slots), s

    def caches():
        return torch.zeros(6, dim, width - 1, dtype=dtype, device="cuda"), torch.zeros(6, dim, device="cuda")

    slots = _i32([5, 0, 3, 2])
    starts = np.concatenate([[0], np.cumsum(lengths)])
    windows, states = caches()
    want, _ = layer(x, res, windows, states, ssm.request_tables(_i32(lengths), total, slots=slots))
    kept = states[slots.long()].clone()
    windows, states = caches()
    got = torch.empty_like(want)
    done = [0] * 4
    for take in ([20, 64, 0, 61], [15, 64, 0, 0]):
        rows = np.concatenate([np.arange(starts[r] + done[r], starts[r] + done[r] + n) for r, n in enumerate(take)])
        at = torch.from_numpy(rows).cuda()
        tables = ssm.request_tables(_i32(take), len(rows) + 3, context=_i32(done), slots=slots)
        pad = lambda v: torch.cat([v[at], v.new_full((3, dim), float("nan"))])  # noqa: E731
        out, _ = layer(pad(x), pad(res), windows, states, tables)
        assert not out[len(rows):].any()
        got[at] = out[:len(rows)]
        done = [a + b for a, b in zip(done, take)]
    while any(d < n for d, n in zip(done, lengths)):
        live = [r for r in range(4) if done[r] < lengths[r]]
        at = torch.tensor([starts[r] + done[r] for r in live], device="cuda")
        out, _ = layer(x[at], res[at], windows, states, slots=slots[live])
        got[at] = out
        for r in live:
            done[r] += 1
    # outputs that differ by fp32 rounding may round to neighbours in 16 bits
    _close(got, want.double().cpu().numpy(), 2 * TOL[dtype])
    _close(states[slots.long()], kept.double().cpu().numpy(), 2 * STATE_TOL)


def test_a_layer_trains():
    """Norm, projection and recurrence as one graph against the same in fp64 (fp32 throughout)."""
    b, n, dim = 2, 90, 32
    g = _gen(41)
    t = {"x": _rand(g, b, n, dim), "res": _rand(g, b, n, dim), "weight": _rand(g, dim, std=0.1) + 1,
         "proj": _rand(g, dim, 3 * dim, std=dim**-0.5), "decay": _decay(g, dim)}
    dout = _rand(g, b, n, dim)
    leaves = {k: v.clone().requires_grad_() for k, v in t.items()}
    out, s = ssm.rms_norm_fn(leaves["x"], leaves["weight"], residual=leaves["res"], prenorm=True)
    u, gate, ig = (out.double() @ leaves["proj"].double()).float().split(dim, 2)
    y = ssm.gated_scan_fn(u, gate, leaves["decay"], input_gate=ig)
    got = torch.autograd.grad(y + s, list(leaves.values()), dout)
    ref = {k: v.double().cpu().requires_grad_() for k, v in t.items()}
    rs = ref["x"] + ref["res"]
    ro = rs / torch.sqrt(rs.square().mean(-1, keepdim=True) + 1e-5) * ref["weight"]
    u, gate, ig = (ro @ ref["proj"]).split(dim, 2)
    a = torch.exp(-8.0 * torch.nn.functional.softplus(ref["decay"], threshold=700.0) * torch.sigmoid(gate))
    h, hs = torch.zeros(b, dim, dtype=torch.float64), []
    for k in range(n):
        h = a[:, k] * h + torch.sqrt(1 - a[:, k] ** 2) * torch.sigmoid(ig[:, k]) * u[:, k]
        hs.append(h)
    ry = torch.stack(hs, 1) + rs
    _close(y + s, ry.detach().numpy(), 2 * STATE_TOL)
    for k, v, w in zip(leaves, got, torch.autograd.grad(ry, list(ref.values()), dout.cpu().double())):
        _close(v, w.numpy(), 3 * GRAD_TOL, k)


def test_streams_and_repeats():
    """On a side stream, the same bits in every run, forward and backward."""
    p = _scan_problem((2, 700, 96), torch.bfloat16, seed=42)
    q = _norm_problem((300, 520), torch.bfloat16, "same", seed=43)
    base = None
    for _ in range(3):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
            out = ssm.gated_scan_fn(**leaves)
            norm = {k: v.clone().requires_grad_() for k, v in q.items()}
            n, kept = ssm.rms_norm_fn(**norm, prenorm=True)
            got = [out, n, kept, *torch.autograd.grad(out, list(leaves.values()), torch.ones_like(out)),
                   *torch.autograd.grad((n, kept), list(norm.values()), (torch.ones_like(n), torch.ones_like(kept)))]
        s.synchronize()
        base = base or got
        for a, b in zip(got, base):
            assert torch.equal(a, b)


def test_calls_at_once():
    """Two streams at the same time, each in clusters and in segments with a workspace, forward and backward."""
    problems = [[_scan_problem(shape, torch.bfloat16, seed=60 + i) for shape in ((2, 700, 640), (1, 5000, 64))] for i in range(2)]

    def work(ps):
        got = []
        for p in ps:
            leaves = {k: v.detach().requires_grad_() for k, v in p.items()}
            out = ssm.gated_scan_fn(**leaves)
            got += [out.detach(), *torch.autograd.grad(out, list(leaves.values()), torch.ones_like(out))]
        return got

    want = [work(ps) for ps in problems]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in problems]
    got = []
    for _ in range(20):
        for s, ps in zip(streams, problems):
            with torch.cuda.stream(s):
                got.append(work(ps))
    torch.cuda.synchronize()
    for i, run in enumerate(got):
        for a, b in zip(run, want[i % 2]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("lengths", [[40, 0, 25], [1500, 0, 900]])  # clusters; segments with a workspace
def test_graphs_share_no_workspace(lengths):
    """Two captured graphs, replayed in turn with new inputs: serving, and a training step."""
    n = sum(lengths)
    p, t, st = _packed_problem(lengths, 64, torch.bfloat16, seed=44, spare=0)
    q = _norm_problem((n, 64), torch.bfloat16, "same", seed=45)
    tables = ssm.request_tables(_i32(lengths), n, **t)
    leaves = {k: v[None].clone().requires_grad_() if k != "decay" else v.clone().requires_grad_() for k, v in p.items()}
    norm = {k: v.clone().requires_grad_() for k, v in q.items()}
    dout = torch.ones_like(leaves["x"])

    def serve():
        rows, scale, s = ssm.rms_norm_quant_fn(**q, prenorm=True, group_size=32)
        a = ssm.packed_gated_scan_fn(**p, tables=tables, state=st)
        one = {k: (v if k == "decay" else v[:3]) for k, v in p.items()}
        return rows, scale, s, a, ssm.gated_state_update(st, slots=t["slots"], **one), st

    def train():
        out = ssm.gated_scan_fn(**leaves)
        n = ssm.rms_norm_fn(**norm)
        return [out, n, *torch.autograd.grad(out, list(leaves.values()), dout), *torch.autograd.grad(n, list(norm.values()), torch.ones_like(n))]

    keep = st.clone()
    graphs, held = [], []
    for work in (serve, train):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            work()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(work())
        graphs.append(graph)
    for turn in range(2):
        with torch.no_grad():
            for v in (p["x"], q["x"], leaves["x"], norm["x"]):
                v.copy_(_rand(_gen(50 + turn), *v.shape, dtype=v.dtype))
        st.copy_(keep)
        want = [v.clone().float() for v in serve()] + [v.clone().float() for v in train()]
        st.copy_(keep)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held[0] + tuple(held[1]), want):
            assert torch.equal(a.float(), b)


def test_empty_batches():
    p = _scan_problem((0, 5, 64), torch.bfloat16)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    out, last = ssm.gated_scan_fn(**leaves, return_last_state=True)
    assert out.shape == (0, 5, 64) and last.shape == (0, 64)
    grads = dict(zip(leaves, torch.autograd.grad(out, list(leaves.values()), torch.zeros_like(out))))
    assert not grads["decay"].any() and grads["x"].shape == (0, 5, 64)
    q = {k: v.clone().requires_grad_() for k, v in _norm_problem((0, 64), torch.bfloat16, "fp32").items()}
    out, s = ssm.rms_norm_fn(**q, prenorm=True)
    grads = torch.autograd.grad((out, s), list(q.values()), (out.detach(), s.detach()))
    assert out.shape == (0, 64) and not grads[1].any()
    assert ssm.rms_norm_quant_fn(torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda"))[1].shape == (0, 1)
    st = torch.ones(2, 64, device="cuda")
    x = torch.zeros(0, 64, device="cuda")
    assert ssm.gated_state_update(st, x, x, torch.zeros(64, device="cuda"), slots=_i32([])).shape == (0, 64)
    tables = ssm.request_tables(_i32([0]), 0)
    assert ssm.packed_gated_scan_fn(x, x, torch.zeros(64, device="cuda"), tables, state=st).shape == (0, 64)
    assert (st == 1).all()


def test_caches_count_their_versions():
    p, t, st = _packed_problem([3], 64, torch.float32, seed=46, spare=0)
    tables = ssm.request_tables(_i32([3]), 3, **t)
    for call in (lambda: ssm.packed_gated_scan_fn(**p, tables=tables, state=st),
                 lambda: ssm.gated_state_update(st, **{k: (v if k == "decay" else v[:1]) for k, v in p.items()})):
        before = st._version
        call()
        assert st._version == before + 1


def test_refusals():
    p, t, st = _packed_problem([3], 64, torch.bfloat16, seed=47, spare=0)
    tables = ssm.request_tables(_i32([3]), 3, **t)
    dense = {k: (v if k == "decay" else v[None]) for k, v in p.items()}
    for k in p:
        with pytest.raises(NotImplementedError):
            ssm.packed_gated_scan_fn(**(p | {k: p[k].clone().requires_grad_()}), tables=tables, state=st)
        with pytest.raises(NotImplementedError):
            ssm.gated_state_update(st, **({n: (v if n == "decay" else v[:1]) for n, v in p.items()} | {"decay": p["decay"].clone().requires_grad_()}))
        with torch.no_grad():
            ssm.packed_gated_scan_fn(**(p | {k: p[k].clone().requires_grad_()}), tables=tables, state=st)
    with pytest.raises(ssm_error()):
        ssm.gated_scan_fn(**{k: (v if k == "decay" else v[:, :0]) for k, v in dense.items()})  # no tokens
    for rate in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ssm_error()):
            ssm.gated_scan_fn(**dense, rate=rate)
    with pytest.raises(ValueError, match="another batch"):
        ssm.packed_gated_scan_fn(**{k: (v if k == "decay" else v[:2]) for k, v in p.items()}, tables=tables, state=st)
    with pytest.raises(TypeError, match="initial_state"):
        ssm.gated_scan_fn(**dense, initial_state=torch.zeros(1, 63, device="cuda"))
    with pytest.raises(ssm_error()):
        ssm.gated_state_update(st, **{k: v if k == "decay" else v[:2] for k, v in p.items()})  # two rows, one slot
    w = torch.ones(64, device="cuda")
    with pytest.raises(ssm_error()):
        ssm.rms_norm_fn(p["x"], w, eps=-1.0)
    with pytest.raises(ssm_error()):
        ssm.rms_norm_fn(torch.zeros(1, 32769, device="cuda"), torch.ones(32769, device="cuda"))
    with pytest.raises(NotImplementedError, match="this operator is forward only"):
        ssm.rms_norm_quant_fn(p["x"], w.clone().requires_grad_())
    with pytest.raises(ValueError, match="group_size"):
        ssm.rms_norm_quant_fn(p["x"], w, group_size=16)
    # twice
    leaf = dense["x"].clone().requires_grad_()
    grad, = torch.autograd.grad(ssm.gated_scan_fn(**(dense | {"x": leaf})).float().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        grad.float().sum().backward()
    leaf = p["x"].clone().requires_grad_()
    grad, = torch.autograd.grad(ssm.rms_norm_fn(leaf, w).float().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        grad.float().sum().backward()
    # an input that was changed between the two passes
    leaf, gate = dense["x"].clone().requires_grad_(), dense["gate"].clone()
    out = ssm.gated_scan_fn(leaf, gate, p["decay"])
    gate.zero_()
    with pytest.raises(RuntimeError, match="modified"):
        out.float().sum().backward()
    with fwad.dual_level():
        dual = fwad.make_dual(dense["x"].float(), torch.ones(1, 3, 64, device="cuda"))
        with pytest.raises(NotImplementedError):
            ssm.gated_scan_fn(dual, dense["gate"].float(), p["decay"])
        with pytest.raises(NotImplementedError):
            ssm.rms_norm_fn(dual, w)


def ssm_error():
    from state_space_model_03_gb300 import api
    return api.SSError
