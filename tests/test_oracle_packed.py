"""Pins of the packed operators' oracle against something other than itself (CPU)."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import packed


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _problem(lengths, heads, groups, headdim, dstate, seed):
    g = np.random.default_rng(seed)
    n = sum(lengths)
    t = lambda *s: torch.from_numpy(g.standard_normal(s))  # noqa: E731
    return dict(x=t(n, heads, headdim), dt=t(n, heads), A=-torch.from_numpy(g.uniform(0.2, 2, heads)), B=t(n, groups, dstate),
                C=t(n, groups, dstate), D=t(heads), z=t(n, heads, headdim), dt_bias=t(heads), dt_softplus=True), g


def test_scan_against_the_unrolled_sum():
    """S_t = sum_k exp(A sum_{j=k+1..t} dt_j) dt_k x_k B_k^T + exp(A sum_j dt_j) S_0, with math.fsum."""
    lengths, heads, groups, p_, n_ = [4, 0, 3], 2, 1, 2, 3
    p, g = _problem(lengths, heads, groups, p_, n_, 1)
    state = torch.from_numpy(g.standard_normal((4, heads, p_, n_)))
    slots, ctx = _i32([2, 0, 3]), _i32([5, 1, 0])
    out, st = packed.head_scan(**p, lengths=_i32(lengths), state=state, slots=slots, context=ctx)
    first = 0
    for r, length in enumerate(lengths):
        for h in range(heads):
            dt = [math.log(1 + math.exp(float(p["dt"][first + i, h] + p["dt_bias"][h]))) for i in range(length)]
            for a in range(p_):
                for t in range(length):
                    y = []
                    for n in range(n_):
                        terms = [math.exp(float(p["A"][h]) * math.fsum(dt[k + 1:t + 1])) * dt[k] * float(p["x"][first + k, h, a])
                                 * float(p["B"][first + k, 0, n]) for k in range(t + 1)]
                        if int(ctx[r]) > 0:
                            terms.append(math.exp(float(p["A"][h]) * math.fsum(dt[:t + 1])) * float(state[int(slots[r]), h, a, n]))
                        y.append(float(p["C"][first + t, 0, n]) * math.fsum(terms))
                        if t == length - 1:
                            assert abs(st[int(slots[r]), h, a, n] - math.fsum(terms)) < 1e-12
                    z = float(p["z"][first + t, h, a])
                    want = (math.fsum(y) + float(p["D"][h] * p["x"][first + t, h, a])) * z / (1 + math.exp(-z))
                    assert abs(out[first + t, h, a] - want) < 1e-12
        first += length
    for s in (0, 1):  # the empty request's slot, and nobody's
        np.testing.assert_array_equal(st[s], state[s].numpy())


def test_scan_against_the_per_channel_oracle():
    """A decay per head is the per-channel scan with the head's A for all its channels and states."""
    n, heads, groups, p_, n_ = 23, 4, 2, 3, 5
    p, _ = _problem([n], heads, groups, p_, n_, 2)
    p = {k: (v.float() if torch.is_tensor(v) else v) for k, v in p.items()}
    out, _ = packed.head_scan(**p, lengths=_i32([n]))
    rep = lambda v: v.repeat_interleave(p_, -1)  # noqa: E731
    chan = lambda v: v.reshape(n, -1).t().unsqueeze(0).contiguous()  # noqa: E731
    ref = oracle.selective_scan_ref(chan(p["x"]), chan(rep(p["dt"])), rep(p["A"])[:, None].expand(-1, n_).contiguous(),
                                    p["B"].permute(1, 2, 0).unsqueeze(0).contiguous(), p["C"].permute(1, 2, 0).unsqueeze(0).contiguous(),
                                    D=rep(p["D"]), z=chan(p["z"]), delta_bias=rep(p["dt_bias"]), delta_softplus=True)
    np.testing.assert_allclose(out.reshape(n, -1).T[None], np.asarray(ref), rtol=0, atol=1e-12)


@pytest.mark.parametrize("cuts", [[7], [3, 4], [1, 1, 5], [0, 7, 0]])
def test_pieces_compose(cuts):
    p, g = _problem([7], 2, 1, 3, 4, 3)
    whole, wst = packed.head_scan(**p, lengths=_i32([7]), state=torch.zeros(1, 2, 3, 4))
    w, b = torch.from_numpy(g.standard_normal((6, 4))), torch.from_numpy(g.standard_normal(6))
    x = p["x"].reshape(7, 6)
    conv, cst = packed.packed_conv1d(x, w, _i32([7]), b, torch.zeros(1, 6, 3), silu_act=True)
    st, cs, at = torch.zeros(1, 2, 3, 4), torch.zeros(1, 6, 3), 0
    for n in cuts:
        q = {k: (v[at:at + n] if k in ("x", "dt", "B", "C", "z") else v) for k, v in p.items()}
        out, new = packed.head_scan(**q, lengths=_i32([n]), state=st, context=_i32([at]))
        np.testing.assert_allclose(out, whole[at:at + n], atol=1e-12)
        c, newc = packed.packed_conv1d(x[at:at + n], w, _i32([n]), b, cs, context=_i32([at]), silu_act=True)
        np.testing.assert_allclose(c, conv[at:at + n], atol=1e-12)
        st, cs, at = torch.from_numpy(new), torch.from_numpy(newc), at + n
    np.testing.assert_allclose(st.numpy(), wst, atol=1e-12)
    np.testing.assert_allclose(cs.numpy(), cst, atol=0)


def test_conv_against_numpy():
    g = np.random.default_rng(4)
    lengths, dim = [9, 1, 2, 0, 5], 3
    x, w = torch.from_numpy(g.standard_normal((17, dim))), torch.from_numpy(g.standard_normal((dim, 4)))
    out, _ = packed.packed_conv1d(x, w, _i32(lengths))
    at = 0
    for n in lengths:
        for c in range(dim):
            if n:
                np.testing.assert_allclose(out[at:at + n, c], np.convolve(x[at:at + n, c].numpy(), w[c].numpy()[::-1])[:n], atol=1e-12)
        at += n


def test_tables_by_hand():
    t = packed.request_tables(_i32([3, 0, 5]), 10, context=_i32([7, 0, 0]), slots=_i32([4, -1, -1]), free_slots=_i32([9, 8]), block=2)
    assert t["offsets"].tolist() == [0, 3, 3, 8]
    assert t["token_request"].tolist() == [0, 0, 0, 2, 2, 2, 2, 2, -1, -1]
    assert t["token_position"].tolist() == [7, 8, 9, 0, 1, 2, 3, 4, 0, 0]
    assert t["blocks"].tolist() == [[0, 0, 2, 0], [0, 2, 1, 1], [2, 3, 2, 0], [2, 5, 2, 1], [2, 7, 1, 2]] + [[-1, 0, 0, 0]] * 3
    assert t["slots"].tolist() == [4, 9, 8]
    assert t["carried"].tolist() == [0, 2, 3, -1, -1]
    assert t["counts"].tolist() == [8, 5, 2, 0]
