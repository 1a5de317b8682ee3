"""Pins of the layer operators' oracle against something other than itself (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import layer as oracle


def _problem(batch, seqlen, dim, seed, ig=True):
    g = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(g.standard_normal(s))  # noqa: E731
    p = dict(x=t(batch, seqlen, dim), gate=t(batch, seqlen, dim), decay=torch.from_numpy(g.uniform(-4, 1, dim)),
             input_gate=t(batch, seqlen, dim) if ig else None, rate=float(g.uniform(1, 9)), initial_state=t(batch, dim))
    return p, t


def test_scan_against_the_unrolled_sum():
    """h_t = sum_k exp(sum_{j=k+1..t} L_j) sqrt(1 - exp(2 L_k)) i_k x_k + exp(sum_j L_j) h_0, with math.fsum."""
    p, _ = _problem(2, 6, 3, 1)
    out, last = oracle.gated_scan(**p)
    for b in range(2):
        for c in range(3):
            sp = math.log(1 + math.exp(float(p["decay"][c])))
            L = [-p["rate"] * sp / (1 + math.exp(-float(p["gate"][b, t, c]))) for t in range(6)]
            u = [float(p["x"][b, t, c]) / (1 + math.exp(-float(p["input_gate"][b, t, c]))) for t in range(6)]
            for t in range(6):
                h = math.fsum([math.exp(math.fsum(L[k + 1:t + 1])) * math.sqrt(1 - math.exp(2 * L[k])) * u[k] for k in range(t + 1)]
                              + [math.exp(math.fsum(L[:t + 1])) * float(p["initial_state"][b, c])])
                assert abs(out[b, t, c] - h) < 1e-12
            assert last[b, c] == out[b, 5, c]


def test_constant_gates_are_a_geometric_sum():
    n, rate, decay, gate = 20, 3.0, -1.5, 0.7
    ones = torch.ones(1, n, 1, dtype=torch.float64)
    out, _ = oracle.gated_scan(ones * 2, ones * gate, torch.tensor([decay], dtype=torch.float64), None, rate)
    a = math.exp(-rate * math.log1p(math.exp(decay)) / (1 + math.exp(-gate)))
    want = [math.sqrt(1 - a * a) * 2 * (1 - a**(t + 1)) / (1 - a) for t in range(n)]
    np.testing.assert_allclose(out[0, :, 0], want, rtol=1e-12)


def test_unit_variance_is_kept():
    """With inputs of unit variance and an open input gate, sqrt(1 - a^2) keeps the state's variance at 1."""
    g = np.random.default_rng(3)
    x = torch.from_numpy(g.standard_normal((1, 4000, 16)))
    out, _ = oracle.gated_scan(x, torch.zeros_like(x), torch.full((16,), -2.0, dtype=torch.float64), None, 8.0)
    assert abs(out[:, 200:].std() - 1) < 0.05


@pytest.mark.parametrize("ig", [True, False])
def test_gradients_against_differences(ig):
    p, t = _problem(2, 5, 3, 4, ig)
    dout, dlast = t(2, 5, 3), t(2, 3)
    grads = oracle.gated_scan_bwd(dout, dlast, **p)

    def loss(q):
        out, last = oracle.gated_scan(**q)
        return float((out * dout.numpy()).sum() + (last * dlast.numpy()).sum())

    step = 1e-6
    for name, grad in grads.items():
        if grad is None:
            assert name == "input_gate" and not ig
            continue
        for at in np.ndindex(grad.shape):
            q = {k: v.clone() if torch.is_tensor(v) else v for k, v in p.items()}
            q[name][at] += step
            up = loss(q)
            q[name][at] -= 2 * step
            assert abs((up - loss(q)) / (2 * step) - grad[at]) < 1e-7, (name, at)


def test_gradients_where_the_decay_closes():
    """As L goes to 0 the gate's gradient goes to 0, and is 0 where L is."""
    p, t = _problem(1, 4, 2, 5, False)
    p["gate"][0, 2, 0] = -800.0  # sigmoid underflows
    grads = oracle.gated_scan_bwd(t(1, 4, 2), None, **p)
    assert all(np.isfinite(g).all() for g in grads.values() if g is not None)
    assert grads["gate"][0, 2, 0] == 0


def test_packed_is_each_request_by_itself():
    p, t = _problem(1, 9, 3, 6)
    x, gate, ig = (p[k][0] for k in ("x", "gate", "input_gate"))
    state = t(4, 3)
    out, new = oracle.packed_gated_scan(x, gate, p["decay"], [4, 0, 3], ig, p["rate"], state, slots=[2, 1, 3], context=[5, 1, 0])
    a, al = oracle.gated_scan(x[None, :4], gate[None, :4], p["decay"], ig[None, :4], p["rate"], state[None, 2])
    b, bl = oracle.gated_scan(x[None, 4:7], gate[None, 4:7], p["decay"], ig[None, 4:7], p["rate"])
    # (numpy's vector and scalar exponentials may differ in the last bit)
    np.testing.assert_allclose(out, np.concatenate([a[0], b[0], np.zeros((2, 3))]), rtol=1e-13)
    np.testing.assert_allclose(new, np.stack([state[0].numpy(), state[1].numpy(), al[0], bl[0]]), rtol=1e-13)


def test_norm_by_hand():
    out, s = oracle.rms_norm(torch.tensor([[3.0, 4.0]]), torch.tensor([1.0, 2.0]), torch.tensor([[0.0, 0.0]]), eps=0.0)
    rms = math.sqrt(12.5)
    np.testing.assert_allclose(out, [[3 / rms, 8 / rms]], rtol=1e-15)
    np.testing.assert_array_equal(s, [[3, 4]])
    # the sum is rounded to the residual's type
    _, s = oracle.rms_norm(torch.tensor([[1.0]]), torch.ones(1), torch.tensor([[256.0]], dtype=torch.bfloat16))
    assert s[0, 0] == 256


def test_norm_gradients_against_differences():
    g = np.random.default_rng(7)
    t = lambda *s: torch.from_numpy(g.standard_normal(s))  # noqa: E731
    x, w, res, dout, dsum = t(3, 5), t(5), t(3, 5), t(3, 5), t(3, 5)
    ds, dw = oracle.rms_norm_bwd(dout, dsum, x, w, res, 0.1)

    def loss():
        out, s = oracle.rms_norm(x, w, res, 0.1)
        return float((out * dout.numpy()).sum() + (s * dsum.numpy()).sum())

    for tensor, grad in ((x, ds), (res, ds), (w, dw)):
        for at in np.ndindex(grad.shape):
            old = float(tensor[at])
            tensor[at] = old + 1e-6
            up = loss()
            tensor[at] = old - 1e-6
            down = loss()
            tensor[at] = old
            assert abs((up - down) / 2e-6 - grad[at]) < 1e-7


def test_scales_by_hand():
    v = np.array([[448.0, -1.0, 0.0, 0.0, 900.0]])
    np.testing.assert_array_equal(oracle.scales(v, 2, True), [[1.0, 2.0**-126, 4.0]])
    np.testing.assert_array_equal(oracle.scales(v, 0, False), [[900.0 / 448.0]])
