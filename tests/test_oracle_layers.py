"""Pins of the layer operators' fp64 oracle (oracle/layers.py): closed forms for the forward
functions, central differences for every gradient.

Differences: with step 1e-5 in fp64 the truncation is of order 1e-10 times the third derivative and
the rounding of order 1e-11, so 1e-6 of the largest gradient holds with room."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import layers as L

STEP, TOL = 1e-5, 1e-6


def differences(f, args, k):
    """The gradient of the scalar f(*args) in args[k], element by element."""
    out = np.zeros_like(args[k])
    for i in np.ndindex(*out.shape):
        vals = []
        for d in (STEP, -STEP):
            moved = [None if v is None else np.array(v) for v in args]
            moved[k][i] += d
            vals.append(f(*moved))
        out[i] = (vals[0] - vals[1]) / (2 * STEP)
    return out


def near(x, ref):
    assert np.max(np.abs(x - ref)) <= TOL * max(1.0, np.max(np.abs(ref)))


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 7]])
def test_scan_gradients_are_the_differences(cu, reverse):
    r = np.random.default_rng(1)
    B, T, D = (2, 7, 3) if cu is None else (1, 7, 3)
    S = B if cu is None else len(cu) - 1
    args = [r.standard_normal((B, T, D)) for _ in range(3)] + [r.standard_normal(D) * 0.5, r.standard_normal(D),
                                                              r.standard_normal((S, D))]
    dout, dhT = r.standard_normal((B, T, D)), r.standard_normal((S, D))

    def loss(x, a, b, A, dt, h0):
        o, hT = L.scan(x, a, b, A, dt, h0, cu, reverse)
        return np.sum(o * dout) + np.sum(hT * dhT)

    got = L.scan_grads(*args[:5], dout, args[5], cu, dhT, reverse)
    for k, grad in enumerate(got):
        near(grad, differences(loss, args, k))


def test_scan_closed_forms():
    # constant gates: h_t = beta sum_k alpha^k x_{t-k} + alpha^{t+1} h0
    T, D = 9, 2
    x = np.arange(1.0, T * D + 1).reshape(1, T, D)
    a, b = np.zeros((1, T, D)), np.full((1, T, D), np.log(3.0))
    A, dt, h0 = np.zeros(D), np.zeros(D), np.array([[2.0, -1.0]])
    o, hT = L.scan(x, a, b, A, dt, h0)  # softplus(0) = ln 2: alpha = 1/2, beta = 3/4
    for t in range(T):
        want = 0.5 ** (t + 1) * h0[0] + sum(0.75 * 0.5 ** k * x[0, t - k] for k in range(t + 1))
        assert np.allclose(o[0, t], want, rtol=1e-13)
    assert np.array_equal(hT[0], o[0, -1])
    # a reversed scan is the scan of the reversed sequence; segments are separate scans
    r = np.random.default_rng(2)
    x, a, b = (r.standard_normal((1, 8, D)) for _ in range(3))
    o1, h1 = L.scan(x, a, b, A, dt, None, [0, 5, 8], True)
    for lo, hi, s in ((0, 5, 0), (5, 8, 1)):
        o2, h2 = L.scan(*(t[:, lo:hi][:, ::-1] for t in (x, a, b)), A, dt)
        assert np.array_equal(o1[:, lo:hi][:, ::-1], o2) and np.array_equal(h1[s], h2[0])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn_gradients_are_the_differences(act):
    r = np.random.default_rng(3)
    args = [r.standard_normal((4, 3)), r.standard_normal((5, 3)), r.standard_normal((5, 3))]
    dh = r.standard_normal((4, 5))
    got = L.ffn_grads(*args, dh, act)
    for k, grad in enumerate(got):
        near(grad, differences(lambda *p: np.sum(L.ffn(*p, act) * dh), args, k))


def test_activation_values():
    v = np.array([0.0, 40.0, -40.0, 1.0])
    assert np.allclose(L.act_and_slope(v, "silu")[0], [0.0, 40.0, 0.0, 1.0 / (1.0 + np.exp(-1.0))], atol=1e-12)
    assert np.allclose(L.act_and_slope(v, "gelu_tanh")[0], [0.0, 40.0, 0.0, 0.8411919906082768], atol=1e-12)


def test_ce_gradients_are_the_differences_and_values():
    r = np.random.default_rng(4)
    args = [r.standard_normal((5, 3)), r.standard_normal((6, 3))]
    t = np.array([0, 5, -100, 6, 2])  # two tokens without a loss
    dl = r.standard_normal(5)
    got = L.ce_grads(*args, t, dl)
    for k, grad in enumerate(got):
        near(grad, differences(lambda x, w: np.sum(L.ce(x, w, t)[0] * dl), args, k))
    loss, lse = L.ce(np.zeros((3, 2)), np.ones((8, 2)), np.array([1, 8, -1]))
    assert np.allclose(loss, [np.log(8.0), 0.0, 0.0]) and np.allclose(lse, np.log(8.0))
