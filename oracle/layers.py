"""fp64 CPU oracle of the layer operators, written from their definitions in numpy.

channel scan     u = a + dt_bias, la = -e^{A_log} softplus(u), alpha = e^{la}, beta = sigmoid(b),
                 h_t = alpha_t h_{t-1} + beta_t x_t, token by token per sequence;
gated ffn        h = act(x w_gate^T) * (x w_up^T);
linear ce        loss_n = log sum_v e^{l_nv} - l_{n, t_n} with l = x w^T.

Each has its gradient written out by the chain rule; the tests hold those to central differences
of the forward functions here. The oracle is test infrastructure and shares no code with the kernels.
"""
from __future__ import annotations

import numpy as np


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy() if hasattr(t, "detach") else np.asarray(t, dtype=np.float64)


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def softplus(x):
    return np.logaddexp(0.0, x)


def spans(B, T, cu, reverse):
    """(batch row, token indices in scan order) of every sequence."""
    if cu is None:
        order = [(b, np.arange(T)) for b in range(B)]
    else:
        cu = [int(c) for c in cu]
        order = [(0, np.arange(cu[i], cu[i + 1])) for i in range(len(cu) - 1)]
    return [(b, idx[::-1] if reverse else idx) for b, idx in order]


def scan(x, a, b, A_log, dt_bias, h0=None, cu=None, reverse=False):
    """(out [B, T, D], hT [S, D])"""
    x, a, b, A_log, dt_bias, h0 = (f64(t) for t in (x, a, b, A_log, dt_bias, h0))
    la = -np.exp(A_log) * softplus(a + dt_bias)
    alpha, beta = np.exp(la), sigmoid(b)
    out = np.zeros_like(x)
    hT = []
    for s, (row, idx) in enumerate(spans(x.shape[0], x.shape[1], cu, reverse)):
        h = np.zeros(x.shape[2]) if h0 is None else h0[s].copy()
        for t in idx:
            h = alpha[row, t] * h + beta[row, t] * x[row, t]
            out[row, t] = h
        hT.append(h)
    return out, np.array(hT).reshape(-1, x.shape[2])


def scan_grads(x, a, b, A_log, dt_bias, dout, h0=None, cu=None, dhT=None, reverse=False):
    """(dx, da, db, dA_log, ddt_bias, dh0) of sum(out * dout) + sum(hT * dhT)"""
    x, a, b, A_log, dt_bias, h0, dout, dhT = (f64(t) for t in (x, a, b, A_log, dt_bias, h0, dout, dhT))
    u = a + dt_bias
    rate = np.exp(A_log)
    la = -rate * softplus(u)
    alpha, beta = np.exp(la), sigmoid(b)
    dx, da, db = (np.zeros_like(x) for _ in range(3))
    dA, ddt = np.zeros_like(A_log), np.zeros_like(A_log)
    dh0 = []
    for s, (row, idx) in enumerate(spans(x.shape[0], x.shape[1], cu, reverse)):
        h = np.zeros(x.shape[2]) if h0 is None else h0[s].copy()
        before = []
        for t in idx:
            before.append(h)
            h = alpha[row, t] * h + beta[row, t] * x[row, t]
        g = np.zeros(x.shape[2]) if dhT is None else dhT[s].copy()
        for k in range(len(idx) - 1, -1, -1):
            t = idx[k]
            g = g + dout[row, t]
            dx[row, t] = beta[row, t] * g
            db[row, t] = beta[row, t] * (1.0 - beta[row, t]) * x[row, t] * g
            dla = alpha[row, t] * before[k] * g
            da[row, t] = -rate * sigmoid(u[row, t]) * dla
            dA += dla * la[row, t]
            ddt += da[row, t]
            g = alpha[row, t] * g
        dh0.append(g)
    return dx, da, db, dA, ddt, np.array(dh0).reshape(-1, x.shape[2])


GELU_C, GELU_A = np.sqrt(2.0 / np.pi), 0.044715


def act_and_slope(v, act):
    if act == "silu":
        s = sigmoid(v)
        return v * s, s + v * s * (1.0 - s)
    th = np.tanh(GELU_C * (v + GELU_A * v ** 3))
    return 0.5 * v * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * v * (1.0 - th ** 2) * GELU_C * (1.0 + 3.0 * GELU_A * v ** 2)


def ffn(x, wg, wu, act="silu"):
    x, wg, wu = f64(x), f64(wg), f64(wu)
    return act_and_slope(x @ wg.T, act)[0] * (x @ wu.T)


def ffn_grads(x, wg, wu, dh, act="silu"):
    """(dx, dw_gate, dw_up) of sum(h * dh)"""
    x, wg, wu, dh = f64(x), f64(wg), f64(wu), f64(dh)
    gate, up = x @ wg.T, x @ wu.T
    val, der = act_and_slope(gate, act)
    dup, dgate = dh * val, dh * up * der
    return dgate @ wg + dup @ wu, dgate.T @ x, dup.T @ x


def ce(x, w, t):
    """(loss [N], lse [N])"""
    l = f64(x) @ f64(w).T
    t = np.asarray(t.cpu() if hasattr(t, "cpu") else t)
    lse = np.logaddexp.reduce(l, axis=1)
    on = (t >= 0) & (t < l.shape[1])
    pick = l[np.arange(len(t)), np.where(on, t, 0)]
    return np.where(on, lse - pick, 0.0), lse


def ce_grads(x, w, t, dloss):
    """(dx, dw) of sum(loss * dloss)"""
    x, w, dloss = f64(x), f64(w), f64(dloss)
    t = np.asarray(t.cpu() if hasattr(t, "cpu") else t)
    l = x @ w.T
    p = np.exp(l - np.logaddexp.reduce(l, axis=1)[:, None])
    on = (t >= 0) & (t < l.shape[1])
    p[np.arange(len(t))[on], t[on]] -= 1.0
    d = np.where(on, dloss, 0.0)[:, None] * p
    return d @ w, d.T @ x
