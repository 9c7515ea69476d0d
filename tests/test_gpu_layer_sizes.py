"""The layer operators at sizes whose launches hold 2^32 threads and more, each against its formula in 64 bits
on the GPU, at the places on both sides of the limit and at the end. Tolerances as in the operators' own tests."""
from __future__ import annotations

import pytest
import torch

from tests._layers import BF16, U16, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    yield binding
    torch.cuda.empty_cache()


def near(x, ref, tol, what):
    x, ref = x.double(), ref.double()
    e = ((x - ref).norm() / ref.norm()).item()
    assert e <= tol, "%s: relative error %.3e > %.1e" % (what, e, tol)


def gates(a, b, A_log, dt_bias):
    la = -A_log.double().exp() * torch.nn.functional.softplus(a.double() + dt_bias.double(), threshold=200.0)
    return la, la.exp(), torch.sigmoid(b.double())


def test_many_sequences(gdr):
    """65,541 sequences of one token and 4096 channels: 2^23 + 640 workgroups of 512 threads."""
    N, D = 65541, 4096
    say("channel scan N %d T 1 D %d" % (N, D))
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.empty(s, device="cuda").normal_(generator=g)
    x, a, b = (new(N, 1, D).to(BF16) for _ in range(3))
    A, dt, h = new(D).abs(), new(D), new(N, D)
    out, hT, states = gdr.channel_scan_fwd(x, a, b, A, dt, h, want_states=True)
    dx, da, db, dA, ddt, dh0 = gdr.channel_scan_bwd(x, a, b, A, dt, states, x, None, h)
    tol = 2e-5 + U16
    rA, rdt = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for lo in range(0, N, 8192):
        r = slice(lo, lo + 8192)
        u = a[r, 0].double() + dt.double()
        la, al, be = gates(a[r, 0], b[r, 0], A, dt)
        h0, xr = h[r].double(), x[r, 0].double()
        ref = al * h0 + be * xr
        near(out[r, 0], ref, tol, "out")
        near(hT[r], ref, 2e-5, "hT")
        up = xr + h0  # dout is x, dhT is h0
        dla = al * h0 * up
        near(dx[r, 0], be * up, tol, "dx")
        near(db[r, 0], be * (1 - be) * xr * up, tol, "db")
        near(da[r, 0], -A.double().exp() * torch.sigmoid(u) * dla, tol, "da")
        near(dh0[r], al * up, 2e-5, "dh0")
        rA += (dla * la).sum(0)
        rdt += (-A.double().exp() * torch.sigmoid(u) * dla).sum(0)
    near(dA, rA, 2e-5, "dA_log")
    near(ddt, rdt, 2e-5, "ddt_bias")


def test_step_of_many_sequences(gdr):
    """2^32 + 2^12 states."""
    N, D = 2 ** 20 + 1, 4096
    say("channel scan step N %d D %d" % (N, D))
    x = torch.empty(N, D, dtype=BF16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    A, dt = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    state = torch.ones(N, D, device="cuda")
    out, same = gdr.channel_scan_step(x, x, x, A, dt, state, state)
    assert same is state
    for r in (slice(0, 64), slice(N // 2, N // 2 + 64), slice(N - 64, N)):
        _, al, be = gates(x[r], x[r], A, dt)
        ref = al + be * x[r].double()
        near(out[r], ref, 2e-5 + U16, "out")
        near(state[r], ref, 2e-5, "state")


def ce_rows(x, w, t, rows, piece=1 << 24):
    """(loss, lse) of the given tokens"""
    parts, pick = [], torch.zeros(len(rows), dtype=torch.float64, device="cuda")
    for lo in range(0, w.shape[0], piece):
        l = (x[rows].double()[:, None, :] * w[lo : lo + piece].double()[None]).sum(-1)
        parts.append(torch.logsumexp(l, 1))
        at = t[rows] - lo
        here = (at >= 0) & (at < l.shape[1])
        pick += torch.where(here, l.gather(1, at.clamp(0, l.shape[1] - 1)[:, None])[:, 0], torch.zeros_like(pick))
    lse = torch.logsumexp(torch.stack(parts), 0)
    return lse - pick, lse


@pytest.mark.parametrize("N,D,V", [(2 ** 16, 1, 2 ** 20 + 200), (2, 8, 2 ** 29 + 100), (2 ** 26 + 17, 8, 3)])
def test_cross_entropy(gdr, N, D, V):
    """Many tokens and a large vocabulary in rows that are not whole 16-byte pieces, a vocabulary past 2^29
    by rows, and more than 2^26 tokens to join."""
    say("linear ce N %d D %d V %d" % (N, D, V))
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(N, D, dtype=BF16, device="cuda").normal_(generator=g)
    w = torch.empty(V, D, dtype=BF16, device="cuda").normal_(generator=g)
    t = torch.empty(N, dtype=torch.int64, device="cuda").random_(0, V, generator=g)
    t[-1] = V - 1
    loss, lse = gdr.linear_ce_fwd(x, w, t)
    rows = torch.tensor(sorted({0, 1, N // 2 - 1, N // 2, N - 2, N - 1}), device="cuda")
    rl, rs = ce_rows(x, w, t, rows)
    near(loss[rows], rl, 1e-5, "loss")
    near(lse[rows], rs, 1e-5, "lse")
    if V > 100:
        return
    dl = torch.full((N,), 1.0, device="cuda")
    dx, dw = gdr.linear_ce_bwd(x, w, t, lse, dl)
    ref = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    for lo in range(0, N, 1 << 22):
        r = slice(lo, lo + (1 << 22))
        p = torch.softmax(x[r].double() @ w.double().T, 1)
        p.scatter_add_(1, t[r, None], torch.full((p.shape[0], 1), -1.0, dtype=torch.float64, device="cuda"))
        near(dx[r], p @ w.double(), 2e-5 + 2 * U16, "dx")
        ref += p.T @ x[r].double()
    near(dw, ref, 2e-5 + 2 * U16, "dw")
