"""Which gradients of linear attention a token that is not finite reaches: those whose formula holds it, and no other.

    dq_t = H_t dout_t    dk_t = G_t v_t    dv_t = G_t^T k_t    dlog_alpha_t = alpha_t <G_t, H_{t-1}>    dh0 = alpha_1 G_1

with H_t of k, v and log_alpha up to t and of h0, and G_t of q and dout from t on, of log_alpha behind t and of dhT."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import linear_attn as O
from tests._attn import attn_case, decay_bound, upstream
from tests._layers import BF16, FP32, cuda, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    return binding


def reached(which, t, T):
    """tokens of dq, dk, dv and dlog_alpha, and whether dh0, that a bad token t of an input may reach"""
    at, on, behind, before, to, none, every = [t], range(t, T), range(t + 1, T), range(t), range(t + 1), [], range(T)
    return {"q": (none, to, to, to, True), "k": (on, none, at, behind, False), "v": (on, at, none, behind, False),
            "log_alpha": (on, before, before, every, True), "dout": (at, to, to, to, True),
            "h0": (every, none, none, every, False), "dhT": (none, every, every, every, True)}[which]


SIZES = [(64, 64, 64, False), (300, 64, 96, False), (700, 64, 64, False), (1100, 128, 64, True)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,dk,dv,packed", SIZES)
@pytest.mark.parametrize("which", ["q", "k", "v", "log_alpha", "dout", "h0", "dhT"])
def test_a_bad_token(gdr, which, T, dk, dv, packed, dtype):
    """One row of one head of the first sequence: other heads, the other sequence and all gradients whose formula does not hold the
    row keep their bits; the gradients of the decays up to a bad key or value keep their value (they come another way then)."""
    say("bad %s T %d dk %d dv %d %s" % (which, T, dk, dv, dtype))
    lens = [T, 70] if packed else [T, T]
    case = attn_case(lens, 2, 2, dk, dv, dtype, 800 + T + dk + dv, packed)
    dout, dhT = upstream(case, 801)
    q, k, v, la, h, cu = cuda(case)
    given = dict(q=q, k=k, v=v, log_alpha=la, dout=dout.cuda(), h0=h, dhT=dhT.cuda())
    back = lambda a: gdr.linear_attn_bwd(a["q"], a["k"], a["v"], a["log_alpha"], a["dout"], a["h0"], cu, a["dhT"])
    clean = back(given)
    ref = O.grads(*case[:4], dout, case[4], case[5], dhT)
    bound = decay_bound(case, dout, dhT, ref, dtype, 4096)
    for bad in (float("nan"), float("inf")):
        if which == "log_alpha" and bad > 0:
            continue  # not a decay
        for t in ([0] if which in ("h0", "dhT") else [0, 5, T // 2 + 3, T - 1]):
            moved = dict(given)
            moved[which] = given[which].clone()
            moved[which][(0, 1, 3, 2) if which in ("h0", "dhT") else (0, 1, t)] = bad
            got = back(moved)
            *rows, state = reached(which, t, T)
            for i, (x, c) in enumerate(zip(got, clean)):
                x, c = x.clone(), c.clone()
                if i == 4:
                    if state:
                        assert not torch.isfinite(x[0, 1]).all()
                        x[0, 1] = c[0, 1]
                else:
                    hit = list(rows[i])
                    if hit:
                        assert not torch.isfinite(x[0, 1, hit].flatten(1) if i < 3 else x[0, 1, hit][:, None]).all(1).any(), (i, t)
                    if i == 3 and which in ("k", "v"):
                        # H before t and G from t on, by recurrences of at most T steps, 2^-24 off a step and independently
                        part = lambda z, lo, hi: z[:1, 1:, lo:hi].double()
                        _, H = O.forward(*(part(z, 0, t) for z in case[:4]), case[4][:1, 1:])
                        later = [part(z, t, T).clone() for z in case[:4]]
                        later[3][:, :, 0] = 0.0  # (not the token's own decay)
                        G = O.grads(*later, part(dout, t, T), None, None, dhT[:1, 1:].double())[4]
                        one = T ** 0.5 * 2 ** -24 * np.linalg.norm(H) * np.linalg.norm(G)
                        off = np.linalg.norm(x[0, 1, :t + 1].double().cpu().numpy() - ref[3][0, 1, :t + 1])
                        assert off <= bound + (t + 1) ** 0.5 * one, (t, off, bound, one)
                        hit = range(T)
                    x[0, 1, list(hit)] = c[0, 1, list(hit)]
                assert torch.equal(x, c), (bad, t, i)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [90, 700])
def test_one_decay_a_head(gdr, T, dtype):
    """A bad value of the last token alone: the head's gradient is the sum of finite ones."""
    case = attn_case([T], 2, 2, 64, 64, dtype, 860, decay="head")
    dout, _ = upstream(case, 861)
    q, k, v, la, h, _ = cuda(case)
    ref = O.grads(*case[:4], dout, case[4])
    for t, whole in ((T - 1, True), (T - 2, False)):
        moved = v.clone()
        moved[0, 1, t] = float("nan")
        got = gdr.linear_attn_bwd(q, k, moved, la, dout.cuda(), h)[3]
        assert torch.isfinite(got).tolist() == [True, whole]
        if whole:
            assert np.linalg.norm(got.double().cpu().numpy() - ref[3]) <= 2 * decay_bound(case, dout, None, ref, dtype, 4096)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [90, 700])
def test_shared_heads(gdr, T, dtype):
    """A bad value head: the key head's gradients of the queries from there on and of that key, nothing else of other value heads."""
    case = attn_case([T], 1, 3, 64, 64, dtype, 870)
    dout, dhT = upstream(case, 871)
    q, k, v, la, h, _ = cuda(case)
    args = lambda v: (q, k, v, la, dout.cuda(), h, None, dhT.cuda())
    clean, t = gdr.linear_attn_bwd(*args(v)), 37
    moved = v.clone()
    moved[0, 1, t] = float("nan")
    got = gdr.linear_attn_bwd(*args(moved))
    assert torch.equal(got[0][:, :, :t], clean[0][:, :, :t]) and torch.isnan(got[0][:, :, t:]).all()
    assert torch.isnan(got[1][:, :, t]).all() and torch.equal(torch.cat([got[1][:, :, :t], got[1][:, :, t + 1:]], 2), torch.cat([clean[1][:, :, :t], clean[1][:, :, t + 1:]], 2))
    assert torch.equal(got[2], clean[2]) and torch.equal(got[4], clean[4])
    assert torch.equal(got[3][:, [0, 2]], clean[3][:, [0, 2]]) and torch.isfinite(got[3][:, 1, :t + 1]).all() and torch.isnan(got[3][:, 1, t + 1:]).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [130, 900])
def test_decays_that_leave_nothing(gdr, T, dtype):
    """alpha of 0 to the last bit of fp32 has a gradient of 0, whatever the sums it is taken from."""
    case = attn_case([T], 1, 2, 64, 64, dtype, 880)
    dout, dhT = upstream(case, 881)
    q, k, v, la, h, _ = cuda(case)
    for least in (float("-inf"), -1e30, -500.0, -104.0):
        cut = la.clone()
        cut[0, 0, 70:73], cut[0, 1, T - 1] = least, least
        got = gdr.linear_attn_bwd(q, k, v, cut, dout.cuda(), h, None, dhT.cuda())[3]
        assert not got[0, 0, 70:73].any() and got[0, 1, T - 1] == 0
        assert got[0, 0, :70].all() and got[0, 0, 73:].all()
    head = torch.tensor([float("-inf"), -0.1], device="cuda")
    got = gdr.linear_attn_bwd(q, k, v, head, dout.cuda(), h, None, dhT.cuda())[3]
    assert got[0] == 0 and got[1] != 0
