"""Linear attention over sequences of thousands of tokens, against the sum over pairs of tokens in 64 bits on the GPU:

    out_t = sum_{s <= t} e^{c_t - c_s} (q_t . k_s) v_s + e^{c_t} h0^T q_t,   hT = sum_s e^{c_T - c_s} k_s v_s^T + e^{c_T} h0

for each sequence and value head, its gradients by automatic differentiation. Tolerances as in tests/_attn.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests._attn import TOL, attn_case, decay_bound, upstream
from tests._layers import BF16, FP32, U16, check, cuda, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    yield binding
    torch.cuda.empty_cache()


def by_pairs(q, k, v, la, h0, cu, dout, dhT):
    """out, hT, dq, dk, dv, dla, dh0 in 64 bits"""
    B, Hk, T, _ = q.shape
    Hv, head = v.shape[1], la.dim() == 1
    spans = [(b, 0, T) for b in range(B)] if cu is None else [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]
    new = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")
    out, hT, dq, dk, dv, dla, dh0 = new(v), new(h0), new(q), new(k), new(v), new(la), new(h0)
    for s, (b, lo, hi) in enumerate(spans):
        for j in range(Hv):
            i = j // (Hv // Hk)
            d = lambda t: t.double().requires_grad_()
            x, y, z, h = d(q[b, i, lo:hi]), d(k[b, i, lo:hi]), d(v[b, j, lo:hi]), d(h0[s, j])
            a = d(la[j].expand(hi - lo) if head else la[b, j, lo:hi])
            c = a.cumsum(0)
            ahead = torch.ones(hi - lo, hi - lo, dtype=torch.bool, device="cuda").triu(1)
            w = (c[:, None] - c[None, :]).masked_fill(ahead, float("-inf")).exp()
            o = (w * (x @ y.T)) @ z + c.exp()[:, None] * (x @ h)
            total = c[-1] if hi > lo else c.sum()
            e = ((total - c).exp()[:, None] * y).T @ z + total.exp() * h
            g = torch.autograd.grad((o * dout[b, j, lo:hi]).sum() + (e * dhT[s, j]).sum(), (x, y, z, a, h))
            out[b, j, lo:hi], hT[s, j] = o.detach(), e.detach()
            dq[b, i, lo:hi] += g[0]
            dk[b, i, lo:hi] += g[1]
            dv[b, j, lo:hi], dh0[s, j] = g[2], g[4]
            if head:
                dla[j] += g[3].sum()
            else:
                dla[b, j, lo:hi] = g[3]
    return [t.cpu().numpy() for t in (out, hT, dq, dk, dv, dla, dh0)]


def compare(gdr, lens, Hk, Hv, dk, dv, dtype, seed, packed, decay):
    say("long: %d sequences of %d tokens in all, Hk %d Hv %d dk %d dv %d %s %s" % (len(lens), sum(lens), Hk, Hv, dk, dv, dtype, decay))
    case = attn_case(lens, Hk, Hv, dk, dv, dtype, seed, packed, decay)
    dout, dhT = upstream(case, seed + 1)
    q, k, v, la, h, cu = cuda(case)
    gout, gh = cuda((dout, dhT))
    ref = by_pairs(q, k, v, la, h, case[5], gout, gh)
    r = U16 if dtype == BF16 else 0.0
    out, hT = gdr.linear_attn_fwd(q, k, v, la, h, cu)
    check(out, ref[0], TOL[dtype] + r, "out")
    check(hT, ref[1], TOL[dtype], "hT")
    got = gdr.linear_attn_bwd(q, k, v, la, gout, h, cu, gh)
    for name, x, y in zip(("dq", "dk", "dv"), got, ref[2:5]):
        check(x, y, TOL[dtype] + r, name)
    off = float(np.linalg.norm(got[3].double().cpu().numpy() - ref[5]))
    assert off <= decay_bound(case, dout, dhT, ref[2:], dtype, 4096), "dlog_alpha: %.3e off, of %.3e" % (off, np.linalg.norm(ref[5]))
    check(got[4], ref[6], TOL[dtype], "dh0")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens,Hk,Hv,decay", [([40] * 30 + [3000] + [40] * 33, 16, 16, "layer"), ([0, 20] * 25 + [2600] + [90] * 60 + [1200], 8, 16, "head"),
                                              ([2100] + [33] * 63 + [64], 16, 16, "slow")])
def test_one_long_sequence_among_many(gdr, lens, Hk, Hv, decay, dtype):
    """1024 workgroups and more of packed sequences, of which the forward cuts the long ones alone."""
    compare(gdr, lens, Hk, Hv, 64, 64, dtype, 900 + len(lens), True, decay)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens,Hk,Hv,dk,dv,packed,decay", [
    ([4300] * 3, 16, 32, 64, 32, False, "layer"), ([4300] * 3, 32, 32, 64, 64, False, "head"), ([4097], 32, 96, 64, 32, False, "slow"),
    ([4500] + [9] * 31, 16, 32, 64, 64, True, "layer"), ([0, 3] * 8 + [8300] + [9] * 20, 32, 32, 64, 96, True, "head"), ([5000], 8, 8, 128, 256, False, "layer")])
def test_segments_of_4096_tokens(gdr, lens, Hk, Hv, dk, dv, packed, decay, dtype):
    """So many heads that the backward is cut only where its sums would run over more than 4096 tokens, the last segment short
    (of four tokens, of one), and a plain cut."""
    compare(gdr, lens, Hk, Hv, dk, dv, dtype, 930 + len(lens) + dv, packed, decay)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens,Hk,Hv,dk,dv,packed,decay", [([6100], 40, 40, 64, 64, False, "layer"), ([3001, 17, 0, 2999], 20, 40, 64, 128, True, "head"),
                                                           ([2500, 2500], 24, 24, 128, 96, False, "slow")])
def test_segments_of_many_chunks(gdr, lens, Hk, Hv, dk, dv, packed, decay, dtype):
    compare(gdr, lens, Hk, Hv, dk, dv, dtype, 960 + len(lens) + dv, packed, decay)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_other_boundaries_in_one_graph(gdr, dtype):
    """A captured forward and backward, replayed with other packed boundaries of as many tokens: one long document here, another
    there, none at all, empty sequences; every replay has the eager calls' bits."""
    H, S = 16, 64
    lens = [[40] * 30 + [3000] + [40] * 33, [3000] + [40] * 63, [86] * 48 + [87] * 16, [0] * 50 + [2000, 0, 17, 3503] + [0] * 10]
    T = sum(lens[0])
    assert all(sum(x) == T and len(x) == S for x in lens)
    say("boundaries in a graph %s" % dtype)
    case = attn_case(lens[0], H, H, 64, 64, dtype, 990, True)
    dout, dhT = cuda(upstream(case, 991))
    q, k, v, la, h, cu = cuda(case)
    bounds = [torch.tensor([0] + x).cumsum(0).to(torch.int32).cuda() for x in lens]
    both = lambda: (*gdr.linear_attn_fwd(q, k, v, la, h, cu), *gdr.linear_attn_bwd(q, k, v, la, dout, h, cu, dhT))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for i in (1, 2, 3, 0, 2, 1):
        cu.copy_(bounds[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, both())), i


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens,H,packed", [([2000] * 3, 4, False), ([40] * 30 + [3000] + [40] * 33, 16, True), ([0, 700, 1, 0, 2500, 900], 2, True), ([60000], 1, False)])
def test_states_in_place(gdr, lens, H, packed, dtype):
    """The final states may replace the initial ones, of sequences that are cut too: all reads of them come before."""
    say("states in place %d sequences of %d tokens %s" % (len(lens), sum(lens), dtype))
    q, k, v, la, h, cu = cuda(attn_case(lens, H, H, 64, 64, dtype, 995 + len(lens), packed))
    out, hT = gdr.linear_attn_fwd(q, k, v, la, h, cu)
    for _ in range(5):
        state = h.clone()
        again, same = gdr.linear_attn_fwd(q, k, v, la, state, cu, hT=state)
        assert same is state and torch.equal(again, out) and torch.equal(state, hT)
