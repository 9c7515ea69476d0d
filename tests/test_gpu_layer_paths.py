"""The layer operators against the fp64 oracle at sizes that take them through every way of laying a call out
(tests/_layer_shapes.py): scans of several blocks a workgroup, whole and in chunks, the large tile of the products in
each of their forms, sliced products, many columns by rows. Tolerances are the operators' own tests'."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import layers as L
from tests import test_gpu_channel_scan as scan
from tests import test_gpu_gated_ffn as ffn
from tests import test_gpu_linear_ce as ce
from tests._layer_shapes import CES, FFNS, SCANS
from tests._layers import BF16, FP32, check, cuda, say, scan_case

pytestmark = pytest.mark.gpu
DT = {2: BF16, 4: FP32}


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lens,D,packed,es,_", SCANS)
def test_scans(gdr, lens, D, packed, es, _, reverse):
    scan.compare(gdr, lens, D, DT[es], 300 + D, packed=packed, reverse=reverse)


@pytest.mark.parametrize("lens,D,packed,es,_", SCANS)
def test_scans_with_slow_decay(gdr, lens, D, packed, es, _):
    """States that remember every token of a sequence: a wrong carry between blocks or chunks shows whole. The
    reference is the 64-bit recurrence over the gates as the kernels form them (the step's, of a state of 1 and of an
    input of 1): over 5000 remembered tokens the exponential's own error, -7e-9 a token in the mean on this card, is
    2e-5 by itself."""
    D, dtype = min(D, 1024) if not packed else D, DT[es]
    say("channel scan lens %s D %d %s slow, own gates" % (lens, D, dtype))
    x, a, b, A, dt, h, cu = scan_case(lens, D, dtype, 310, packed=packed, regime="slow")
    dout, dh = scan.upstream(x, len(lens), 311)
    gx, ga, gb, gA, gdt, gh, gcu, gdout, gdh = cuda((x, a, b, A, dt, h, cu, dout, dh))
    flat = lambda t: t.reshape(-1, D)
    zero, one = torch.zeros_like(flat(gx)), torch.ones_like(flat(gx))
    alpha = gdr.channel_scan_step(zero, flat(ga), flat(gb), gA, gdt, one.float())[1]
    beta = gdr.channel_scan_step(one, flat(ga), flat(gb), gA, gdt, zero.float())[1]
    alpha, beta = (L.f64(t.view(x.shape)) for t in (alpha, beta))
    out, hT, states = gdr.channel_scan_fwd(gx, ga, gb, gA, gdt, gh, gcu, want_states=True)
    got = gdr.channel_scan_bwd(gx, ga, gb, gA, gdt, states, gdout, gcu, gdh)
    X, up = L.f64(x), L.f64(dout)
    ref, dx, rT, d0 = (np.zeros_like(v) for v in (X, X, L.f64(h), L.f64(h)))
    for s, (row, idx) in enumerate(L.spans(x.shape[0], x.shape[1], cu, False)):
        state, g = L.f64(h)[s], L.f64(dh)[s]
        for t in idx:
            ref[row, t] = state = alpha[row, t] * state + beta[row, t] * X[row, t]
        rT[s] = state
        for t in idx[::-1]:
            g = g + up[row, t]
            dx[row, t] = beta[row, t] * g
            g = alpha[row, t] * g
        d0[s] = g
    for name, p, q in (("out", out, ref), ("hT", hT, rT), ("dx", got[0], dx), ("dh0", got[5], d0)):
        check(p, q, scan.TOL[p.dtype], name)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lens,D,packed,es,_", SCANS)
def test_scans_with_the_state_in_place(gdr, lens, D, packed, es, _, reverse):
    x, a, b, A, dt, h, cu = cuda(scan_case(lens, D, DT[es], 320, packed=packed))
    want, hT, _ = gdr.channel_scan_fwd(x, a, b, A, dt, h, cu, reverse=reverse)
    state = h.clone()
    out, same, _ = gdr.channel_scan_fwd(x, a, b, A, dt, state, cu, reverse=reverse, hT=state)
    assert same is state and torch.equal(out, want) and torch.equal(state, hT)


@pytest.mark.parametrize("M,D,F,es,_", FFNS)
def test_feed_forward(gdr, M, D, F, es, _):
    ffn.compare(gdr, M, D, F, DT[es])


@pytest.mark.parametrize("N,D,V,es,_", CES)
def test_cross_entropy(gdr, N, D, V, es, _):
    ce.compare(gdr, N, D, V, DT[es])


CONSTANT = [(609, 128, 1000), (609, 1032, 999), (38, 24, 33001), (4872, 1032, 2500), (58000, 8, 4801)]


@pytest.mark.parametrize("N,D,V", CONSTANT)
@pytest.mark.parametrize("power", [0, -30, -100])
def test_a_mean_over_tokens_loses_nothing_in_bf16(gdr, N, D, V, power):
    """Every token's dloss is 1/15 (times a power of two), which is 3.4e-3 of itself from the nearest bf16 number:
    rounded into dl it would be a common error of all results. The results' own rounding is 1.63e-3 of them (2^-8 /
    sqrt 3 over a uniform mantissa, at random), dl's large entries, p - 1, lose about p, 1e-3 at random: 2.2e-3 in all."""
    say("linear ce N %d D %d V %d, constant dloss, 2^%d" % (N, D, V, power))
    x, w, t, _ = ce.make(N, D, V, BF16, 330)
    dl = torch.full((N,), 2.0 ** power / 15.0)
    gx, gw, gt, gdl = (v.cuda() for v in (x, w, t, dl))
    lse = gdr.linear_ce_fwd(gx, gw, gt)[1]
    got = gdr.linear_ce_bwd(gx, gw, gt, lse, gdl)
    for name, p, q in zip(("dx", "dw"), got, L.ce_grads(x, w, t, dl)):
        check(p, q, 2.2e-3, name)


@pytest.mark.parametrize("value", [0.0, 1e-40, 1e-36, 3e37, 1e38])
def test_extreme_gradients_of_the_loss(gdr, value):
    """Past the range in which a common factor and its inverse are both normal numbers dl is formed without one."""
    x, w, t, _ = ce.make(40, 64, 300, BF16, 340)
    x, w = x * 0.125, w * 0.125
    dl = torch.full((40,), value)
    gx, gw, gt, gdl = (v.cuda() for v in (x, w, t, dl))
    lse = gdr.linear_ce_fwd(gx, gw, gt)[1]
    for name, p, q in zip(("dx", "dw"), gdr.linear_ce_bwd(gx, gw, gt, lse, gdl), L.ce_grads(x, w, t, dl)):
        if value < 1e-37:  # products below the smallest normal number, 1.2e-38, may vanish
            assert torch.isfinite(p).all() and p.abs().max().item() <= abs(q).max() + 64 * 1.2e-38
        else:
            check(p, q, ce.GRAD[BF16], name)
