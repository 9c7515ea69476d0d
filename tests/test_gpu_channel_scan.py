"""The channel scan (``gdr_channel_scan_fwd``, ``_bwd``, ``_step``) against the fp64 oracle.

Tolerances (relative Frobenius). Everything is computed in fp32 from the inputs as given. The gates'
exponentials and logarithms are good to about 2^-22; a state remembers at most some hundred tokens
in the "layer" regime and all of them in the "slow" one, whose decays differ from 1 by less than
2^-10 so that their own error is relative to that difference; errors add up over the remembered
tokens at random: 2e-5 leaves a factor of ten. bf16 outputs are rounded once more: 2^-8."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import layers as L
from tests._layers import BF16, FP32, U16, check, cuda, rel, say, scan_case

pytestmark = pytest.mark.gpu
TOL = {FP32: 2e-5, BF16: 2e-5 + U16}


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    return binding


def upstream(x, S, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(x.shape, generator=g).to(x.dtype), torch.randn(S, x.shape[2], generator=g)


def compare(gdr, lens, D, dtype, seed, packed=False, regime="layer", reverse=False, h0=True, dhT=True):
    say("channel scan lens %s D %d %s packed %s %s reverse %s" % (lens, D, dtype, packed, regime, reverse))
    x, a, b, A, dt, h, cu = scan_case(lens, D, dtype, seed, packed, regime, h0)
    dout, dh = upstream(x, len(lens), seed + 1)
    dh = dh if dhT else None
    gx, ga, gb, gA, gdt, gh, gcu, gdout, gdh = cuda((x, a, b, A, dt, h, cu, dout, dh))
    out, hT, states = gdr.channel_scan_fwd(gx, ga, gb, gA, gdt, gh, gcu, reverse=reverse, want_states=True)
    plain, hT2, none = gdr.channel_scan_fwd(gx, ga, gb, gA, gdt, gh, gcu, reverse=reverse)
    assert none is None and torch.equal(out, plain) and torch.equal(hT, hT2)
    got = gdr.channel_scan_bwd(gx, ga, gb, gA, gdt, states, gdout, gcu, gdh, reverse=reverse)
    again = gdr.channel_scan_bwd(gx, ga, gb, gA, gdt, states, gdout, gcu, gdh, reverse=reverse)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    ro, rh = L.scan(x, a, b, A, dt, h, cu, reverse)
    check(out, ro, TOL[dtype], "out")
    check(hT, rh, TOL[FP32], "hT")
    ref = L.scan_grads(x, a, b, A, dt, dout, h, cu, dh, reverse)
    for name, p, q in zip(("dx", "da", "db", "dA_log", "ddt_bias", "dh0"), got, ref):
        assert p.dtype == (dtype if name in ("dx", "da", "db") else FP32)
        check(p, q, TOL[p.dtype], name)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [1, 2, 7, 255, 256, 257, 1000])
def test_lengths(gdr, T, dtype):
    compare(gdr, [T, T], 96, dtype, 10 + T)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [1, 2, 15, 31, 33, 64, 130, 1001])
def test_channels(gdr, D, dtype):
    compare(gdr, [300], D, dtype, 50 + D)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lens", [[0, 5, 0, 1, 700, 0], [256, 256, 1], [3], [0, 0], [511, 513, 2, 1, 1, 90]])
def test_packed(gdr, lens, reverse, dtype):
    compare(gdr, lens, 40, dtype, 90 + sum(lens), packed=True, reverse=reverse)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("regime", ["slow", "wild"])
def test_regimes(gdr, regime, dtype):
    compare(gdr, [600, 600], 72, dtype, 130, regime=regime)


@pytest.mark.parametrize("lens,D,packed", [([6000], 33, False), ([9000], 64, False), ([5000, 40, 0, 4000], 48, True)])
def test_few_channels_next_to_the_length(gdr, lens, D, packed):
    compare(gdr, lens, D, FP32, 140, packed=packed)
    compare(gdr, lens, D, BF16, 141, packed=packed, reverse=True)


def test_no_initial_state_and_no_final_gradient(gdr):
    compare(gdr, [100, 100], 64, FP32, 150, h0=False, dhT=False)


def test_no_tokens(gdr):
    x, a, b, A, dt, h, _ = cuda(scan_case([4, 4], 20, FP32, 160))
    e = torch.empty(2, 0, 20, device="cuda")
    out, hT, states = gdr.channel_scan_fwd(e, e, e, A, dt, h, want_states=True)
    assert out.shape == e.shape and torch.equal(hT, h)
    got = gdr.channel_scan_bwd(e, e, e, A, dt, states, e, None, h)
    assert torch.equal(got[5], h) and not got[3].any() and not got[4].any()
    e = torch.empty(0, 3, 20, device="cuda")
    got = gdr.channel_scan_bwd(e, e, e, A, dt, gdr.channel_scan_fwd(e, e, e, A, dt, want_states=True)[2], e)
    assert not got[3].any() and not got[4].any()


def test_state_in_place_and_resume(gdr):
    x, a, b, A, dt, h, _ = cuda(scan_case([700, 700], 96, FP32, 170))
    whole, hT, _ = gdr.channel_scan_fwd(x, a, b, A, dt, h)
    state = h.clone()
    parts = []
    for lo, hi in ((0, 300), (300, 301), (301, 700)):
        o, s, _ = gdr.channel_scan_fwd(*(t[:, lo:hi].contiguous() for t in (x, a, b)), A, dt, state, hT=state)
        assert s is state
        parts.append(o)
    assert rel(torch.cat(parts, 1), whole.double().cpu().numpy()) < 2e-6
    assert rel(state, hT.double().cpu().numpy()) < 2e-6


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N,D", [(1, 1), (1, 2048), (3, 33), (256, 520)])
def test_step(gdr, N, D, dtype):
    say("channel scan step N %d D %d %s" % (N, D, dtype))
    x, a, b, A, dt, h, _ = scan_case([1] * N, D, dtype, 180 + D)
    ro, rh = L.scan(x, a, b, A, dt, h)
    gx, ga, gb = (t[:, 0].contiguous().cuda() for t in (x, a, b))
    state = h.cuda()
    out, new = gdr.channel_scan_step(gx, ga, gb, A.cuda(), dt.cuda(), state)
    check(out, ro[:, 0], TOL[dtype], "out")
    check(new, rh, TOL[FP32], "state")
    assert torch.equal(state.cpu(), h)
    out2, same = gdr.channel_scan_step(gx, ga, gb, A.cuda(), dt.cuda(), state, state)
    assert same is state and torch.equal(state, new) and torch.equal(out, out2)


def test_gradient_against_differences(gdr):
    """fp32 on the GPU: the loss's change along a random direction of every input against the
    gradient's product with it. Central differences with step 1/64: truncation of relative order
    step^2 = 2.4e-4 times a third derivative of order one next to the first, rounding of the two
    losses (each about 1e-6 of sums of order 1e2) over 2/64: 2e-2 of a slope of order 10 to 100 is
    allowed."""
    x, a, b, A, dt, h, _ = cuda(scan_case([40, 40], 16, FP32, 190))
    dout, dh = (t.cuda() for t in upstream(x, 2, 191))
    args = [x, a, b, A, dt, h]
    _, _, states = gdr.channel_scan_fwd(*args, want_states=True)
    got = gdr.channel_scan_bwd(*args[:5], states, dout, None, dh)
    g = torch.Generator().manual_seed(192)

    def loss(p):
        o, hT, _ = gdr.channel_scan_fwd(*p)
        return ((o.double() * dout).sum() + (hT.double() * dh).sum()).item()

    for k, grad in enumerate(got):
        d = torch.randn(args[k].shape, generator=g).cuda()
        d = torch.sign(grad) * d.abs()  # along the gradient's signs, so that the slope is large
        e = 1.0 / 64
        moved = lambda s: [t + s * e * d if i == k else t for i, t in enumerate(args)]
        slope = (loss(moved(1)) - loss(moved(-1))) / (2 * e)
        want = (grad.double() * d).sum().item()
        assert abs(slope - want) <= 2e-2 * abs(want), (k, slope, want)


def test_own_stream_and_graph(gdr):
    x, a, b, A, dt, h, cu = cuda(scan_case([300, 0, 41], 64, BF16, 200, packed=True))
    dout, dh = (t.cuda() for t in upstream(x, 3, 201))

    def step():
        o, hT, st = gdr.channel_scan_fwd(x, a, b, A, dt, h, cu, want_states=True)
        return (o, hT) + gdr.channel_scan_bwd(x, a, b, A, dt, st, dout, cu, dh)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        fresh = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, fresh))


def test_refusals(gdr):
    x, a, b, A, dt, h, _ = cuda(scan_case([8, 8], 16, FP32, 210))
    with pytest.raises(ValueError, match="a must have shape"):
        gdr.channel_scan_fwd(x, a[:, :4].contiguous(), b, A, dt)
    with pytest.raises(ValueError, match="b must be"):
        gdr.channel_scan_fwd(x, a, b.bfloat16(), A, dt)
    with pytest.raises(ValueError, match="contiguous"):
        gdr.channel_scan_fwd(x.transpose(0, 1).contiguous().transpose(0, 1), a, b, A, dt)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        gdr.channel_scan_fwd(x.half(), a.half(), b.half(), A, dt)
    with pytest.raises(ValueError, match="states"):
        gdr.channel_scan_bwd(x, a, b, A, dt, torch.empty(3, device="cuda"), x)
    with pytest.raises(gdr.GdrError, match="out overlaps x"):
        gdr.channel_scan_fwd(x, a, b, A, dt, out=x)
    with pytest.raises(gdr.GdrError, match="B == 1"):
        gdr.channel_scan_fwd(x, a, b, A, dt, None, torch.zeros(2, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("reverse", [False, True])
def test_long_scan_with_the_state_in_place(gdr, reverse):
    """Few channels, many tokens: the final state written over the initial one must not reach the
    workgroups that still have to start from it."""
    x, a, b, A, dt, h, cu = cuda(scan_case([20000, 3000, 0], 32, FP32, 220, packed=True))
    want, hT, _ = gdr.channel_scan_fwd(x, a, b, A, dt, h, cu, reverse=reverse)
    state = h.clone()
    out, same, _ = gdr.channel_scan_fwd(x, a, b, A, dt, state, cu, reverse=reverse, hT=state)
    assert same is state and torch.equal(out, want) and torch.equal(state, hT)


@pytest.mark.parametrize("T", [1, 300, 5000])
def test_empty_batch(gdr, T):
    _, _, _, A, dt, _, _ = cuda(scan_case([4], 20, FP32, 230))
    e = torch.empty(0, T, 20, device="cuda")
    out, hT, states = gdr.channel_scan_fwd(e, e, e, A, dt, want_states=True)
    assert out.shape == e.shape and hT.shape == (0, 20)
    got = gdr.channel_scan_bwd(e, e, e, A, dt, states, e)
    assert got[0].shape == e.shape and got[5].shape == (0, 20) and not got[3].any() and not got[4].any()


def train(gdr, x, a, b, A, dt, h, dout, reverse=False):
    out, hT, states = gdr.channel_scan_fwd(x, a, b, A, dt, h, reverse=reverse, want_states=True)
    return (out, hT) + gdr.channel_scan_bwd(x, a, b, A, dt, states, dout, reverse=reverse)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("T,D,B", [(3, 20, 1), (40, 64, 2), (300, 36, 1), (300, 4000, 2)])
def test_a_bad_value_stays_in_its_channel(gdr, T, D, B, reverse, dtype):
    """NaN or infinity in the inputs of one channel, at a token that ends or begins a sequence's ragged block:
    every result of the other channels keeps its bits."""
    x, a, b, A, dt, h, _ = cuda(scan_case([T] * B, D, dtype, 240 + T))
    dout = upstream(x, B, 241)[0].cuda()
    want = train(gdr, x, a, b, A, dt, h, dout, reverse)
    for t in sorted({0, T - 1, T // 256 * 256 % T, (T - 1) % 256}):
        for d in (0, 17):
            for name, bad in (("x", "inf"), ("x", "nan"), ("a", "nan"), ("b", "nan"), ("dout", "nan")):
                ins = dict(x=x, a=a, b=b, dout=dout)
                ins[name] = ins[name].clone()
                ins[name][0, t, d] = float(bad)
                got = train(gdr, ins["x"], ins["a"], ins["b"], A, dt, h, ins["dout"], reverse)
                keep = torch.arange(D) != d
                for k, (p, q) in enumerate(zip(got, want)):
                    assert torch.equal(p[..., keep], q[..., keep]), (t, d, name, bad, k)


@pytest.mark.parametrize("T", [40, 256, 300])
def test_an_infinite_last_input(gdr, T):
    """The last token's input reaches no state that a token begins with: the gates' gradients stay finite."""
    x, a, b, A, dt, h, _ = cuda(scan_case([T], 24, FP32, 250))
    dout, dh = (t.cuda() for t in upstream(x, 1, 251))
    x[0, T - 1, 3] = float("inf")
    states = gdr.channel_scan_fwd(x, a, b, A, dt, h, want_states=True)[2]
    dx, da, db, dA, ddt, dh0 = gdr.channel_scan_bwd(x, a, b, A, dt, states, dout, None, dh)
    assert all(torch.isfinite(t).all() for t in (dx, da, dA, ddt, dh0))
    assert torch.isinf(db[0, T - 1, 3]) and torch.isfinite(db[0, : T - 1]).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("T,D,B", [(40, 20, 1), (700, 36, 1), (300, 4000, 2)])
def test_a_nan_reaches_what_depends_on_it(gdr, T, D, B, reverse, dtype):
    """NaN in each input of one channel in turn: the results that are not finite are the oracle's."""
    x, a, b, A, dt, h, _ = scan_case([T] * B, D, dtype, 260 + T)
    dout = upstream(x, B, 261)[0]
    t, d = T // 2 + 3, 7
    for name in ("x", "a", "b", "dout"):
        say("channel scan NaN in %s, T %d D %d %s reverse %s" % (name, T, D, dtype, reverse))
        ins = dict(x=x, a=a, b=b, dout=dout)
        ins[name] = ins[name].clone()
        ins[name][0, t, d] = float("nan")
        got = train(gdr, *cuda((ins["x"], ins["a"], ins["b"], A, dt, h, ins["dout"])), reverse)
        # the oracle on the channel with the NaN
        one = [v[..., d : d + 1] for v in (ins["x"], ins["a"], ins["b"], A, dt, h)]
        ref = L.scan(*one, None, reverse) + L.scan_grads(*one[:5], ins["dout"][..., d : d + 1], one[5], None, None, reverse)
        for k, (p, q) in enumerate(zip(got, ref)):
            assert np.array_equal(torch.isfinite(p[..., d : d + 1]).cpu().numpy(), np.isfinite(q)), (name, k)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("level", [-20.0, -10.0, -6.0, 6.0, 10.0, 14.0, 17.0, 25.0, 40.0])
def test_gradient_of_open_and_shut_gates(gdr, level, dtype):
    """db = beta (1 - beta) x g keeps its bits where beta is 1 but for a small part, which the 64-bit reference
    forms as sigmoid(-b). The exponent's own rounding, 40 log2(e) 2^-24, is within the tolerances."""
    x, a, b, A, dt, h, _ = scan_case([300], 24, dtype, 270)
    b = torch.full_like(b, level)
    dout, dh = upstream(x, 1, 271)
    ref = L.scan_grads(x, a, b, A, dt, dout, h, None, dh)
    db = ref[0] * L.f64(x) / (1.0 + np.exp(level))
    gx, ga, gb, gA, gdt, gh, gdout, gdh = cuda((x, a, b, A, dt, h, dout, dh))
    states = gdr.channel_scan_fwd(gx, ga, gb, gA, gdt, gh, want_states=True)[2]
    got = gdr.channel_scan_bwd(gx, ga, gb, gA, gdt, states, gdout, None, gdh)
    check(got[2], db, TOL[dtype], "db")
    check(got[0], ref[0], TOL[dtype], "dx")
