"""Linear cross entropy (``gdr_linear_ce_fwd``, ``_bwd``) against the fp64 oracle.

Tolerances (relative Frobenius). The loss and lse come from fp32 logits (sums of D products of the
inputs as given) and fp32 exponentials: 1e-5 (of the losses' norm) in either type. Gradients, fp32:
1e-5 for the products and 2^-22 times the logits' range of about 10 for the exponentials: 2e-5. bf16:
the piece's gradient and the result are each rounded once, 2 * 2^-8."""
from __future__ import annotations

import pytest
import torch

from oracle import layers as L
from tests._layers import BF16, FP32, U16, check, rel, say

pytestmark = pytest.mark.gpu
LOSS = 1e-5
GRAD = {FP32: 2e-5, BF16: 2e-5 + 2 * U16}


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    return binding


def make(N, D, V, dtype, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    t = torch.randint(0, V, (N,), generator=g)
    if N > 3:
        t[1], t[2], t[3] = -100, V, V - 1
    return n(N, D).to(dtype), (n(V, D) * scale * D ** -0.5).to(dtype), t, torch.rand(N, generator=g)


def compare(gdr, N, D, V, dtype, seed=1, scale=2.0):
    say("linear ce N %d D %d V %d %s" % (N, D, V, dtype))
    x, w, t, dl = make(N, D, V, dtype, seed, scale)
    gx, gw, gt, gdl = (v.cuda() for v in (x, w, t, dl))
    loss, lse = gdr.linear_ce_fwd(gx, gw, gt)
    got = gdr.linear_ce_bwd(gx, gw, gt, lse, gdl)
    l2, s2 = gdr.linear_ce_fwd(gx, gw, gt)
    again = gdr.linear_ce_bwd(gx, gw, gt, lse, gdl)
    torch.cuda.synchronize()
    assert torch.equal(loss, l2) and torch.equal(lse, s2) and all(torch.equal(p, q) for p, q in zip(got, again))
    rl, rs = L.ce(x, w, t)
    check(loss, rl, LOSS, "loss")
    check(lse, rs, LOSS, "lse")
    for name, p, q in zip(("dx", "dw"), got, L.ce_grads(x, w, t, dl)):
        assert p.dtype == dtype
        check(p, q, GRAD[dtype], name)
    off = (t < 0) | (t >= V)
    assert not loss.cpu()[off].any() and not got[0].cpu()[off].any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 33, 64, 65, 129, 257, 600])
def test_tokens(gdr, N, dtype):
    compare(gdr, N, 128, 1000, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D,V", [(1, 1), (1, 7), (3, 2), (8, 31), (24, 33), (40, 255), (64, 257), (100, 513), (136, 5001), (513, 300)])
def test_widths(gdr, D, V, dtype):
    compare(gdr, 20, D, V, dtype)
    compare(gdr, 150, D, V, dtype)
    compare(gdr, 3, D, V, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_several_pieces(gdr, dtype):
    """Many tokens: the vocabulary is taken in more than one piece."""
    compare(gdr, 60001, 8, 4801, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_pieces_of_few_tokens(gdr, dtype):
    """Few tokens and a vocabulary past the longest row of a piece, 2^20."""
    compare(gdr, 5, 16, 2 ** 20 + 1001, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_tiles_ragged(gdr, dtype):
    compare(gdr, 1100, 264, 3001, dtype)


@pytest.mark.parametrize("N,D,V", [(4097, 72, 3201), (4097, 3336, 40), (40, 3600, 3593)])
def test_large_outputs(gdr, N, D, V):
    """Wide in turn in each product's result: the logits, dx and dw."""
    compare(gdr, N, D, V, BF16)


@pytest.mark.parametrize("N", [4, 200])
def test_sharp_logits(gdr, N):
    """Logits up to some hundreds: all but one probability vanish, exponentials must not overflow."""
    compare(gdr, N, 64, 700, FP32, scale=80.0)
    x, w, t, dl = (v.cuda() for v in make(N, 64, 700, BF16, 3, scale=4000.0))
    loss, lse = gdr.linear_ce_fwd(x, w, t)
    dx, dw = gdr.linear_ce_bwd(x, w, t, lse, dl)
    assert all(torch.isfinite(v).all() for v in (loss, lse, dx, dw))


@pytest.mark.parametrize("N", [6, 300])
def test_masked_vocabulary_and_masked_tokens(gdr, N):
    """Vocabulary rows that push logits to the type's lowest value bear no probability; with every
    target outside the vocabulary the loss and the gradients are zero, whatever dloss holds."""
    x, w, t, dl = make(N, 40, 500, FP32, 5)
    x[:, 0] = 1.0
    w[100:400] = 0.0
    w[100:400, 0] = torch.finfo(FP32).min
    t[:] = 7
    gx, gw, gt, gdl = (v.cuda() for v in (x, w, t, dl))
    loss, lse = gdr.linear_ce_fwd(gx, gw, gt)
    keep = torch.cat([w[:100], w[400:]])
    check(loss, L.ce(x, keep, t)[0], LOSS, "loss")
    dx, dw = gdr.linear_ce_bwd(gx, gw, gt, lse, gdl)
    assert not dw[100:400].any()
    check(dx, L.ce_grads(x, keep, t, dl)[0], GRAD[FP32], "dx")
    none = torch.full_like(gt, -1)
    loss, lse2 = gdr.linear_ce_fwd(gx, gw, none)
    assert not loss.any() and torch.equal(lse, lse2)
    dx, dw = gdr.linear_ce_bwd(gx, gw, none, lse, torch.full_like(gdl, float("nan")))
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("N", [4, 200])
def test_a_bad_row_stays_in_its_row(gdr, N):
    x, w, t, dl = (v.cuda() for v in make(N, 64, 333, BF16, 6))
    want, _ = gdr.linear_ce_fwd(x, w, t)
    bad = x.clone()
    bad[0, 3] = float("nan")
    got, _ = gdr.linear_ce_fwd(bad, w, t)
    assert torch.equal(got[1:], want[1:]) and torch.isnan(got[0])


def test_no_tokens(gdr):
    x, w, t, dl = (v.cuda() for v in make(3, 32, 48, BF16, 7))
    loss, lse = gdr.linear_ce_fwd(x[:0], w, t[:0])
    dx, dw = gdr.linear_ce_bwd(x[:0], w, t[:0], lse, loss)
    assert loss.shape == (0,) and dx.shape == (0, 32) and not dw.any()


def test_gradient_against_differences(gdr):
    """fp32: the loss along a direction of each input against the gradient (step 1/128, as in the
    feed-forward's test)."""
    x, w, t, dl = (v.cuda() for v in make(20, 24, 60, FP32, 8))
    loss, lse = gdr.linear_ce_fwd(x, w, t)
    for k, grad in enumerate(gdr.linear_ce_bwd(x, w, t, lse, dl)):
        g = torch.Generator().manual_seed(9 + k)
        d = torch.sign(grad) * torch.randn(grad.shape, generator=g).abs().cuda() * 0.2
        e = 1.0 / 128
        f = lambda s: (gdr.linear_ce_fwd(*[v + s * e * d if i == k else v for i, v in enumerate((x, w))], t)[0].double() * dl).sum().item()
        slope, want = (f(1) - f(-1)) / (2 * e), (grad.double() * d).sum().item()
        assert abs(slope - want) <= 2e-2 * abs(want), (k, slope, want)


@pytest.mark.parametrize("N", [2, 90])
def test_own_stream_and_graph(gdr, N):
    x, w, t, dl = (v.cuda() for v in make(N, 136, 900, BF16, 10))

    def step():
        loss, lse = gdr.linear_ce_fwd(x, w, t)
        return (loss, lse) + gdr.linear_ce_bwd(x, w, t, lse, dl)

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
    x, w, t, dl = (v.cuda() for v in make(6, 16, 24, FP32, 11))
    with pytest.raises(ValueError, match="weight must have shape"):
        gdr.linear_ce_fwd(x, w[:, :8].contiguous(), t)
    with pytest.raises(ValueError, match="targets must be"):
        gdr.linear_ce_fwd(x, w, t.int())
    with pytest.raises(ValueError, match="lse must have shape"):
        gdr.linear_ce_bwd(x, w, t, dl[:3], dl)
    with pytest.raises(gdr.GdrError, match="workspace"):
        gdr.linear_ce_bwd(x, w, t, dl, dl.clone(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N,D,V", [(1, 16, 40), (6, 64, 333), (7, 13, 50), (300, 64, 333), (520, 100, 2000), (60001, 8, 4801)])
def test_rows_without_a_loss_may_hold_anything(gdr, N, D, V, dtype):
    """NaN and infinity in x where the target is outside the vocabulary: no loss, and no gradient of the weights or
    of any token, to the bit."""
    x, w, t, dl = make(N, D, V, dtype, 12)
    t[:: 3] = -100
    gx, gw, gt, gdl = (v.cuda() for v in (x, w, t, dl))
    off = (gt < 0) | (gt >= V)
    loss, lse = gdr.linear_ce_fwd(gx, gw, gt)
    want = gdr.linear_ce_bwd(gx, gw, gt, lse, gdl)
    for value in ("nan", "inf"):
        bad = gx.clone()
        bad[off] = float(value)
        got, lse2 = gdr.linear_ce_fwd(bad, gw, gt)
        assert torch.equal(got, loss) and torch.equal(lse2[~off], lse[~off])
        bdl = torch.where(off, torch.full_like(gdl, float(value)), gdl)
        assert all(torch.equal(p, q) for p, q in zip(gdr.linear_ce_bwd(bad, gw, gt, lse2, bdl), want))
