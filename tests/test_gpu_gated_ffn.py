"""The gated feed-forward block (``gdr_gated_ffn_fwd``, ``_bwd``) against the fp64 oracle.

Tolerances (relative Frobenius). fp32: sums of D, F or M products in fp32, errors at random, and
exponentials good to about 2^-22: 1e-5. bf16 forward: one rounding of the result, 2^-8, and the
fp32 part. bf16 backward: the kept gate and up, the gradient entering the products and the result
are each rounded once; the activation's slope moves by no more than its argument does: five
roundings, 5 * 2^-8."""
from __future__ import annotations

import pytest
import torch

from oracle import layers as L
from tests._layers import BF16, FP32, U16, check, say

pytestmark = pytest.mark.gpu
FWD = {FP32: 1e-5, BF16: 1e-5 + U16}
BWD = {FP32: 1e-5, BF16: 5 * U16}


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    return binding


def make(M, D, F, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    return (n(M, D).to(dtype), (n(F, D) * D ** -0.5).to(dtype), (n(F, D) * D ** -0.5).to(dtype), n(M, F).to(dtype))


def compare(gdr, M, D, F, dtype, act="silu", seed=1):
    say("gated ffn M %d D %d F %d %s %s" % (M, D, F, dtype, act))
    x, wg, wu, dh = make(M, D, F, dtype, seed)
    gx, gwg, gwu, gdh = (t.cuda() for t in (x, wg, wu, dh))
    h, gate, up = gdr.gated_ffn_fwd(gx, gwg, gwu, act=act, want_saved=True)
    h2, no1, no2 = gdr.gated_ffn_fwd(gx, gwg, gwu, act=act)
    assert no1 is None and no2 is None and torch.equal(h, h2)
    got = gdr.gated_ffn_bwd(gx, gwg, gwu, gate, up, gdh, act=act)
    again = gdr.gated_ffn_bwd(gx, gwg, gwu, gate, up, gdh, act=act)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    check(h, L.ffn(x, wg, wu, act), FWD[dtype], "h")
    check(gate, L.f64(x) @ L.f64(wg).T, FWD[dtype], "gate")
    check(up, L.f64(x) @ L.f64(wu).T, FWD[dtype], "up")
    for name, p, q in zip(("dx", "dw_gate", "dw_up"), got, L.ffn_grads(x, wg, wu, dh, act)):
        assert p.dtype == dtype
        check(p, q, BWD[dtype], name)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 129, 257, 515])
def test_tokens(gdr, M, dtype):
    compare(gdr, M, 256, 320, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D,F", [(1, 1), (3, 5), (8, 9), (24, 17), (40, 127), (64, 130), (100, 33), (136, 1023), (513, 64)])
def test_widths(gdr, D, F, dtype):
    compare(gdr, 37, D, F, dtype)
    compare(gdr, 300, D, F, dtype)
    compare(gdr, 2, D, F, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M", [5, 200])
def test_gelu(gdr, M, dtype):
    compare(gdr, M, 128, 192, dtype, act="gelu_tanh")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_tiles_ragged(gdr, dtype):
    compare(gdr, 1000, 520, 1301, dtype)
    compare(gdr, 2049, 264, 515, dtype)


@pytest.mark.parametrize("M,D,F", [(4097, 72, 1601), (4097, 3336, 24), (33, 3600, 3592)])
def test_large_outputs(gdr, M, D, F):
    """Wide in turn in each product's result: h and its projections, dx, and the weights' gradients."""
    compare(gdr, M, D, F, BF16)


def test_no_tokens(gdr):
    x, wg, wu, _ = (t.cuda() for t in make(3, 32, 48, BF16, 2))
    e, eh = x[:0], torch.empty(0, 48, dtype=BF16, device="cuda")
    h, gate, up = gdr.gated_ffn_fwd(e, wg, wu, want_saved=True)
    assert h.shape == (0, 48)
    dx, dwg, dwu = gdr.gated_ffn_bwd(e, wg, wu, gate, up, eh)
    assert dx.shape == (0, 32) and not dwg.any() and not dwu.any()


def test_leading_dimensions(gdr):
    x, wg, wu, dh = (t.cuda() for t in make(12, 32, 48, FP32, 3))
    h, gate, up = gdr.gated_ffn_fwd(x, wg, wu, want_saved=True)
    h3, gate3, up3 = gdr.gated_ffn_fwd(x.view(3, 4, 32), wg, wu, want_saved=True)
    assert h3.shape == (3, 4, 48) and torch.equal(h3.view(12, 48), h)
    dx3 = gdr.gated_ffn_bwd(x.view(3, 4, 32), wg, wu, gate3, up3, dh.view(3, 4, 48))[0]
    assert torch.equal(dx3.view(12, 32), gdr.gated_ffn_bwd(x, wg, wu, gate, up, dh)[0])


@pytest.mark.parametrize("M", [3, 100])
def test_a_bad_row_stays_in_its_row(gdr, M):
    """NaN and infinity in one token's input, and large gates, leave the other tokens as they were."""
    x, wg, wu, _ = (t.cuda() for t in make(M, 64, 96, BF16, 4))
    want = gdr.gated_ffn_fwd(x, wg, wu)[0]
    bad = x.clone()
    bad[1, 5], bad[1, 9] = float("nan"), float("inf")
    got = gdr.gated_ffn_fwd(bad, wg, wu)[0]
    keep = [i for i in range(M) if i != 1]
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[1]).any()
    for act in ("silu", "gelu_tanh"):
        big = (x * 1e4).bfloat16()
        h, gate, up = gdr.gated_ffn_fwd(big, wg, wu, act=act, want_saved=True)
        assert torch.isfinite(h).all()
        assert all(torch.isfinite(t).all() for t in gdr.gated_ffn_bwd(big, wg, wu, gate, up, want, act=act))


def test_gradient_against_differences(gdr):
    """fp32: the loss along a direction of each input against the gradient. Step 1/128 relative to
    inputs of order one: truncation below 1e-3 of the slope, rounding of the losses below 1e-3 of it."""
    x, wg, wu, dh = (t.cuda() for t in make(20, 24, 36, FP32, 5))
    args = [x, wg, wu]
    _, gate, up = gdr.gated_ffn_fwd(*args, want_saved=True)
    for k, grad in enumerate(gdr.gated_ffn_bwd(*args, gate, up, dh)):
        g = torch.Generator().manual_seed(6 + k)
        d = torch.sign(grad) * torch.randn(grad.shape, generator=g).abs().cuda() * (1.0 if k == 0 else 24 ** -0.5)
        e = 1.0 / 128
        f = lambda s: (gdr.gated_ffn_fwd(*[t + s * e * d if i == k else t for i, t in enumerate(args)])[0].double() * dh).sum().item()
        slope, want = (f(1) - f(-1)) / (2 * e), (grad.double() * d).sum().item()
        assert abs(slope - want) <= 2e-2 * abs(want), (k, slope, want)


@pytest.mark.parametrize("M", [1, 70, 300])
def test_own_stream_and_graph(gdr, M):
    x, wg, wu, dh = (t.cuda() for t in make(M, 136, 200, BF16, 7))

    def step():
        h, gate, up = gdr.gated_ffn_fwd(x, wg, wu, want_saved=True)
        return (h,) + gdr.gated_ffn_bwd(x, wg, wu, gate, up, dh)

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
    x, wg, wu, dh = (t.cuda() for t in make(6, 16, 24, FP32, 8))
    with pytest.raises(ValueError, match="w_up must have shape"):
        gdr.gated_ffn_fwd(x, wg, wu[:8])
    with pytest.raises(ValueError, match="act must be"):
        gdr.gated_ffn_fwd(x, wg, wu, act="tanh")
    with pytest.raises(ValueError, match="contiguous"):
        gdr.gated_ffn_fwd(x, wg.t().contiguous().t(), wu)
    with pytest.raises(ValueError, match="gate must"):
        gdr.gated_ffn_bwd(x, wg, wu, dh.bfloat16(), dh, dh)
    with pytest.raises(gdr.GdrError, match="workspace"):
        gdr.gated_ffn_bwd(x, wg, wu, dh, dh.clone(), dh.clone(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("F", [12, 500, 36, 16, 13])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_padding_of_the_gradients_rows(gdr, F, dtype):
    """The backward's workspace begins with dG and dU, rows of F rounded up to 8 columns. The columns past F
    hold zeros and nothing that lies behind a row of gate, up or dh; here each is the head of a larger
    tensor of ones."""
    M, D, ld = 5, 16, (F + 7) // 8 * 8
    x, wg, wu, _ = (t.cuda() for t in make(M, D, F, dtype, 9))
    heads = [torch.ones(M * F + 64, dtype=dtype, device="cuda")[: M * F].view(M, F) for _ in range(3)]
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    gdr.gated_ffn_bwd(x, wg, wu, *heads, workspace=ws)
    kept = ws[: 2 * M * ld * x.element_size()].view(dtype).view(2, M, ld)
    assert torch.isfinite(kept).all() and kept[:, :, :F].any()
    assert not kept[:, :, F:].any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_slope_of_huge_gates(gdr, act, dtype):
    """Past a few tens the activation is nearly 0 or the identity, its slope 0 or 1, up to the type's largest
    values: each element within the backward's tolerance of the 64-bit one, or of 1."""
    v = torch.tensor([50.0, 1e3, 2e4, 3e13, 3e19, 1e30, 3e38])
    gate = torch.cat([v, -v]).to(dtype).cuda()[None]
    F = gate.shape[1]
    up, dh = torch.ones_like(gate), torch.ones_like(gate)
    x, w = torch.ones(1, 8, dtype=dtype, device="cuda"), torch.zeros(F, 8, dtype=dtype, device="cuda")
    dx, dwg, dwu = gdr.gated_ffn_bwd(x, w, w, gate, up, dh, act=act)
    val, slope = L.act_and_slope(L.f64(gate[0]), act)
    assert not dx.any()
    for got, ref in ((dwg, slope), (dwu, val)):
        assert (abs(L.f64(got) - ref[:, None]) <= BWD[dtype] * (1.0 + abs(ref[:, None]))).all()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,D,F", [(300, 256, 320), (33, 512, 1000), (1000, 520, 1301), (2050, 1032, 2200), (300, 100, 333)])
def test_gradients_with_two_roundings(gdr, M, D, F, act):
    """bf16 with gate and up kept in fp32, as is the default: dG and dU are rounded as operands and the gradients as
    results, each about 1.65e-3 of them at random, 2.35e-3 together; a third rounding makes it 2.9e-3 and more."""
    say("gated ffn M %d D %d F %d %s" % (M, D, F, act))
    x, wg, wu, dh = make(M, D, F, BF16, 20)
    gx, gwg, gwu, gdh = (t.cuda() for t in (x, wg, wu, dh))
    h, gate, up = gdr.gated_ffn_fwd(gx, gwg, gwu, act=act, want_saved=True)
    assert gate.dtype == up.dtype == FP32
    check(gate, L.f64(x) @ L.f64(wg).T, FWD[FP32], "gate")
    check(up, L.f64(x) @ L.f64(wu).T, FWD[FP32], "up")
    got = gdr.gated_ffn_bwd(gx, gwg, gwu, gate, up, gdh, act=act)
    for name, p, q in zip(("dx", "dw_gate", "dw_up"), got, L.ffn_grads(x, wg, wu, dh, act)):
        assert p.dtype == BF16
        check(p, q, 2.6e-3, name)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,D,F", [(1, 64, 96), (40, 64, 97), (300, 256, 320), (2049, 264, 515), (5558, 1864, 2199), (30, 33, 50)])
def test_kept_in_bf16(gdr, M, D, F, act):
    say("gated ffn, kept in bf16, M %d D %d F %d %s" % (M, D, F, act))
    x, wg, wu, dh = make(M, D, F, BF16, 21)
    gx, gwg, gwu, gdh = (t.cuda() for t in (x, wg, wu, dh))
    h, gate, up = gdr.gated_ffn_fwd(gx, gwg, gwu, act=act, want_saved=True, saved_dtype=BF16)
    h2, gate2, up2 = gdr.gated_ffn_fwd(gx, gwg, gwu, act=act, want_saved=True)
    assert torch.equal(h, h2) and torch.equal(gate, gate2.bfloat16()) and torch.equal(up, up2.bfloat16())
    got = gdr.gated_ffn_bwd(gx, gwg, gwu, gate, up, gdh, act=act)
    wide = gdr.gated_ffn_bwd(gx, gwg, gwu, gate.float(), up.float(), gdh, act=act)
    assert all(torch.equal(p, q) for p, q in zip(got, wide))
    for name, p, q in zip(("dx", "dw_gate", "dw_up"), got, L.ffn_grads(x, wg, wu, dh, act)):
        check(p, q, BWD[BF16], name)


def test_refusals_of_kept_types(gdr):
    x, wg, wu, dh = (t.cuda() for t in make(6, 16, 24, BF16, 22))
    h, gate, up = gdr.gated_ffn_fwd(x, wg, wu, want_saved=True)
    with pytest.raises(ValueError, match="saved_dtype must be"):
        gdr.gated_ffn_fwd(x, wg, wu, want_saved=True, saved_dtype=torch.float16)
    with pytest.raises(ValueError, match="saved_dtype must be"):
        gdr.gated_ffn_fwd(x.float(), wg.float(), wu.float(), want_saved=True, saved_dtype=BF16)
    with pytest.raises(ValueError, match="up must be"):
        gdr.gated_ffn_bwd(x, wg, wu, gate, up.bfloat16(), dh)
    with pytest.raises(ValueError, match="gate must be"):
        gdr.gated_ffn_bwd(x, wg, wu, gate.half(), up.half(), dh)
    with pytest.raises(ValueError, match="dh must be"):
        gdr.gated_ffn_bwd(x, wg, wu, gate, up, dh.float())


@pytest.mark.parametrize("M,D,F", [(300, 33, 50), (300, 100, 333), (40, 513, 64), (1021, 12, 801)])
def test_gradients_with_one_rounding(gdr, M, D, F):
    """bf16 rows that are not whole 16-byte pieces: the products are fp32 ones, dG and dU enter them unrounded, and only
    the results are rounded, 1.65e-3 of them at random (some thousand values at least: within 0.25e-3 of that)."""
    say("gated ffn M %d D %d F %d" % (M, D, F))
    x, wg, wu, dh = make(M, D, F, BF16, 23)
    gx, gwg, gwu, gdh = (t.cuda() for t in (x, wg, wu, dh))
    h, gate, up = gdr.gated_ffn_fwd(gx, gwg, gwu, want_saved=True)
    got = gdr.gated_ffn_bwd(gx, gwg, gwu, gate, up, gdh)
    for name, p, q in zip(("dx", "dw_gate", "dw_up"), got, L.ffn_grads(x, wg, wu, dh)):
        check(p, q, 1.9e-3, name)
