"""Steps of linear attention and gradients of the norms in launches of 2^32 threads and more, where workgroups go along y too: new states
and gradients against their formulas in 64 bits at the beginning, around the row's end and at the end. Tolerances as in the operators' own tests."""
from __future__ import annotations

import pytest
import torch

from tests._attn import TOL
from tests._layers import BF16, FP32, U16, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    torch.cuda.empty_cache()
    yield binding
    torch.cuda.empty_cache()


def near(x, ref, tol, what):
    assert torch.isfinite(x).all()
    e = ((x.double() - ref).norm() / ref.norm()).item()
    assert e <= tol, "%s: relative error %.3e > %.1e" % (what, e, tol)


@pytest.mark.parametrize("dtype,head", [(BF16, False), (FP32, True)])
def test_steps(gdr, dtype, head):
    """2^18 + 37 sequences of 8 heads of 256 value channels: 2^24 and more workgroups of 256 threads, 137 GB of states in place."""
    N, Hk, Hv, dk, dv = (1 << 18) + 37, 2, 8, 64, 256
    say("linear attention step N %d %s" % (N, dtype))
    g = torch.Generator(device="cuda").manual_seed(20)
    new = lambda *s: torch.empty(s, device="cuda").normal_(generator=g)
    q, k, v = (new(N, H, d).to(dtype) for H, d in ((Hk, dk), (Hk, dk), (Hv, dv)))
    la = -new(Hv).abs() if head else -new(N, Hv).abs()
    state = torch.empty(N, Hv, dk, dv, device="cuda")
    windows = [slice(0, 60), slice((1 << 17) - 30, (1 << 17) + 60), slice(N - 60, N)]
    before = [state[r].normal_(generator=g).clone() for r in windows]
    out, same = gdr.linear_attn_step(q, k, v, la, state, state)
    assert same is state
    heads = torch.arange(Hv, device="cuda") // (Hv // Hk)
    for r, h in zip(windows, before):
        a = (la if head else la[r]).double().exp().expand(h.shape[0], Hv)
        exact = a[..., None, None] * h.double() + k[r][:, heads].double()[..., None] * v[r].double()[..., None, :]
        near(state[r], exact, TOL[FP32], "state")
        near(out[r], (q[r][:, heads].double()[..., None, :] @ exact)[..., 0, :], TOL[FP32] + (U16 if dtype == BF16 else 0.0), "out")


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_of_many_tokens(gdr, interleaved):
    """2^28 + 21 tokens of one query and one key head of 8 channels: 2^24 and more workgroups forward, whose turns the backward's 1024
    take. The weights' gradients are held to 64-bit sums over all tokens of the gradients' own terms."""
    T = (1 << 28) + 21
    say("norms of %d tokens, gradients" % T)
    g = torch.Generator(device="cuda").manual_seed(21)
    q, k, doq, dok = (torch.empty(1, T, 1, 8, dtype=BF16, device="cuda").normal_(generator=g) for _ in range(4))
    doq, dok = doq.view(1, 1, T, 8), dok.view(1, 1, T, 8)
    w_q, w_k = (torch.rand(8, device="cuda", generator=g) + 0.5 for _ in range(2))
    f = torch.tensor([0.3, 1e-3, 1e-5, 1e-7], device="cuda")
    dq, dk, dw_q, dw_k = gdr.qk_norm_rope_bwd(q, k, w_q, w_k, f, doq, dok, interleaved=interleaved)

    def parts(x, dy, w, r):
        """the gradient of x and the terms of the weight's, of tokens r"""
        angle = torch.arange(r.start, r.stop, device="cuda")[:, None].double() * f.double()
        x, dy = x[0, r, 0].double(), dy[0, 0, r].double()
        a, b = (dy[:, ::2], dy[:, 1::2]) if interleaved else (dy[:, :4], dy[:, 4:])
        a, b = a * angle.cos() + b * angle.sin(), b * angle.cos() - a * angle.sin()
        turned = torch.stack([a, b], -1).flatten(1) if interleaved else torch.cat([a, b], -1)
        n = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        u = turned * w.double()
        return n * u - x * n ** 3 * (u * x).mean(-1, keepdim=True), turned * x * n

    for x, dy, w, dx, dw, name in ((q, doq, w_q, dq, dw_q, "dq"), (k, dok, w_k, dk, dw_k, "dk")):
        for r in (slice(0, 100), slice((1 << 28) - 50, (1 << 28) + 21), slice((1 << 27) - 50, (1 << 27) + 50)):
            near(dx[0, r, 0], parts(x, dy, w, r)[0], 2e-6 + U16, name)
        total = torch.zeros(8, dtype=torch.float64, device="cuda")
        for lo in range(0, T, 1 << 24):
            total += parts(x, dy, w, slice(lo, min(T, lo + (1 << 24))))[1].sum(0)
        near(dw, total, 2e-6, "dw of " + name)
