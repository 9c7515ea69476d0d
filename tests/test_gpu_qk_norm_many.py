"""Norms of queries and keys over tens of thousands of tokens (those calls take another kernel, and their weights' sums are
longer) against their formulas in 64 bits on the GPU. Tolerances as in tests/test_gpu_qk_norm.py."""
from __future__ import annotations

import pytest
import torch

from tests._layers import BF16, FP32, U16, say
from tests._qk_cases import LONG, MANY

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    yield binding
    torch.cuda.empty_cache()


def turned(x, angle, interleaved):
    """x [B, T, H, d], its first pairs turned by angle [B, T, rot / 2]"""
    r = angle.shape[-1]
    at = torch.arange(r, device=x.device)
    a, b = (2 * at, 2 * at + 1) if interleaved else (at, r + at)
    c, s = angle.cos()[:, :, None], angle.sin()[:, :, None]
    y = x.clone()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def exact(x, w, angle, dy, interleaved):
    """y [B, H, T, d], dx [B, T, H, d], dw [d] in 64 bits"""
    x, w, g = x.double(), w.double(), turned(dy.double().transpose(1, 2), -angle, interleaved)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = turned(x * r * w, angle, interleaved).transpose(1, 2)
    dw = (g * x * r).sum((0, 1, 2))
    u = g * w
    return y, r * u - x * r ** 3 * (u * x).mean(-1, keepdim=True), dw


def near(x, ref, tol, what):
    assert torch.isfinite(x).all()
    e = ((x.double() - ref).norm() / ref.norm()).item()
    assert e <= tol, "%s: relative error %.3e > %.1e" % (what, e, tol)


def compare(gdr, B, T, Hq, Hk, d, rot, dtype, interleaved):
    say("many norms B %d T %d Hq %d Hk %d d %d rot %d %s interleaved %s" % (B, T, Hq, Hk, d, rot, dtype, interleaved))
    g = torch.Generator(device="cuda").manual_seed(1000 + T + d)
    n = lambda *s: torch.empty(s, device="cuda").normal_(generator=g)
    rows = (n(B, T, (Hq + Hk) * d + 8) * n(B, T, 1).exp()).to(dtype)
    q, k = rows[..., :Hq * d].unflatten(-1, (Hq, d)), rows[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    w_q, w_k = 1.0 + 0.3 * n(d), 1.0 + 0.3 * n(d)
    f = torch.exp(-9.0 * torch.rand(rot // 2, device="cuda", generator=g)) if rot else None
    pos = torch.randint(-5, 100000, (B, T), device="cuda", generator=g)
    doq, dok = n(B, Hq, T, d).to(dtype), n(B, Hk, T, d).to(dtype)
    angle = pos.double()[..., None] * (f.double() if rot else torch.zeros(0, device="cuda", dtype=torch.float64))
    oq, ok = gdr.qk_norm_rope_fwd(q, k, w_q, w_k, f, pos, eps=EPS, interleaved=interleaved)
    dq, dk, dw_q, dw_k = gdr.qk_norm_rope_bwd(q, k, w_q, w_k, f, doq, dok, pos, eps=EPS, interleaved=interleaved)
    r = U16 if dtype == BF16 else 0.0
    for name, x, w, y, dy, dx, dw in (("q", q, w_q, oq, doq, dq, dw_q), ("k", k, w_k, ok, dok, dk, dw_k)):
        ry, rx, rw = exact(x, w, angle, dy, interleaved)
        near(y, ry, 1e-6 + r, "o" + name)
        near(dx, rx, 2e-6 + r, "d" + name)
        near(dw, rw, 2e-6, "dw_" + name)
    # without positions: each batch row from 0 on, with the same bits as positions that say so
    at = torch.arange(T, device="cuda").expand(B, T).contiguous()
    for a, b in zip(gdr.qk_norm_rope_fwd(q, k, w_q, None, f, eps=EPS, interleaved=interleaved), gdr.qk_norm_rope_fwd(q, k, w_q, None, f, at, eps=EPS, interleaved=interleaved)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", MANY)
def test_many_tokens(gdr, B, T, Hq, Hk, d, rot, interleaved, dtype):
    compare(gdr, B, T, Hq, Hk, d, rot, dtype, interleaved)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", LONG)
def test_long_sums(gdr, B, T, Hq, Hk, d, rot, dtype):
    compare(gdr, B, T, Hq, Hk, d, rot, dtype, False)
