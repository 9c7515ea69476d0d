"""Linear attention where the terms of a result cancel: what is formed on the way (states, scores, decayed values) has to
enter the matrix products with 24 bits, as fp32 has.

A result is held to the root of the sum of its terms' squares, not to itself. Of each term's factors the operands' three bf16
parts leave 2^-25, the exponential 2^-23 and a product 2^-24; the sums round some twelve times, each 2^-24 of no more than
that root, independently: 2^-22.2. Together 2^-21.9; 7e-7 leaves a factor of 2.8. Two parts, off by 2^-17 at most and 2^-18.3 in the
mean, are over 4 times past it. bf16 results are rounded once more, 2^-8 of the result itself, which is 2^-12 of the terms here."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import linear_attn as O
from tests._layers import BF16, FP32, U16, say

pytestmark = pytest.mark.gpu
OF_TERMS = 7e-7


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    return binding


def held(got, exact, terms, dtype, what):
    off = np.linalg.norm(got.double().cpu().numpy() - exact)
    size, of = np.linalg.norm(exact), np.linalg.norm(terms)
    assert size < 2 ** -9 * of  # (the terms do cancel)
    assert off <= (U16 if dtype == BF16 else 0.0) * size + OF_TERMS * of, "%s: %.2e of the terms" % (what, off / of)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dk,dv", [(64, 32), (64, 96), (128, 128), (128, 256)])
def test_states_read(gdr, dk, dv, dtype):
    """Queries with opposite neighbouring channels read states whose neighbouring rows are 2^-12 apart; the keys are zero."""
    say("states read dk %d dv %d %s" % (dk, dv, dtype))
    g = torch.Generator().manual_seed(700 + dk + dv)
    T, H = 70, 2
    q = torch.randn(1, H, T, dk // 2, generator=g).to(dtype)
    q = torch.stack([q, -q], -1).flatten(-2)
    h = torch.randn(1, H, dk // 2, dv, generator=g)
    h = torch.stack([h, h * (1 + 2 ** -12 * torch.rand(h.shape, generator=g))], 3).flatten(2, 3)
    k, v, la = torch.zeros_like(q), torch.randn(1, H, T, dv, generator=g).to(dtype), -1e-3 * torch.rand(1, H, T, generator=g)
    out, _ = gdr.linear_attn_fwd(*(t.cuda() for t in (q, k, v, la, h)))
    terms = np.sqrt(O.forward(q.double() ** 2, k, v, 2 * la, h.double() ** 2)[0])
    held(out, O.forward(q, k, v, la, h)[0], terms, dtype, "out")


def opposite(dtype, T, H, dk, dv, seed):
    """x, y, z, la: tokens 2i and 2i + 1 have the same y and opposite z, decays are about 2^-12 a token."""
    g = torch.Generator().manual_seed(seed)
    twice = lambda t: t.repeat_interleave(2, 2)
    x, y = (torch.randn(1, H, T, dk, generator=g).to(dtype), twice(torch.randn(1, H, T // 2, dk, generator=g)).to(dtype))
    z = twice(torch.randn(1, H, T // 2, dv, generator=g)).to(dtype)
    z[:, :, 1::2] *= -1
    return x, y, z, -2 ** -11 * torch.rand(1, H, T, generator=g)


def pairs(x, y, z, c):
    """sqrt(sum over j <= i and channels of (e^{c_i - c_j} x_i y_j z_j)^2)"""
    x, y, z, c = (t.double().numpy() for t in (x, y, z, c))
    w = np.tril(np.exp(2 * (c[..., :, None] - c[..., None, :])))
    return np.sqrt((w * np.matmul(x ** 2, np.swapaxes(y ** 2, -1, -2))) @ z ** 2)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dk,dv", [(64, 96), (128, 128), (128, 160)])
@pytest.mark.parametrize("T", [64, 250])
def test_opposite_tokens(gdr, T, dk, dv, dtype):
    """Within a chunk the scores carry what is left of two tokens, from chunk to chunk the states."""
    say("opposite tokens T %d dk %d dv %d %s" % (T, dk, dv, dtype))
    q, k, v, la = opposite(dtype, T, 2, dk, dv, 720 + dk + dv)
    out, _ = gdr.linear_attn_fwd(*(t.cuda() for t in (q, k, v, la)))
    exact, terms = O.forward(q, k, v, la)[0], pairs(q, k, v, la.double().cumsum(2))
    held(out[:, :, 1::2], exact[:, :, 1::2], terms[:, :, 1::2], dtype, "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dk,dv", [(64, 96), (128, 128), (128, 160)])
@pytest.mark.parametrize("T", [64, 250])
def test_opposite_gradients(gdr, T, dk, dv, dtype):
    """The same for the values' gradient, from the last token on, in a launch of its own and together with dq and dk."""
    say("opposite gradients T %d dk %d dv %d %s" % (T, dk, dv, dtype))
    k, q, dout, la = opposite(dtype, T, 2, dk, dv, 740 + dk + dv)
    got = gdr.linear_attn_bwd(*(t.cuda() for t in (q, k, torch.zeros_like(dout), la, dout)))[2]
    exact = O.grads(q, k, torch.zeros_like(dout), la, dout)[2]
    c = torch.cat([la, torch.zeros(1, 2, 1)], 2).flip(2).double().cumsum(2)[:, :, :T]  # up to the token before, from the last one on
    terms = pairs(*(t.flip(2) for t in (k, q, dout)), c)[:, :, ::-1]
    held(got[:, :, ::2], exact[:, :, ::2], terms[:, :, ::2], dtype, "dv")
