"""Inputs and comparisons shared by the tests of the layer operators."""
from __future__ import annotations

import math
import sys

import numpy as np
import torch

BF16, FP32 = torch.bfloat16, torch.float32
U16 = 2.0 ** -8  # half the spacing of bfloat16 (2^-7 in [1, 2)): the most one rounding moves a value


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def rel(x, ref):
    """Relative Frobenius error; every value has to be finite."""
    x = x.detach().cpu().double().numpy() if hasattr(x, "detach") else np.asarray(x, dtype=np.float64)
    assert x.shape == ref.shape, (x.shape, ref.shape)
    assert np.all(np.isfinite(x)), "non-finite values"
    if x.size == 0:
        return 0.0
    n = float(np.linalg.norm(ref))
    d = float(np.linalg.norm(x - ref))
    return d / n if n > 0 else (math.inf if d > 0 else 0.0)


def check(x, ref, tol, what):
    e = rel(x, ref)
    assert e <= tol, "%s: relative error %.3e > %.1e" % (what, e, tol)


def scan_case(lens, D, dtype, seed, packed=False, regime="layer", h0=True):
    """x, a, b, A_log, dt_bias, h0, cu. Regimes: "layer" (the library's layer initialisation), "slow"
    (decays of e^-0.001 a token and slower) and "wild" (gate inputs of +-60: decays that are 0 or 1
    to the last bit, input gates that are shut or open)."""
    g = torch.Generator().manual_seed(seed)
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    n = lambda *s: torch.randn(*s, generator=g)
    x, a, b = (n(B, T, D) for _ in range(3))
    A_log = torch.log(1.0 + 15.0 * torch.rand(D, generator=g))
    dt = torch.exp(torch.rand(D, generator=g) * math.log(100.0) + math.log(1e-3))
    dt_bias = torch.log(torch.expm1(dt))
    if regime == "slow":
        dt_bias = dt_bias - 8.0
    elif regime == "wild":
        a = 60.0 * torch.sign(a) * (a.abs() > 0.3)
        b = 60.0 * torch.sign(b) * (b.abs() > 0.3)
    cu = None
    if packed:
        cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    return (x.to(dtype), a.to(dtype), b.to(dtype), A_log, dt_bias, n(len(lens), D) if h0 else None, cu)


def cuda(ts):
    return [None if t is None else t.cuda() for t in ts]
