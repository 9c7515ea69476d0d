"""Arguments that the layer operators' Python entry points refuse before any call, with the type of error and the
text that say which argument it was."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_70_amd import binding
    binding.lib()
    return binding


def test_what_is_no_tensor(gdr):
    x, w, t = torch.ones(4, 16, device="cuda"), torch.ones(8, 16, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (None, np.ones((8, 16), dtype=np.float32), [[1.0] * 16] * 8):
        with pytest.raises(TypeError, match="w_gate must be a torch.Tensor"):
            gdr.gated_ffn_fwd(x, bad, w)
        with pytest.raises(TypeError, match="w_up must be a torch.Tensor"):
            gdr.gated_ffn_fwd(x, w, bad)
        with pytest.raises(TypeError, match="weight must be a torch.Tensor"):
            gdr.linear_ce_fwd(x, bad, t)
        with pytest.raises(TypeError, match="targets must be a torch.Tensor"):
            gdr.linear_ce_fwd(x, w, bad)
    with pytest.raises(ValueError, match="w_gate must be a GPU tensor|w_gate is on"):
        gdr.gated_ffn_fwd(x, w.cpu(), w)
    w = torch.nn.Parameter(w)  # a subclass is taken
    assert gdr.gated_ffn_fwd(x, w, w)[0].shape == (4, 8) and gdr.linear_ce_fwd(x, w, t)[0].shape == (4,)


@pytest.mark.parametrize("shape", [(), (0,), (1,), (3, 1), (1, 3), (3, 4)])
def test_shapes_of_the_packed_boundaries(gdr, shape):
    x, p = torch.ones(1, 8, 16, device="cuda"), torch.zeros(16, device="cuda")
    cu = torch.zeros(shape, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="cu_seqlens must have shape"):
        gdr.channel_scan_fwd(x, x, x, p, p, None, cu)
    with pytest.raises(ValueError, match="cu_seqlens must have shape"):
        gdr.channel_scan_bwd(x, x, x, p, p, torch.zeros(64, device="cuda"), x, cu)
