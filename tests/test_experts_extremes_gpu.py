"""The experts' layer and routing at the ends of their types' ranges. Bounds: _experts_ref.py, or derived here."""
import pytest
import torch

import _experts_ref as R
from test_experts_gpu import BF16, F16, hc, ids, layer, on_gpu, within  # noqa: F401

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------------------------------- unequal features --

@pytest.mark.parametrize("dtype", [BF16, F16], ids=ids)
@pytest.mark.parametrize("factor", [100.0, 1000.0, 10000.0])
@pytest.mark.parametrize("tokens", [30, 200])
def test_small_features_beside_large_ones(hc, tokens, factor, dtype):  # noqa: F811
    """One feature of sixteen is `factor` times as large as the others: those keep their digits, whatever the number of tokens."""
    x, gate, up, down, e, w = layer(60, tokens, 4, 2, 128, 64, dtype)
    down = down / 16
    down[:, :, 5::16] = (down[:, :, 5::16].float() * factor).to(dtype)
    y = hc.expert_mlp(*on_gpu((x, gate, up, down, e, w)))
    want, tol = R.experts(x, gate, up, down, e, w, stored=False)
    within(y, want, tol)
