"""The experts' layer in each of its forms, held to that form's own bound (_experts_ref.py)."""
import math

import pytest
import torch

import _experts_ref as R
from test_experts_gpu import BF16, F16, hc, ids, layer, on_gpu, within  # noqa: F401

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------------------------------------- widths --

def padded(t, step):
    """t on the GPU, the axis next to its contiguous one in steps of `step`, NaN between."""
    turned = t.dim() == 3 and t.stride(2) != 1
    m = t.transpose(1, 2) if turned else t
    wide = torch.full((*m.shape[:-1], step), math.nan, dtype=t.dtype, device="cuda")
    wide[..., :m.shape[-1]] = m
    got = wide[..., :m.shape[-1]]
    return got.transpose(1, 2) if turned else got


@pytest.mark.parametrize("dtype", [BF16, F16], ids=ids)
@pytest.mark.parametrize("rows_out", [False, True], ids=["outputs", "inputs"])
@pytest.mark.parametrize("tokens", [3, 40, 300])
@pytest.mark.parametrize("hidden,inner", [(130, 70), (66, 2), (9, 129), (259, 33)])
def test_widths_that_eight_does_not_divide(hc, hidden, inner, tokens, rows_out, dtype):  # noqa: F811
    """Rows of any width in aligned steps reach the tensor cores, in tiles that are more than half full among others: the last
    inputs and features are nobody's, and what lies between rows is neither read nor written."""
    x, gate, up, down, e, w = args = layer(70, tokens, 3, 2, hidden, inner, dtype, rows_out)
    step = lambda n: -(-n // 8) * 8 + 8  # noqa: E731
    up_step, down_step = (step(hidden), step(inner)) if rows_out else (step(inner), step(hidden))
    out = torch.full((tokens, step(hidden)), 7.0, dtype=dtype, device="cuda")
    y = hc.expert_mlp(padded(x, step(hidden)), padded(gate, up_step), padded(up, up_step), padded(down, down_step), e.cuda(), w.cuda(),
                      out=out[:, :hidden])
    within(y, *R.experts(*args, stored=False))
    assert (out[:, hidden:] == 7.0).all()


# ------------------------------------------------------------------------------------------- a single expert --

def test_strides_of_a_single_expert_say_nothing(hc):  # noqa: F811
    """gate and up of one expert out of buffers whose experts lie at different steps."""
    for tokens in (3, 70):
        x, gate, up, down, e, w = layer(64, tokens, 1, 1, 64, 32, BF16)
        g = torch.zeros(2, 64, 32, dtype=BF16, device="cuda")[:1].copy_(gate)
        u = torch.zeros(2, 100, 32, dtype=BF16, device="cuda")[:1, :64].copy_(up)
        assert g.stride() != u.stride()
        y = hc.expert_mlp(x.cuda(), g, u, *on_gpu((down, e, w)))
        within(y, *R.experts(x, gate, up, down, e, w))
