"""The experts' layer in each of its forms, held to that form's own bound (_experts_ref.py): the general kernels keep inner values in
float32, the tensor cores' forms round them to the tensors' type, and all keep an expert's result in float32."""
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


# --------------------------------------------------------------------------------------- each form's own bound --

@pytest.mark.parametrize("dtype", [BF16, F16], ids=ids)
@pytest.mark.parametrize("rows_out", [False, True], ids=["outputs", "inputs"])
@pytest.mark.parametrize("tokens,experts,k,hidden,inner", [(1, 8, 3, 640, 192), (40, 3, 2, 264, 200), (131, 5, 2, 200, 448), (400, 6, 3, 512, 384)])
def test_each_form_has_its_own_bound(hc, tokens, experts, k, hidden, inner, rows_out, dtype):  # noqa: F811
    args = layer(71, tokens, experts, k, hidden, inner, dtype, rows_out)
    within(hc.expert_mlp(*on_gpu(args)), *R.experts(*args, stored=False), "tensor cores")
    exact, tol = R.experts(*args, rounded=False, stored=False)
    within(hc.expert_mlp(*on_gpu(args), flags=hc.HC_FLAG_FORCE_GENERAL), exact, tol, "general")
    x, *rest = on_gpu(args)
    odd = torch.zeros(tokens, hidden + 1, dtype=dtype, device="cuda")
    odd[:, 1:] = x
    within(hc.expert_mlp(odd[:, 1:], *rest), exact, tol, "odd rows")


# ---------------------------------------------------------------------------------------------- equal runs --

@pytest.mark.parametrize("rows_out", [False, True], ids=["outputs", "inputs"])
@pytest.mark.parametrize("tokens,experts,k,hidden,inner", [
    (61, 64, 6, 640, 384), (61, 64, 6, 1000, 264), (33, 200, 2, 264, 1160), (500, 900, 1, 136, 136), (300, 40, 3, 1096, 520),
    (151, 160, 1, 512, 320), (77, 154, 8, 320, 264)])
def test_more_small_tiles_than_multiprocessors(hc, tokens, experts, k, hidden, inner, rows_out):  # noqa: F811
    """Tiles of 32 pairs, laid end to end and cut into equal runs whose ends fall inside tiles of several blocks of inputs: sums of
    two pieces of the inner product, two planes of the outer one."""
    args = layer(72, tokens, experts, k, hidden, inner, BF16, rows_out, skew=0.5)
    assert tokens * k <= 24 * experts
    pairs = sum(-(-n // 32) for n in torch.bincount(args[4].flatten().long(), minlength=experts).tolist())
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert pairs * -(-inner // 128) > sms and hidden > 64
    y = hc.expert_mlp(*on_gpu(args))
    within(y, *R.experts(*args, stored=False))
    for _ in range(3):
        assert torch.equal(hc.expert_mlp(*on_gpu(args)), y)
    assert hc.debug_wait_timeouts() == 0


def test_runs_of_a_batch_that_changes(hc):  # noqa: F811
    """The cuts move with the experts' counts: the same captured call on other choices, and with fewer and fewer rows in use."""
    x, gate, up, down, e, w = args = on_gpu(layer(73, 61, 64, 6, 640, 384, BF16))
    g = torch.cuda.CUDAGraph()
    hc.expert_mlp(*args)
    with torch.cuda.graph(g):
        y = hc.expert_mlp(*args)
    for seed, live in ((74, 61), (75, 40), (76, 21), (77, 3), (78, 60)):
        more = layer(seed, 61, 64, 6, 8, 8, BF16)
        e.copy_(more[4])
        e[live:] = -1
        w.copy_(more[5])
        g.replay()
        within(y, *R.experts(*(t.cpu() for t in args), stored=False))


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
