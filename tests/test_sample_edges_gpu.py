"""The choice of tokens where runs of logits are no numbers, against the plain float64 form of _experts_ref.py."""
import math

import pytest
import torch

from test_sample_gpu import BF16, F16, F32, check, hc, ids, rnd, uniforms  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=ids)
@pytest.mark.parametrize("rows", [30, 80])
def test_runs_of_nothing(hc, rows, dtype):  # noqa: F811
    """Runs of NaN and of minus infinity, each alone and mixed, longer than what a warp weighs at once, in the middle of a row and
    at its ends: they count as nothing. (Small calls keep whole rows, large ones read them by chunks.)"""
    vocab = 40009
    x = rnd(90, rows, vocab + 3, dtype=dtype, scale=2.0)[:, 1:vocab + 1]
    for r in range(rows):
        value = (math.nan, -math.inf)[r & 1]
        at, n = 37 * r, (512, 700, 1500, 5000, 39000)[r % 5]
        x[r, at:at + n] = value
        if r % 3 == 0:
            x[r, at + 5:at + n:7] = (-math.inf, math.nan)[r & 1]
        if r % 4 == 0:
            x[r, -600:] = math.nan
    clean = torch.where(torch.isnan(x), -math.inf, x.float()).to(dtype)
    for seed, kw in ((91, dict()), (92, dict(temperature=0.5)), (93, dict(top_p=0.9)), (94, dict(top_k=30))):
        u = uniforms(seed, rows)
        tokens = check(hc, x, u, **kw)
        assert torch.equal(tokens, hc.token_sample(clean.cuda(), u.cuda(), **kw))
        assert torch.isfinite(x[torch.arange(rows), tokens.cpu().long()]).all()
