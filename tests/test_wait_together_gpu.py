"""Warps that go on together after bounded waits of their own: one that gives up takes the others with it, and none is left at the
barrier where they would have met (failure detection without a GPU fault: nothing is in flight when the waits run out)."""
import pytest
import torch

from test_experts_gpu import BF16, hc, layer, on_gpu, within  # noqa: F401
import _experts_ref as R

pytestmark = pytest.mark.gpu


def test_one_warp_s_wait_ends_all(hc):  # noqa: F811
    hc.debug_wait_timeouts(reset=True)
    try:
        assert (hc.debug_wait_together(0) == 1.0).all() and hc.debug_wait_timeouts() == 0
        for stuck in (1, 2, 4, 8, 6, 15):
            out = hc.debug_wait_together(stuck, limit_cycles=200_000)
            torch.cuda.synchronize()
            assert torch.isnan(out).all()
            assert hc.debug_wait_timeouts(reset=True) == 32 * bin(stuck).count("1")
        # the context is still healthy
        args = layer(100, 61, 64, 6, 256, 128, BF16)
        within(hc.expert_mlp(*on_gpu(args)), *R.experts(*args, stored=False))
        assert hc.debug_wait_timeouts() == 0
    finally:
        hc.debug_wait_timeouts(reset=True)


def test_limits_are_checked_on_the_host(hc):  # noqa: F811
    out = torch.zeros(128, device="cuda")
    f, bad = hc._binding.lib().hc_debug_wait_together, hc._binding.HC_ERR_INVALID_ARG
    assert f(out.data_ptr(), 1, 10, None) == bad and f(out.data_ptr(), 16, 2_000_000, None) == bad
    assert f(None, 1, 2_000_000, None) == bad
