"""examples/paged_beam.py: the operators together, as a decoder uses them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import paged_beam
    return paged_beam


def prompt(n):
    return torch.randint(0, 101, (n,), generator=torch.Generator().manual_seed(n)).cuda()


@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("compact_at", [None, 4])
def test_beams_match_a_run_from_the_start(ex, window, compact_at):
    """The logits of the last step, formed token by token over forked and moved pages, are those of the whole sequences read at
    once into fresh pages (float32: 1e-3 of the logits' size, for a few hundred roundings of 6e-8 through three layers; a wrong
    page or position moves them by their own size)."""
    model = ex.Decoder(dtype=torch.float32, window=window)
    p = prompt(61)
    path, scores, logits = ex.beam_search(model, p, beams=5, steps=9, page=4, compact_at=compact_at)
    assert path.shape == (5, 9) and bool((scores[:-1] >= scores[1:]).all())
    # every beam of the last step but its last token, as one batch of chunks
    fed = path[:, :-1]
    n = p.numel() + fed.shape[1]
    cache = ex.Cache(len(model.qkv), 5 * (n // 4 + 2), 4, model.kv_heads, model.dim, torch.float32, 5, n // 4 + 1)
    assert int(cache.grow(torch.full((5,), n, dtype=torch.int32, device="cuda"))) == 0
    whole = torch.cat((p.expand(5, -1), fed), 1)
    cu = torch.arange(0, 5 * n + 1, n, dtype=torch.int32, device="cuda")
    all_logits = model(cache, whole.flatten(), cu).view(5, n, -1)
    # which of them the last step's five parents were follows from their logits
    last = all_logits[:, -1]
    for row in last:
        assert float((logits - row).abs().amax(1).min()) <= 1e-3 * float(row.abs().max())


def test_half_precision_runs_and_repeats(ex):
    model = ex.Decoder()
    p = prompt(150)
    a = ex.beam_search(model, p, compact_at=3)
    b = ex.beam_search(model, p)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert bool(torch.isfinite(a[1]).all())


def test_a_step_in_a_graph(ex):
    """One decode step captured and replayed: lengths and tables are read on the device."""
    model = ex.Decoder()
    cache = ex.Cache(len(model.qkv), 40, 16, model.kv_heads, model.dim, model.dtype, 3, 8)
    n = torch.tensor([20, 5, 33], dtype=torch.int32, device="cuda")
    cache.grow(n)
    cu = torch.tensor([0, 20, 25, 58], dtype=torch.int32, device="cuda")
    model(cache, prompt(58), cu)
    cache.grow(torch.ones(3, dtype=torch.int32, device="cuda"))
    token = torch.tensor([1, 2, 3], device="cuda")
    want = model(cache, token)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model(cache, token)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = model(cache, token)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
