"""examples/paged_experts.py: routing, the experts' layer and the choice of tokens between the block and the paged attention, as a
decoder uses them."""
import os
import sys

import pytest
import torch

import _experts_ref as R

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import paged_experts
    return paged_experts


def prompts(*lens):
    g = torch.Generator().manual_seed(5)
    return [torch.randint(0, 101, (n,), generator=g).cuda() for n in lens]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_every_call_follows_its_definition(ex, monkeypatch, dtype):
    """The calls that a chunk of prompts and the single tokens behind it make, each against the float64 form on what it was
    given there (of a padded batch, whose last rows are no token's)."""
    hc, calls = ex.hc, []

    def keep(name):
        f = getattr(hc, name)

        def call(*args, **kw):
            got = f(*args, **kw)
            calls.append((name, args, kw, got))
            return got
        monkeypatch.setattr(hc, name, call)

    for name in ("expert_route", "expert_mlp", "token_sample"):
        keep(name)
    model = ex.ExpertDecoder(dtype=dtype)
    p = prompts(40, 3, 17)
    cache = ex.Cache(len(model.qkv), 5 * 4, 16, model.kv_heads, model.dim, dtype, 5, 4)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache.grow(ints(40, 3, 17, 0, 0))
    logits = model(cache, torch.cat(p), ints(0, 40, 43, 60, 60, 60))
    filters = dict(temperature=0.9, top_k=30, top_p=0.9, min_p=0.01, return_logprob=True)
    token, _ = hc.token_sample(logits[[39, 42, 59]], torch.tensor([0.1, 0.5, 0.9]).cuda(), **filters)
    cache.grow(ints(1, 1, 1, 0, 0))
    token = torch.cat((token, ints(0, 0))).long()
    logits = model(cache, token, ints(0, 1, 2, 3, 3, 3), live=ints(3))
    hc.token_sample(logits, torch.rand(5, generator=torch.Generator().manual_seed(6)).cuda(), **filters)
    # (the calls on places that nobody has count as well: their results are defined)
    assert [c[0] for c in calls] == (["expert_route", "expert_mlp"] * 3 + ["token_sample"]) * 2
    cpu = lambda t: t.cpu() if isinstance(t, torch.Tensor) else t  # noqa: E731
    for name, args, kw, got in calls:
        args, kw = [cpu(a) for a in args], {k: cpu(v) for k, v in kw.items()}
        if name == "expert_route":
            live = None if kw["live"] is None else int(kw["live"])
            ids, w, tol = R.route(*args, **{**kw, "live": live})
            assert torch.equal(got[0].cpu(), ids)
            assert ((got[1].double().cpu() - w).abs() <= tol).all()
        elif name == "expert_mlp":
            y, tol = R.experts(*args)
            assert ((got.double().cpu() - y).abs() <= tol).all()
        else:
            kw.pop("return_logprob")
            want, logs, tol, sure = R.sample(*args, **kw)
            assert all(sure)
            assert got[0].tolist() == list(want)
            assert all(abs(a - b) <= t for a, b, t in zip(got[1].tolist(), logs, tol))


def test_generation_runs_and_repeats(ex):
    """Captured steps over padded places give the same tokens again, and greedy ones are the likeliest of their logits."""
    model = ex.ExpertDecoder()
    p = prompts(150, 7, 61)
    kw = dict(places=8, temperature=0.8, top_k=40, top_p=0.95)
    a, b = ex.generate(model, p, 9, **kw), ex.generate(model, p, 9, **kw)
    assert a[0].shape == (3, 9) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (a[0] >= 0).all() and (a[0] < 101).all() and (a[1] <= 0).all()
    c = ex.generate(model, p, 9, seed=1, **kw)
    assert not torch.equal(a[0], c[0])
    d, logs = ex.generate(model, p, 4, temperature=0.0)
    assert not logs.any() and torch.equal(d, ex.generate(model, p, 4, seed=7, top_k=1)[0])


def test_example_runs(ex, capsys):
    ex.main()
    assert len(capsys.readouterr().out.splitlines()) == 3
