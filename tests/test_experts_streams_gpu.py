"""Routing, the experts' layer and the choice of tokens on other streams and devices than the current one."""
import pytest
import torch

import test_paged_edges_gpu as P
from test_experts_gpu import BF16, F32, hc, layer, on_gpu, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


def calls_with_streams(hc):  # noqa: F811
    """(what, call(stream=...)), each giving a tuple of tensors, of every kernel of the three operators."""
    tup = lambda x: x if isinstance(x, tuple) else (x,)  # noqa: E731
    few, many, f32 = (on_gpu(layer(80, n, 8, 2, 256, 128, t)) for n, t in ((20, BF16), (900, BF16), (60, F32)))
    scores, bias, x = rnd(81, 500, 64).cuda(), rnd(82, 64).cuda(), rnd(83, 40, 70000, scale=2.0).cuda()
    u = torch.rand(40, generator=torch.Generator().manual_seed(84)).cuda()
    return [("expert_route", lambda **kw: hc.expert_route(scores, 6, bias=bias, groups=8, top_groups=3, **kw))] + [
        ("expert_mlp " + what, lambda a=a, **kw: tup(hc.expert_mlp(*a, **kw))) for what, a in (("few", few), ("many", many), ("f32", f32))] + [
        (f"token_sample {k}", lambda k=k, **kw: hc.token_sample(x, u, return_logprob=True, **k, **kw))
        for k in (dict(), dict(top_k=50, min_p=0.01), dict(top_p=0.99))]


def test_memory_on_two_streams(hc, monkeypatch):  # noqa: F811
    monkeypatch.setattr(P, "calls_with_streams", calls_with_streams)
    P.test_other_streams_do_not_take_memory_that_is_still_in_use(hc)
    P.test_results_of_another_stream_are_not_handed_out_too_early(hc)


def test_inputs_without_another_reference(hc):  # noqa: F811
    """The caller's last references go with the call, which the other stream has yet to run, and their memory is asked for again."""
    x, gate, up, down, _, _ = on_gpu(layer(85, 300, 8, 2, 256, 128, BF16))
    scores, u = rnd(86, 300, 8).cuda(), torch.rand(300, generator=torch.Generator().manual_seed(87)).cuda()
    first = hc.expert_route(scores, 2)
    want = hc.expert_mlp(x, gate, up, down, *first)
    token = hc.token_sample(want, u, temperature=0.7, top_k=20)
    again = hc.expert_route(scores * 2, 3, bias=scores[0] * 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        # (made and complete before the other stream's turn, which a long kernel puts off)
        a, b, c = hc.expert_route(scores, 2), x.clone(), [scores * 2, scores[0] * 0.1]
        d, e = want.clone(), u.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        y = hc.expert_mlp(b, gate, up, down, *a, stream=side)
        t = hc.token_sample(d, e, temperature=0.7, top_k=20, stream=side)
        r = hc.expert_route(c[0], 3, bias=c[1], stream=side)
        sizes = [v.numel() * v.element_size() for v in (*a, b, *c, d, e)]
        del a, b, c, d, e
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(t, token)
        assert all(torch.equal(p, q) for p, q in zip(r, again))
        del junk


def test_tensors_of_another_device_than_the_current_one(hc, monkeypatch):  # noqa: F811
    """The call makes the tensors' device the current one (here, where there is but one, the current one is said to be another)."""
    from hyper_connection_rank_gb300 import _experts, _paged
    entered = []
    real = torch.cuda.device

    def device(index):
        entered.append(index)
        return real(index)
    for what, call in calls_with_streams(hc):
        want = [t.clone() for t in call()]
        with monkeypatch.context() as m:
            for module in (_experts, _paged):
                m.setattr(module, "_current_device", lambda: 3)
            m.setattr(torch.cuda, "device", device)
            got = call()
        assert entered and set(entered) == {0}, what
        entered.clear()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), what


def test_tensors_of_different_devices_are_refused(hc):  # noqa: F811
    scores, bias, live = rnd(88, 30, 8).cuda(), torch.zeros(8).cuda(), torch.tensor([30], dtype=torch.int32).cuda()
    args = on_gpu(layer(89, 30, 8, 2, 64, 32, BF16))
    work = torch.empty(hc.expert_mlp_workspace_size(*args), dtype=torch.uint8, device="cuda")
    x, rows = rnd(90, 30, 100).cuda(), [torch.full((30,), 0.5, device="cuda") for _ in range(4)]
    k = torch.full((30,), 5, dtype=torch.int32, device="cuda")
    calls = [
        (lambda a: hc.expert_route(a[0], 2, bias=a[1], live=a[2]), [scores, bias, live]),
        (lambda a: hc.expert_mlp(*a[:6], out=a[6], workspace=a[7]), [*args, torch.empty_like(args[0]), work]),
        (lambda a: hc.expert_mlp_workspace_size(*a), args),
        (lambda a: hc.token_sample(a[0], a[1], temperature=a[2], top_p=a[3], min_p=a[4], top_k=a[5]), [x, *rows, k]),
    ]
    for n, (call, tensors) in enumerate(calls):
        call(tensors)
        for i in range(len(tensors)):
            bad = [t.as_subclass(P.Elsewhere) if j == i else t for j, t in enumerate(tensors)]
            with pytest.raises(ValueError):
                call(bad)
                pytest.fail(f"call {n}: tensor {i} was taken")
