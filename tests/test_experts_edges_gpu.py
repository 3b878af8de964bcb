"""Calls of the experts' layer, routing and the choice of tokens that the documentation allows but that ordinary use seldom makes,
and the refusals that need a GPU."""
import math
import os
import subprocess
import sys

import pytest
import torch

import _experts_ref as R
from test_experts_gpu import BF16, F16, F32, hc, ids, layer, on_gpu, rnd, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32], ids=ids)
@pytest.mark.parametrize("tokens,experts,k,hidden,inner", [(3, 1024, 32, 72, 16), (1100, 1024, 32, 16, 24), (40, 471, 3, 64, 72)])
def test_most_experts(hc, tokens, experts, k, hidden, inner, dtype):  # noqa: F811
    """As many experts and choices as there can be; so many that the small tiles' CTAs no longer share an SM."""
    args = layer(40, tokens, experts, k, hidden, inner, dtype)
    y = hc.expert_mlp(*on_gpu(args))
    want, tol = R.experts(*args)
    within(y, want, tol)


@pytest.mark.parametrize("tokens", [1, 2, 300])
def test_widest_rows(hc, tokens):  # noqa: F811
    for hidden, inner in ((65536, 8), (8, 65536)):
        args = layer(41, tokens, 1, 1, hidden, inner, BF16)
        want, tol = R.experts(*args)
        within(hc.expert_mlp(*on_gpu(args)), want, tol)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=ids)
@pytest.mark.parametrize("inner", [1, 8])
def test_one_input(hc, dtype, inner):  # noqa: F811
    """Axes of one element, whose strides say nothing."""
    x, gate, up, down, e, w = layer(42, 20, 3, 2, 8, inner, dtype)
    want, tol = R.experts(x, gate, up, down, e, w)
    for g, d in ((gate, down), (gate.transpose(1, 2).contiguous().transpose(1, 2), down.transpose(1, 2).contiguous().transpose(1, 2))):
        u = torch.empty_strided(up.shape, g.stride(), dtype=dtype).copy_(up)
        within(hc.expert_mlp(*on_gpu((x, g, u, d, e, w))), want, tol)
    x1, g1, u1 = x[:, :1], gate[:, :1], up[:, :1]
    d1 = down[:, :, :1]
    want, tol = R.experts(x1, g1, u1, d1, e, w)
    within(hc.expert_mlp(*[t.cuda() for t in (x1, g1, u1, d1, e, w)]), want, tol)


@pytest.mark.parametrize("tokens", [1, 30, 400])
def test_rows_of_any_step(hc, tokens):  # noqa: F811
    """One row of x many times (a step of 0), single rows of a matrix with odd ones, rows of out at odd places."""
    x, gate, up, down, e, w = layer(43, tokens, 4, 2, 64, 72, BF16)
    one = x[:1].expand(tokens, -1)
    want, tol = R.experts(one, gate, up, down, e, w)
    g = on_gpu((gate, up, down, e, w))
    out = torch.full((tokens, 67), 3.0, dtype=BF16, device="cuda")
    within(hc.expert_mlp(x[:1].cuda().expand(tokens, -1), *g, out=out[:, 1:65]), want, tol)
    assert (out[:, 0] == 3.0).all() and (out[:, 65:] == 3.0).all()
    odd = torch.zeros(5, 65, dtype=BF16, device="cuda")
    odd[:1, :64] = x[:1].cuda()
    y = hc.expert_mlp(odd[:1, :64], *g[:3], g[3][:1], g[4][:1])
    assert torch.equal(y, hc.expert_mlp(x[:1].cuda(), *g[:3], g[3][:1], g[4][:1]))


def test_calls_at_once(hc):  # noqa: F811
    """Two streams, each with its own workspace, both forms side by side; weights made by a kernel just before the call."""
    small, large = on_gpu(layer(44, 20, 8, 2, 512, 256, BF16)), on_gpu(layer(45, 900, 8, 2, 512, 256, BF16))
    want = [hc.expert_mlp(*a) for a in (small, large)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, (s, a) in enumerate(zip(sides, (small, large))):
            got[i].append(hc.expert_mlp(*a, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
    for a, w in ((small, want[0]), (large, want[1])):
        x, gate, up, down, e, k = a
        for _ in range(5):
            y = hc.expert_mlp(x, gate.clone(), up.clone(), down.clone(), e.clone(), k.clone())
            assert torch.equal(y, w)
    assert hc.debug_wait_timeouts() == 0


def test_calls_one_after_another(hc):  # noqa: F811
    """Calls of different forms in one workspace, back to back, each on the last one's results."""
    small, large = on_gpu(layer(46, 20, 8, 2, 256, 128, BF16)), on_gpu(layer(47, 900, 8, 2, 256, 128, BF16))
    work = torch.empty(max(hc.expert_mlp_workspace_size(*a) for a in (small, large)), dtype=torch.uint8, device="cuda")

    def chain(sync):
        x, z, got = small[0], large[0], []
        for _ in range(4):
            x = hc.expert_mlp(x, *small[1:], workspace=work)
            z = hc.expert_mlp(z, *large[1:], workspace=work)
            z[:20] += x
            got += [x, z.clone()]
            if sync:
                torch.cuda.synchronize()
        return got
    for a, b in zip(chain(True), chain(False)):
        assert torch.equal(a, b)


def test_a_padded_batch(hc):  # noqa: F811
    """Rows behind the last token's: no experts, no weights, zeros from the layer, whatever lies there."""
    x, gate, up, down, _, _ = on_gpu(layer(48, 64, 8, 2, 128, 64, BF16))
    logits = rnd(49, 64, 8, dtype=BF16).cuda()
    x[37:], logits[40:] = math.nan, math.nan
    live = torch.tensor([37], dtype=torch.int32, device="cuda")
    e, w = hc.expert_route(logits, 2, live=live)
    y = hc.expert_mlp(x, gate, up, down, e, w)
    assert (e[37:] == -1).all() and not w[37:].any() and not y[37:].any()
    want, tol = R.experts(*(t.cpu() for t in (x[:37], gate, up, down, e[:37], w[:37])))
    within(y[:37], want, tol)


def test_large_steps(hc):  # noqa: F811
    """Offsets that pass 32 bits: rows of x, of logits and of weights some gigabytes apart."""
    step = (1 << 31) + 64
    big = torch.empty(step + 4096, dtype=BF16, device="cuda")
    x, gate, up, down, e, w = layer(50, 2, 2, 1, 64, 16, BF16)
    e[0], e[1] = 0, 1
    rows = big.as_strided((2, 64), (step, 1)).copy_(x)
    want, tol = R.experts(x, gate, up, down, e, w)
    within(hc.expert_mlp(rows, *on_gpu((gate, up, down, e, w))), want, tol)
    experts = big.as_strided((2, 64, 16), (step, 16, 1)).copy_(gate)
    for flags in (0, hc.HC_FLAG_FORCE_GENERAL):
        within(hc.expert_mlp(x.cuda(), experts, torch.as_strided(big, (2, 64, 16), (step, 16, 1)), *on_gpu((down, e, w)), flags=flags),
               *R.experts(x, gate, gate, down, e, w))
    logits = rnd(51, 2, 300, dtype=BF16)
    far = big.as_strided((2, 300), (step, 1)).copy_(logits)
    assert torch.equal(hc.expert_route(far, 5)[0], hc.expert_route(logits.cuda(), 5)[0])
    u = torch.tensor([0.3, 0.8]).cuda()
    for kw in (dict(), dict(top_k=7), dict(top_p=0.9)):
        assert torch.equal(hc.token_sample(far, u, **kw), hc.token_sample(logits.cuda(), u, **kw))


def test_sampling_at_once(hc):  # noqa: F811
    """Every kind of call on two streams side by side."""
    x, u = rnd(52, 60, 30000, scale=2.0).cuda(), torch.rand(60, generator=torch.Generator().manual_seed(53)).cuda()
    kinds = [dict(), dict(top_k=50), dict(top_p=0.9), dict(top_k=3000), dict(temperature=torch.linspace(0, 2, 60).cuda())]
    want = [hc.token_sample(x, u, **k) for k in kinds]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [[hc.token_sample(x, u, stream=s, **k) for s in sides] for _ in range(3) for k in kinds]
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        assert all(torch.equal(y, want[i % len(kinds)]) for y in pair)


FIRST_CALLS = """
import torch, hyper_connection_rank_gb300 as hc
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
logits, x, weights = rand(3, 70000), rand(40, 64).half(), [rand(8, *s).half() for s in ((64, 32), (64, 32), (32, 64))]
many, u, scores = rand(900, 64).half(), torch.rand(3, generator=g, device="cuda"), rand(40, 8)
ids = torch.randint(0, 8, (900, 2), generator=g, device="cuda", dtype=torch.int32)
share = torch.rand(900, 2, generator=g, device="cuda")
def run():
    e, w = hc.expert_route(scores, 2)
    return [hc.token_sample(logits, u), hc.token_sample(logits, u, top_p=0.9), hc.token_sample(logits, u, top_k=9), e, w,
            hc.expert_mlp(x, *weights, e, w), hc.expert_mlp(many, *weights, ids, share),
            hc.expert_mlp(x.float(), *[t.float() for t in weights], e, w)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
print("the same")
"""


def test_first_calls_in_a_capture(hc):  # noqa: F811
    """A process whose first call of each kind is captured: what is asked of the device once must not disturb the capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "the same" in got.stdout, got.stderr[-2000:]


# ---------------------------------------------------------------------------------------------- refusals --

def test_mlp_refusals(hc):  # noqa: F811
    x, gate, up, down, e, w = on_gpu(layer(54, 6, 4, 2, 64, 32, BF16))
    size = hc.expert_mlp_workspace_size(x, gate, up, down, e, w)
    work = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    call = lambda *a, **kw: hc.expert_mlp(*a, **kw)  # noqa: E731
    bad = [
        lambda: call(x.cpu(), gate, up, down, e, w), lambda: call(x, gate.cpu(), up, down, e, w),
        lambda: call(x.double(), gate, up, down, e, w), lambda: call(x, gate.half(), up, down, e, w),
        lambda: call(x, gate, up[:3], down, e, w), lambda: call(x, gate, up.transpose(1, 2).contiguous().transpose(1, 2), down, e, w),
        lambda: call(x, gate, up, down.transpose(1, 2), e, w), lambda: call(x[:, :32], gate, up, down, e, w),
        lambda: call(x, gate, up, down, e.long(), w), lambda: call(x, gate, up, down, e, w.half()),
        lambda: call(x, gate, up, down, e[:, :1], w), lambda: call(x, gate, up, down, e.t().contiguous().t(), w),
        lambda: call(x, gate, up, down, e[:, :0], w[:, :0]), lambda: call(x, gate[::1, ::2, ::2], up[::1, ::2, ::2], down, e, w),
        lambda: call(x.t().contiguous().t(), gate, up, down, e, w), lambda: call(x, gate, up, down, e, w, out=x),
        lambda: call(x, gate, up, down, e, w, out=x[:5]), lambda: call(x, gate, up, down, e, w, out=x.float()),
        lambda: call(x, gate, up, down, e, w, out=torch.empty(64, 6, dtype=BF16, device="cuda").t()),
        lambda: call(x, gate, up, down, e, w, out=gate.view(-1, 64)[:6]),
        lambda: call(x, gate, up, down, e, w, out=torch.empty(1, 64, dtype=BF16, device="cuda").expand(6, -1)),
        lambda: call(x, gate, up, down, e, w, workspace=work[:size - 1]), lambda: call(x, gate, up, down, e, w, workspace=work[8:]),
        lambda: call(x, gate, up, down, e, w, workspace=torch.empty(size, dtype=torch.uint8)),
        lambda: call(x, gate, up, down, e, w, flags=8)]
    for f in bad:
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            f()
    assert call(x, gate, up, down, e, w, workspace=work).shape == x.shape


def test_route_and_sample_refusals(hc):  # noqa: F811
    x, u = rnd(55, 4, 64).cuda(), torch.rand(4).cuda()
    bad = [
        lambda: hc.expert_route(x.double(), 2), lambda: hc.expert_route(x[0], 2), lambda: hc.expert_route(x.t(), 2),
        lambda: hc.expert_route(x, 0), lambda: hc.expert_route(x, 65), lambda: hc.expert_route(x, 33),
        lambda: hc.expert_route(x, 2, scoring="max"), lambda: hc.expert_route(x, 2, groups=5), lambda: hc.expert_route(x, 9, groups=8, top_groups=1),
        lambda: hc.expert_route(x, 2, groups=8, top_groups=2, group_best=3), lambda: hc.expert_route(x, 2, bias=x[0, :63].contiguous()),
        lambda: hc.expert_route(x, 2, bias=x[0].half()), lambda: hc.expert_route(x, 2, live=torch.tensor([2], device="cuda")),
        lambda: hc.expert_route(x, 2, scale=math.nan), lambda: hc.token_sample(x, u[:3]), lambda: hc.token_sample(x, u.double()),
        lambda: hc.token_sample(x.long(), u), lambda: hc.token_sample(x, u.cpu()), lambda: hc.token_sample(x.t(), u),
        lambda: hc.token_sample(x, u, top_k=torch.full((4,), 3, device="cuda")), lambda: hc.token_sample(x, u, top_p=u[:2]),
        lambda: hc.token_sample(x, u, temperature=u.double()), lambda: hc.token_sample(x[:, :0], u)]
    for f in bad:
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            f()
