"""The experts' layer and routing at the ends of their types' ranges. Bounds: _experts_ref.py, or derived here."""
import math

import pytest
import torch

import _experts_ref as R
from test_experts_gpu import BF16, F16, F32, hc, ids, layer, on_gpu, rnd, route_check, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ activation --

@pytest.mark.parametrize("dtype", [BF16, F32], ids=ids)
@pytest.mark.parametrize("general", [False, True], ids=["", "general"])
@pytest.mark.parametrize("tokens", [2, 200])
def test_activation_over_the_whole_range(hc, tokens, general, dtype):  # noqa: F811
    """silu(g) u where g u overflows, and where exp(-g) does. Every sum has one product, so that g, u and h down are as given.

    silu: the exponential's argument is off by 2 |g| v of the result (v = 2^-24: the constant and the product), exponential and
    quotient by 8 v, a product 1 v; h and the result are rounded to T (u each, a unit at 2^-126 of subnormal numbers: 2^-133 in bf16
    and 2^-149 in float32, of h by way of down)."""
    pairs = [(g, u) for g in (-5.0, -10.0, -30.0, -79.0, -80.5, -88.0, -89.0, -100.0, -120.0, -150.0, -170.0, 5.0, 80.0, 100.0, 300.0)
             for u in (3e38, -1e38, 4e37, 1e30, 1.0)]
    pairs += [(-1e20, 1e25), (-1e30, 3e38), (1e20, 1e10), (3e38, 0.5), (-0.0, 3e38), (0.0, -3e38), (-3e38, 1.0)]

    def value(g, u):
        return g * torch.exp(torch.minimum(g, torch.zeros_like(g))) / (1 + torch.exp(-g.abs())) * u

    # (what is beyond the type is infinite, and an infinity times one of down's zeros is no number)
    g, u = torch.tensor(pairs).to(dtype).t()
    fits = value(g.double(), u.double()).abs() < 3.3e38
    g, u = g[fits], u[fits]
    inner = -(-len(g) // 8) * 8
    g, u = (torch.nn.functional.pad(t, (0, inner - len(t))) for t in (g, u))
    x = torch.zeros(tokens, 128, dtype=dtype)
    x[:, 3] = 1.0
    gate, up = torch.zeros(1, 128, inner, dtype=dtype), torch.zeros(1, 128, inner, dtype=dtype)
    gate[0, 3], up[0, 3] = g, u
    scale = 2.0 ** -10
    down = torch.nn.functional.pad(torch.eye(inner, dtype=dtype), (0, 128 - inner))[None] * scale
    e, w = torch.zeros(tokens, 1, dtype=torch.int32), torch.ones(tokens, 1)
    y = hc.expert_mlp(*on_gpu((x, gate, up, down, e, w)), flags=hc.HC_FLAG_FORCE_GENERAL if general else 0)
    g, u = g.double(), u.double()
    h = value(g, u)
    unit = {BF16: 2.0 ** -133, F32: 2.0 ** -149}[dtype]
    of_t = 2 * R.U[dtype]
    tol = h.abs() * ((2 * g.abs().clamp(max=200) + 12) * R.V + of_t * 1.01) + 2 * unit
    got = y.double().cpu() / scale
    assert torch.isfinite(got).all()
    within(got[:, :inner], h.expand(tokens, -1), (tol + 2 * unit / scale).expand(tokens, -1))


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


# ------------------------------------------------------------------------------------- large inner values in fp16 --

FORMS = ["aligned", "general", "odd"]


def in_form(hc, args, form):  # noqa: F811
    """The layer's result through aligned rows, through the general kernels, and through rows at odd places."""
    x, gate, up, down, e, w = on_gpu(args)
    if form == "odd":
        wide = torch.zeros(x.shape[0], x.shape[1] + 3, dtype=x.dtype, device="cuda")
        wide[:, 1:-2] = x
        x = wide[:, 1:-2]
    return hc.expert_mlp(x, gate, up, down, e, w, flags=hc.HC_FLAG_FORCE_GENERAL if form == "general" else 0)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("tokens", [2, 60, 200, 500])
def test_inner_values_past_the_largest_float16(hc, tokens, form):  # noqa: F811
    """silu(256) * 2048 = 524288 is beyond float16, 64 of them by 2^-12 are 8192, which it holds; all sums are exact."""
    x, gate, up, down, e, w = layer(10, tokens, 2, 1, 64, 64, F16)
    x, gate, up, down = (torch.full_like(t, v) for t, v in ((x, 4.0), (gate, 1.0), (up, 8.0), (down, 2.0 ** -12)))
    assert (in_form(hc, (x, gate, up, down, e, w), form) == 8192.0).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows_out", [False, True], ids=["outputs", "inputs"])
@pytest.mark.parametrize("tokens,inner", [(3, 64), (40, 200), (200, 136), (300, 1160)])
def test_some_inner_values_past_the_largest_float16(hc, tokens, inner, rows_out, form):  # noqa: F811
    """A few of them, in some rows, of either sign, beside an infinite one that stays in its row and a row without experts."""
    x, gate, up, down, e, w = layer(61, tokens, 3, 2, 136, inner, F16, rows_out)
    x[::3] *= 100.0
    up *= 30.0
    down *= 2.0 ** -9
    e[tokens // 2] = -1
    y = in_form(hc, (x, gate, up, down, e, w), form)
    want, tol = R.experts(x, gate, up, down, e, w, stored=False)
    assert torch.isfinite(want).all() and want.abs().max() < 60000
    within(y, want, tol)
    x[0, 0] = math.inf
    z = in_form(hc, (x, gate, up, down, e, w), form)
    assert torch.equal(z[1:], y[1:]) and not torch.isfinite(z[0]).any()


@pytest.mark.parametrize("tokens", [30, 300])
def test_excess_of_a_captured_call(hc, tokens):  # noqa: F811
    """Values past float16 in some replays and not in others, in a workspace that held anything before; the same expert several
    times for a token, widths that eight does not divide, more than 1024 inner values."""
    hidden, inner, k = 131, 1050, 5
    x, gate, up, down, e, w = layer(65, tokens, 4, 4, 136, 1056, F16)
    e, w = torch.cat((e, e[:, :1]), 1), torch.cat((w, w[:, 1:2]), 1)
    down = down * 2.0 ** -9
    gpu = on_gpu((x, gate, up, down, e, w))
    cut = lambda x, g, u, d, e, w: (x[:, :hidden], g[:, :hidden, :inner], u[:, :hidden, :inner], d[:, :inner, :hidden], e, w)  # noqa: E731
    args = cut(*gpu)
    assert args[4].shape[1] == k
    work = torch.empty(hc.expert_mlp_workspace_size(*args), dtype=torch.uint8, device="cuda").random_(0, 256)
    hc.expert_mlp(*args, workspace=work)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = hc.expert_mlp(*args, workspace=work)
    for by in (300.0, 1.0, 200.0):
        scaled = x.clone()
        scaled[1::4] = scaled[1::4] * by
        gpu[0].copy_(scaled)
        graph.replay()
        cpu = cut(scaled, gate, up, down, e, w)
        want, tol = R.experts(*cpu, stored=False)
        past = max((v @ gate[0, :hidden, :inner].double() * (v @ up[0, :hidden, :inner].double())).abs().max() for v in [cpu[0].double()])
        assert (past > 65504) == (by > 1)
        within(y, want, tol)
        first = y.clone()
        graph.replay()
        assert torch.equal(first, y)


# -------------------------------------------------------------------------------------------------- routing --

@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,each", [(2, 2), (8, 4), (3, 7)])
@pytest.mark.parametrize("large", [30.0, 100.0, 1000.0, 1e5])
def test_biases_that_cancel(hc, large, groups, each, scoring):  # noqa: F811
    """A group's two best values are a large one and its negative but for little: their sum keeps only what float32 has at the
    large one's size, and the groups are closer than that. (float64 orders them as the real numbers do down to some 1e-16 of the
    large one, a hundredth of the smallest steps here.)"""
    g = torch.Generator().manual_seed(62)
    n, step = 300, large * 2.0 ** -26
    at = torch.randint(-30, 31, (n, groups, each), generator=g)
    # (the two that count are the first two; their places add up to another number in every group)
    at[:, :, 1] = torch.rand(n, 60, generator=g).argsort(1)[:, :groups] - 30 - at[:, :, 0]
    x = torch.rand(n, 1, 1, generator=g) * 0.5 + at * step
    bias = torch.full((groups, each), -4 * large)
    bias[:, 0], bias[:, 1] = large, -large
    for top in (1, groups - 1):
        route_check(hc, x.reshape(n, -1).contiguous(), 2, bias=bias.flatten(), scoring=scoring, groups=groups, top_groups=top,
                    group_best=2)
        closed = bias.clone()
        for value in (-1e9, -math.inf):  # a group that only goes along where no other is left, and does not blur the others
            closed[1] = value
            route_check(hc, x.reshape(n, -1).contiguous(), 2, bias=closed.flatten(), scoring=scoring, groups=groups, top_groups=top,
                        group_best=2)


def test_infinite_logits_leave_equal_scores(hc):  # noqa: F811
    """Beside a logit of plus infinity all others have the score 0 of a softmax: equal, so in the order of their index, whether a
    bias of zeros or none is given."""
    x = rnd(63, 6, 24)
    x[0, 0] = math.inf
    x[1, [3, 17]] = math.inf
    x[2, 5], x[2, 9], x[2, 2] = math.inf, -math.inf, math.nan
    x[3, 23], x[3, :6] = math.inf, -math.inf
    x[4, :] = math.inf
    for dtype in (F32, F16, BF16):
        r = x.to(dtype)
        for k in (1, 3, 24):
            for bias in (None, torch.zeros(24).cuda()):
                e, w = hc.expert_route(r.cuda(), k, bias=bias)
                for t in range(5):
                    high = (r[t] == math.inf).nonzero().flatten().tolist()
                    order = high + [i for i in range(24) if i not in high]
                    assert e[t].tolist() == order[:k], (dtype, k, t)
                    share = torch.tensor([1.0 / min(k, len(high)) if i in high else 0.0 for i in order[:k]])
                    assert torch.equal(w[t].cpu(), share)
        # groups of four: those with an infinite logit by their number of them, the others equal
        for best in (1, 2):
            for bias in (None, torch.zeros(24).cuda()):
                e, _ = hc.expert_route(r[1:2].cuda(), 12, bias=bias, groups=6, top_groups=3, group_best=best)
                assert e[0].tolist() == [3, 17] + [i for i in (*range(8), *range(16, 20)) if i not in (3, 17)]
