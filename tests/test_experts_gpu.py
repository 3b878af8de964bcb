"""Routing to experts and the experts' layer on the GPU against the plain float64 forms and bounds of _experts_ref.py."""
import math

import pytest
import torch

import _experts_ref as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None  # noqa: E731


@pytest.fixture(scope="module")
def hc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import hyper_connection_rank_gb300 as hc
    return hc


def rnd(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def within(got, want, tol, what=""):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN elsewhere"
    over = (got - want).abs() - tol
    assert over.numel() == 0 or over.max() <= 0, f"{what}: {over.max():.3e} over the bound"


# ---------------------------------------------------------------------------------------------- experts --

def layer(seed, tokens, experts, k, hidden, inner, dtype, rows_out=False, spare=0, skew=1.0):
    """(x, gate, up, down, ids, weights) on the CPU; spare: elements between rows of x."""
    x = rnd(seed, tokens, hidden + spare, dtype=dtype)[:, :hidden]

    def weight(s, rows, cols):
        if rows_out:
            return rnd(s, experts, cols, rows, dtype=dtype, scale=rows ** -0.5).transpose(1, 2)
        return rnd(s, experts, rows, cols, dtype=dtype, scale=rows ** -0.5)

    score = rnd(seed + 4, tokens, experts) + skew * rnd(seed + 5, experts)
    w, e = score.topk(k)
    return x, weight(seed + 1, hidden, inner), weight(seed + 2, hidden, inner), weight(seed + 3, inner, hidden), e.int(), \
        torch.softmax(w, -1)


def on_gpu(args):
    """The same tensors on the GPU, with the same strides."""
    got = []
    for t in args:
        g = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
        got.append(g.copy_(t))
    return got


def check(hc, args, flags=0, what="", **kw):
    y = hc.expert_mlp(*on_gpu(args), flags=flags, **kw)
    want, tol = R.experts(*args)
    within(y, want, tol, what)
    return y


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=ids)
@pytest.mark.parametrize("rows_out", [False, True], ids=["outputs", "inputs"])
@pytest.mark.parametrize("tokens,experts,k,hidden,inner", [
    (1, 1, 1, 64, 64), (1, 8, 3, 128, 64), (1, 16, 8, 640, 192), (2, 3, 3, 72, 136), (5, 40, 2, 320, 200), (7, 4, 1, 1000, 88),
    (33, 4, 2, 264, 72), (61, 64, 6, 256, 128), (100, 5, 2, 136, 264), (131, 3, 1, 128, 448), (257, 2, 2, 200, 64),
    (300, 6, 3, 512, 384), (520, 4, 1, 64, 520), (900, 3, 2, 136, 712)])
def test_mlp_sizes(hc, tokens, experts, k, hidden, inner, rows_out, dtype):
    """Every form (tiles of 32 and of 256 pairs; float32), tiles that are not full, widths that no tile divides."""
    check(hc, layer(1, tokens, experts, k, hidden, inner, dtype, rows_out), what="mlp")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=ids)
@pytest.mark.parametrize("tokens,experts,k,hidden,inner", [(1, 1, 1, 1, 1), (3, 2, 1, 7, 5), (40, 3, 2, 65, 33), (70, 2, 2, 63, 129)])
def test_mlp_odd_widths(hc, tokens, experts, k, hidden, inner, dtype):
    """Rows that are not 16-byte aligned take the general kernels, in either layout."""
    for rows_out in (False, True):
        check(hc, layer(2, tokens, experts, k, hidden, inner, dtype, rows_out), what="odd")


@pytest.mark.parametrize("tokens", [1, 20, 60, 200, 500])
def test_mlp_general_agrees(hc, tokens):
    args = layer(3, tokens, 4, 2, 192, 128, F16)
    check(hc, args, flags=hc.HC_FLAG_FORCE_GENERAL, what="general")
    check(hc, args, what="tensor cores")


@pytest.mark.parametrize("tokens", [3, 90, 150, 700])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=ids)
def test_mlp_rows_without_experts(hc, tokens, dtype):
    """Entries outside the experts take no part, whatever their weights; a row without any other is zero."""
    x, gate, up, down, e, w = layer(4, tokens, 6, 3, 128, 64, dtype)
    e[::3] = -1
    w[::3] = math.nan
    e[1, 1], w[1, 1] = 6, math.inf
    e[2, 0], w[2, 0] = -2 ** 31, -math.inf
    y = hc.expert_mlp(*on_gpu((x, gate, up, down, e, w)))
    clean = torch.where((e >= 0) & (e < 6), w, 0.0)
    want, tol = R.experts(x, gate, up, down, e, clean)
    within(y, want, tol)
    assert not y[::3].any()


def test_mlp_nobody(hc):
    x, gate, up, down, e, w = on_gpu(layer(5, 40, 4, 2, 128, 64, BF16))
    e.fill_(-1)
    y = torch.full_like(x, math.nan)
    assert hc.expert_mlp(x, gate, up, down, e, w, out=y) is y
    assert not y.any()
    assert hc.expert_mlp(x[:0], gate, up, down, e[:0], w[:0]).shape == (0, 128)


@pytest.mark.parametrize("tokens,experts", [(90, 16), (200, 3), (300, 4)])
def test_mlp_one_expert_takes_all(hc, tokens, experts):
    """All tokens at one expert among several, the same expert twice for a token, experts in the order of no list."""
    x, gate, up, down, e, w = layer(6, tokens, experts, 2, 192, 136, BF16)
    e[:] = experts - 1
    check(hc, (x, gate, up, down, e, w), what="one expert")
    e[:, 0] = torch.arange(tokens) % experts
    e[:, 1] = (tokens - torch.arange(tokens)) % experts
    check(hc, (x, gate, up, down, e, w), what="both ways")


@pytest.mark.parametrize("tokens", [4, 60, 150, 300])
def test_mlp_strides(hc, tokens):
    """Rows of x and of out with room between them, experts with room between them, one matrix for gate and up."""
    args = layer(7, tokens, 3, 2, 136, 72, F16, spare=24)
    x, gate, up, down, e, w = on_gpu(args)
    both = torch.full((3, 136, 160), math.nan, dtype=F16, device="cuda")
    both[:, :, :72], both[:, :, 80:152] = gate, up
    wide = torch.full((3, 80, 144), math.nan, dtype=F16, device="cuda")
    wide[:, :72, :136] = down
    out = torch.full((tokens, 152), 7.0, dtype=F16, device="cuda")
    y = hc.expert_mlp(x, both[:, :, :72], both[:, :, 80:152], wide[:, :72, :136], e, w, out=out[:, :136])
    want, tol = R.experts(*args)
    within(y, want, tol)
    assert (out[:, 136:] == 7.0).all()


def test_mlp_shared_expert(hc):
    """One expert's weights under every number (a stride of 0)."""
    x, gate, up, down, e, w = layer(8, 30, 1, 1, 64, 64, BF16)
    gate, up, down = (t.expand(4, -1, -1) for t in (gate, up, down))
    e = (torch.arange(30) % 4).int()[:, None]
    y = hc.expert_mlp(x.cuda(), *(t[:1].cuda().expand(4, -1, -1) for t in (gate, up, down)), e.cuda(), w.cuda())
    want, tol = R.experts(x, gate, up, down, e, w)
    within(y, want, tol)


@pytest.mark.parametrize("tokens", [2, 120, 300, 700])
def test_mlp_bad_values_stay(hc, tokens):
    """An infinity or a NaN reaches the tokens that have it or choose its expert, and no other's results."""
    x, gate, up, down, e, w = layer(9, tokens, 4, 1, 128, 64, BF16)
    e[:] = (torch.arange(tokens) % 2)[:, None].int()
    clean = hc.expert_mlp(*on_gpu((x, gate, up, down, e, w)))
    x[1, 5] = math.nan
    gate[2], up[3], down[3] = math.nan, math.inf, math.nan
    y = hc.expert_mlp(*on_gpu((x, gate, up, down, e, w)))
    assert torch.isnan(y[1]).all()
    keep = torch.arange(tokens) != 1
    assert torch.equal(y[keep], clean[keep])


def test_mlp_large_inner_values(hc):
    """float16 inner values past 65504 are cut to it, in every form alike."""
    for tokens in (2, 60, 200, 500):
        x, gate, up, down, e, w = layer(10, tokens, 2, 1, 64, 64, F16)
        x, gate, up, down = (torch.full_like(t, v) for t, v in ((x, 4.0), (gate, 1.0), (up, 8.0), (down, 2.0 ** -12)))
        y = hc.expert_mlp(*on_gpu((x, gate, up, down, e, w)))
        # gate = 256, up = 2048: 524288 without the cut
        assert (y.float() - 64 * 65504 * 2.0 ** -12).abs().max() <= 1024 * 2.0 ** -11


@pytest.mark.parametrize("tokens", [1, 50, 250, 900])
def test_mlp_deterministic_and_captured(hc, tokens):
    """The same bits again, on another stream, in a captured graph, and with two graphs that share a workspace."""
    args = on_gpu(layer(11, tokens, 12, 4, 640, 256, BF16))
    y = hc.expert_mlp(*args)
    for _ in range(5):
        assert torch.equal(hc.expert_mlp(*args), y)
    size = hc.expert_mlp_workspace_size(*args)
    work = torch.empty(size, dtype=torch.uint8, device="cuda").random_(0, 256)
    assert torch.equal(hc.expert_mlp(*args, workspace=work), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = hc.expert_mlp(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(z, y)
    outs, graphs = [torch.zeros_like(y) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hc.expert_mlp(*args, out=o, workspace=work)
        graphs.append(g)
    args[0].copy_(args[0].flip(0))
    want = hc.expert_mlp(*args)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert hc.debug_wait_timeouts() == 0


# ---------------------------------------------------------------------------------------------- routing --

def route_check(hc, x, k, **kw):
    gpu = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    live = gpu.get("live")
    e, w = hc.expert_route(x.cuda() if x.is_contiguous() else on_gpu([x])[0], k, **gpu)
    we, ww, tol = R.route(x, k, **{**kw, "live": None if live is None else int(live)})
    assert e.dtype == torch.int32 and w.dtype == F32
    assert torch.equal(e.cpu(), we)
    within(w, ww, tol)
    return e, w


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=ids)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,k,groups,top_groups,best", [
    (1, 1, 1, 1, 1, 1), (1, 128, 8, 1, 1, 1), (5, 33, 32, 1, 1, 1), (3, 1024, 32, 1, 1, 1), (9, 60, 6, 1, 1, 1), (17, 256, 8, 8, 4, 2),
    (4, 6, 2, 3, 1, 1), (6, 160, 6, 8, 3, 1), (5, 64, 5, 32, 7, 2), (5, 96, 3, 32, 2, 1), (3, 1020, 9, 3, 2, 2), (4, 1020, 9, 17, 5, 2),
    (7, 8, 3, 8, 4, 2), (2, 30, 10, 10, 10, 1)])
def test_route_sizes(hc, tokens, experts, k, groups, top_groups, best, scoring, dtype):
    x = rnd(20, tokens, experts, dtype=dtype, scale=2.0)
    for bias in (None, 0.2 * rnd(21, experts)):
        for renormalise in (True, False):
            route_check(hc, x, k, bias=bias, scoring=scoring, groups=groups, top_groups=top_groups, group_best=best,
                        renormalise=renormalise, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_ties(hc, scoring):
    """Equal values go to the lower index: equal logits, logits and biases that make equal sums, groups that are equal."""
    x = torch.zeros(3, 64)
    x[1, 5::7] = 1.0
    x[2] = rnd(22, 64).mul(2).round().div(2)
    for bias in (None, torch.zeros(64), torch.arange(64).remainder(4) * 0.25):
        for groups, top in ((1, 1), (8, 3)):
            for best in (1, 2):
                route_check(hc, x, 9, bias=bias, scoring=scoring, groups=groups, top_groups=top, group_best=best)


def test_route_close_values(hc):
    """Values that differ by less than float32 can tell: the order is still that of the real numbers."""
    g = torch.Generator().manual_seed(23)
    base = torch.rand(40, 1, generator=g) * 4 - 2
    steps = torch.randint(-40, 41, (40, 96), generator=g)
    x = base + steps * 2.0 ** -22
    bias = torch.randint(-3, 4, (96,), generator=g) * 2.0 ** -24
    for scoring in ("softmax", "sigmoid"):
        route_check(hc, x, 8, bias=bias, scoring=scoring)
        route_check(hc, x, 8, bias=bias, scoring=scoring, groups=8, top_groups=3, group_best=2)
        route_check(hc, x, 8, scoring=scoring, groups=8, top_groups=3, group_best=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_large_logits(hc, scoring):
    """Scores that no type tells from 1 or from 0 are in the order of their logits, and so are groups by their best."""
    for dtype in (F32, BF16):
        x = rnd(27, 30, 120, dtype=dtype, scale=50.0)
        route_check(hc, x, 9, scoring=scoring)
        route_check(hc, x, 9, scoring=scoring, groups=8, top_groups=3)
        route_check(hc, x, 9, scoring=scoring, groups=24, top_groups=5, renormalise=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_odd_values(hc, scoring):
    """Infinities, NaN, rows of nothing, scores too small for float32, experts closed by their bias."""
    x = rnd(24, 8, 40)
    x[0] = -math.inf
    x[1, 3:] = -math.inf
    x[2, 7] = math.nan
    x[3] = math.nan
    x[5] -= 300.0
    x[6, ::2] -= 500.0
    bias = 0.1 * rnd(25, 40)
    closed = bias.clone()
    closed[::3] = -math.inf
    for renormalise in (True, False):
        for b in (None, bias, closed):
            route_check(hc, x, 6, bias=b, scoring=scoring, renormalise=renormalise)
    x[4, [3, 9]] = math.inf
    e, w = hc.expert_route(x.cuda(), 4, scoring=scoring)
    assert e[4, :2].tolist() == [3, 9] and torch.isfinite(w).all()
    if scoring == "softmax":
        assert w[4].tolist() == [0.5, 0.5, 0.0, 0.0]


def test_route_live_rows_and_strides(hc):
    x = rnd(26, 50, 70, dtype=BF16)[:, 3:43]
    for live in (0, 1, 33, 50, 99):
        e, w = route_check(hc, x, 4, live=torch.tensor([live], dtype=torch.int32))
        assert (e[live:] == -1).all() and not w[live:].any()
    assert hc.expert_route(x.cuda()[:0], 4)[0].shape == (0, 4)


def test_route_captured(hc):
    x = rnd(28, 300, 64).cuda()
    bias = rnd(29, 64).cuda()
    want = hc.expert_route(x, 6, bias=bias, scoring="sigmoid")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = hc.expert_route(x, 6, bias=bias, scoring="sigmoid")
    g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = hc.expert_route(x, 6, bias=bias, scoring="sigmoid", stream=side)
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, other):
        assert torch.equal(a, b) and torch.equal(a, c)
