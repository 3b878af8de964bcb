"""The choice of tokens on the GPU against the plain float64 form of _experts_ref.py."""
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


def uniforms(seed, n):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed))


def check(hc, x, u, least=0.9, **kw):
    """Against the definition in every row that it decides by more than the kernel's weights can be off; `least` of all must
    be such rows."""
    gpu = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    g = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)
    tokens, logs = hc.token_sample(g, u.cuda(), return_logprob=True, **gpu)
    assert tokens.dtype == torch.int32 and logs.dtype == F32
    want, wl, tol, sure = R.sample(x, u, **kw)
    assert sum(sure) >= least * len(sure)
    for r, ok in enumerate(sure):
        if ok:
            assert tokens[r].item() == want[r], f"row {r}"
            assert logs[r].item() == wl[r] or abs(logs[r].item() - wl[r]) <= tol[r], f"row {r}"
    return tokens


FILTERS = [dict(), dict(temperature=0.7), dict(top_k=5), dict(top_k=1), dict(top_p=0.9), dict(top_p=0.3), dict(min_p=0.1),
           dict(top_k=50, top_p=0.8), dict(temperature=1.3, top_k=20, top_p=0.95, min_p=0.02), dict(temperature=0.0),
           dict(top_p=0.0), dict(top_k=10 ** 9, top_p=1.0, min_p=0.0), dict(min_p=1.0), dict(min_p=2.0, top_p=2.0, top_k=-3)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=ids)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (4, 101), (5, 4097), (2, 50001), (40, 4100), (2, 131072)])
def test_sizes_and_filters(hc, rows, vocab, dtype):
    """Slices of one CTA and of several, odd sizes, rows that begin anywhere."""
    x = rnd(1, rows, vocab, dtype=dtype, scale=3.0)
    for i, f in enumerate(FILTERS):
        check(hc, x, uniforms(i, rows), **f)


def test_largest_vocabulary(hc):
    x = rnd(2, 2, 409600, scale=2.5)
    check(hc, x, uniforms(3, 2))
    check(hc, x, uniforms(4, 2), top_k=409599)
    check(hc, x, uniforms(5, 2), top_p=0.99, top_k=200000)


def test_rows_choose_for_themselves(hc):
    n = 64
    x = rnd(3, n, 3001, scale=3.0)
    u = uniforms(6, n)
    t = 0.3 + uniforms(7, n)
    t[::9] = 0.0
    k = torch.randint(-2, 60, (n,), generator=torch.Generator().manual_seed(8)).int()
    p = uniforms(9, n) * 1.2
    m = (uniforms(10, n) - 0.3) * 0.2
    check(hc, x, u, temperature=t, top_k=k, top_p=p, min_p=m)
    nan = torch.full((n,), math.nan)
    a = hc.token_sample(x.cuda(), u.cuda(), top_p=nan.cuda(), min_p=nan.cuda())
    assert torch.equal(a, hc.token_sample(x.cuda(), u.cuda()))


@pytest.mark.parametrize("vocab", [64, 5000, 40000])
def test_equal_logits(hc, vocab):
    """Equal logits are ordered by their index, and their integer sums are exact: the token is known without rounding."""
    x = torch.zeros(6, vocab)
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24, 1.0])
    n = vocab
    got = check(hc, x, u)
    assert got.tolist() == [min(n - 1, math.floor(v * n)) for v in u.tolist()]
    got = check(hc, x, u, top_k=32)
    assert got.tolist() == [min(31, math.floor(v * 32)) for v in u.tolist()]
    got = check(hc, x, u, top_p=0.25)
    assert got.tolist() == [min(n // 4 - 1, math.floor(v * (n // 4))) for v in u.tolist()]
    x[:, 1::2] = -1.0
    check(hc, x, u, top_k=vocab // 2 + 5, least=0.0)
    got = check(hc, x, u, top_k=vocab // 2)
    assert got.tolist() == [2 * min(n // 2 - 1, math.floor(v * (n // 2))) for v in u.tolist()]
    # the last of equal ones stays in part
    got = hc.token_sample(x.cuda(), torch.full((6,), 1.0).cuda(), top_k=vocab // 2 + 5)
    assert got.tolist() == [2 * (vocab // 2 - 1)] * 6 if vocab > 10 else True


def test_coarse_logits(hc):
    """Few distinct values, many of each, so that the border of every filter lies among equal ones."""
    x = rnd(11, 24, 20000).mul(3).round()
    u = uniforms(12, 24)
    for f in (dict(top_k=700), dict(top_p=0.4), dict(top_k=5000, top_p=0.7), dict(top_k=9999, top_p=0.9, min_p=0.01)):
        check(hc, x, u, **f)


def test_close_logits(hc):
    """Logits a few units in the last place apart, and logits over the whole range of float32."""
    g = torch.Generator().manual_seed(13)
    x = 5.0 + torch.randint(0, 3000, (8, 6000), generator=g) * 2.0 ** -21
    check(hc, x, uniforms(14, 8), top_k=1500)
    check(hc, x, uniforms(15, 8), top_p=0.5)
    y = rnd(16, 8, 6000) * 10.0 ** (torch.rand(8, 6000, generator=g) * 70 - 35)
    check(hc, y, uniforms(17, 8), top_k=40)
    check(hc, y, uniforms(18, 8), temperature=1e30, top_p=0.5, least=0.0)


def test_odd_values(hc):
    x = rnd(19, 9, 1000)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 5:] = -math.inf
    x[3, ::2] = math.nan
    x[4, 10:990] = -math.inf
    u = uniforms(20, 9)
    for f in FILTERS:
        got = check(hc, x, u, **f)
        assert got[0] == -1 and got[1] == -1
    x[5, [100, 700]] = math.inf
    tokens, logs = hc.token_sample(x.cuda(), torch.full((9,), 0.75).cuda(), return_logprob=True)
    assert tokens[5] == 700 and abs(logs[5].item() + math.log(2)) < 1e-6
    assert hc.token_sample(x.cuda(), torch.full((9,), 0.25).cuda(), top_p=0.5, top_k=7)[5] == 100
    # uniform outside 0 .. 1
    y = torch.zeros(4, 10).cuda()
    assert hc.token_sample(y, torch.tensor([-1.0, math.nan, 2.0, math.inf]).cuda()).tolist() == [0, 0, 9, 9]
    # temperatures at both ends
    t = torch.tensor([math.inf, 1e-38, 1e-45, 3e38])
    z = torch.tensor([[0.0, 1.0, 2.0, 2.0]]).repeat(4, 1).cuda()
    got = hc.token_sample(z, torch.full((4,), 0.6).cuda(), temperature=t.cuda())
    assert got.tolist() == [2, 3, 3, 2]


def test_large_temperatures_and_masked_logits(hc):
    """A masked token is not drawn however large the temperature."""
    x = torch.full((5, 4000), -math.inf)
    x[:, 1234] = 0.5
    x[:, 3999] = -0.5
    got = hc.token_sample(x.cuda(), torch.linspace(0, 1, 5).cuda(), temperature=torch.tensor([1.0, 1e9, 1e38, math.inf, 1.0]).cuda())
    assert set(got.tolist()) <= {1234, 3999} and got[0] == 1234 and got[3] == 3999


def test_strides(hc):
    x = rnd(21, 6, 5000, dtype=BF16)[:, 7:4500]
    check(hc, x, uniforms(22, 6), top_p=0.9)
    y = rnd(23, 1, 3000).expand(5, -1)
    got = hc.token_sample(y[:1].cuda().expand(5, -1), torch.linspace(0, 0.99, 5).cuda())
    want = R.sample(y, torch.linspace(0, 0.99, 5))[0]
    assert got.tolist() == list(want)
    assert hc.token_sample(x.cuda()[:0], uniforms(1, 0).cuda()).shape == (0,)


def test_distribution(hc):
    """Evenly spaced numbers hit every token as often as its probability says."""
    p = torch.tensor([0.05, 0.4, 0.0, 0.15, 0.25, 0.15])
    x = p.log()[None].expand(1000, -1)
    u = (torch.arange(1000) + 0.5) / 1000
    got = hc.token_sample(p.log()[None].cuda().expand(1000, -1), u.cuda())
    assert torch.bincount(got, minlength=6).tolist() == [50, 400, 0, 150, 250, 150]
    got = hc.token_sample(p.log()[None].cuda().expand(1000, -1), u.cuda(), top_k=2)
    assert x.shape[0] == 1000 and abs(torch.bincount(got, minlength=6)[1].item() - 615) <= 1


def test_captured_and_on_a_stream(hc):
    x, u = rnd(24, 5, 50000).cuda(), uniforms(25, 5).cuda()
    p = torch.full((5,), 0.9).cuda()
    want = hc.token_sample(x, u, top_p=p, return_logprob=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = hc.token_sample(x, u, top_p=p, return_logprob=True)
    for _ in range(3):
        g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = hc.token_sample(x, u, top_p=p, return_logprob=True, stream=side)
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, other):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=ids)
@pytest.mark.parametrize("rows,vocab,scale", [(40, 50001, 2.0), (300, 4099, 3.0), (8, 262144, 1.0), (600, 2047, 0.3), (3, 400001, 6.0),
                                              (44, 50001, 2.0), (600, 4099, 3.0), (1100, 2047, 0.3), (6, 400001, 6.0)])
def test_whole_distribution(hc, rows, vocab, scale, dtype):
    """Large calls that filter nothing, whose rows are read by chunks."""
    x = rnd(30, rows, vocab + 5, dtype=dtype, scale=scale)[:, 3:vocab + 3]
    check(hc, x, uniforms(31, rows))
    check(hc, x, uniforms(32, rows), temperature=0.7)
    t = 0.2 + uniforms(33, rows)
    t[::7] = 0.0
    check(hc, x, uniforms(34, rows), temperature=t)


@pytest.mark.parametrize("n", [64, 128])
def test_whole_distribution_odd_rows(hc, n):
    """(By the kernel for any row, and by chunks first.)"""
    vocab = 20000
    x = rnd(35, n, vocab, scale=2.0)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 5:] = -math.inf
    x[3, ::2] = math.nan
    x[4, 1024:19000] = -math.inf
    x[5] = 0.0
    x[6] = 1e30 * x[6]
    x[7] -= 1e6
    u = uniforms(36, n)
    u[8:12] = torch.tensor([0.0, 1.0, 1.0 - 2.0 ** -24, 2.0 ** -24])
    check(hc, x, u)
    check(hc, x, u, temperature=0.01)
    x[12, 777], x[12, 15000] = math.inf, math.inf
    got = hc.token_sample(x.cuda(), torch.full((n,), 0.75).cuda())
    assert got[12] == 15000 and got[0] == -1
    t = torch.ones(n)
    t[5], t[13], t[14] = math.inf, 1e-38, math.nan
    got = hc.token_sample(x.cuda(), torch.full((n,), 0.5).cuda(), temperature=t.cuda())
    assert got[5] == vocab // 2 and got[13] == int(x[13].argmax()) and got[14] == int(x[14].argmax())
    y = torch.zeros(n, vocab).cuda()
    assert hc.token_sample(y, (torch.arange(n) / n).cuda()).tolist() == [i * vocab // n for i in range(n)]


@pytest.mark.parametrize("k", [2, 100, 1000, 2040, 2049, 3000])
def test_listed_candidates(hc, k):
    """Around the number of tokens that one CTA sorts by itself, with equal logits at the border, with and without top_p."""
    x = rnd(37, 6, 30000, scale=2.0)
    x[3] = x[3].mul(2).round()
    x[4] = x[4].mul(50).round() / 50
    u = uniforms(38, 6)
    check(hc, x, u, top_k=k)
    check(hc, x, u, top_k=k, top_p=0.8, min_p=0.01)
    check(hc, x, u, top_p=0.02 + k / 40000)
    check(hc, x, u, temperature=0.3, top_p=0.9)


@pytest.mark.parametrize("scale", [0.3, 2.0])
def test_many_that_stay(hc, scale):
    """Borders among thousands of tokens: steps that hold few and many, equal logits at the border, one border behind another."""
    x = rnd(39, 5, 130001, scale=scale)
    x[1] = x[1].mul(8).round() / 8
    x[2] = x[2].mul(1000).round() / 1000
    x[3, ::2] = -math.inf
    x[4, 1000:] -= 40.0 * scale
    u = uniforms(40, 5)
    for k in (2500, 20000, 64000, 100000, 130000):
        check(hc, x, u, top_k=k)
        check(hc, x, u, top_k=k, top_p=0.7)
    for p in (0.2, 0.9, 0.999):
        check(hc, x, u, top_p=p)
        check(hc, x, u, top_p=p, temperature=0.5)
    y = rnd(41, 40, 30000, scale=scale, dtype=BF16)
    check(hc, y, uniforms(42, 40), top_k=5000, top_p=0.9, least=0.5)
    check(hc, y, uniforms(43, 40), top_p=0.95, least=0.5)
