"""The paged-cache operators (rotary positions, attention over pages, upkeep of the pages) on the GPU against the plain
float64 forms and bounds of _paged_ref.py."""
import math
import random

import pytest
import torch

import _paged_ref as R

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
    assert torch.equal(torch.isinf(got), torch.isinf(want)), what + ": infinity elsewhere"
    fine = torch.isfinite(want)
    over = (got - want).abs()[fine] - tol[fine]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: {over.max():.3e} over the bound"


# --------------------------------------------------------------------------------------------- rotary --

@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,dim,rot", [(1, 64, 64), (20, 128, 128), (5, 128, 64), (3, 80, 24), (2, 7, 4), (3, 256, 250),
                                           (4, 64, 0), (1, 2, 2), (2, 1024, 1024)])
def test_rotary(hc, dtype, interleaved, heads, dim, rot):
    tokens = 37
    x = rnd(1, tokens, heads, dim, dtype=dtype)
    r = random.Random(dim + rot)
    at = torch.tensor([0, 1, 2, 131071, 2 ** 24 + 1, 2 ** 31 + 7, -1, -5000] + [r.randrange(500000) for _ in range(29)])
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    for inverse, amplitude in [(False, 1.0), (True, 1.25)]:
        want, tol = R.rotate(x, at, f, amplitude, interleaved, inverse)
        got = hc.rotary(x.cuda(), at.cuda(), f.cuda(), amplitude=amplitude, interleaved=interleaved, inverse=inverse)
        within(got, want, tol, "out")
    small = at.clamp(-2 ** 31, 2 ** 31 - 1)
    got = hc.rotary(x.cuda(), small.int().cuda(), f.cuda(), interleaved=interleaved)
    want, tol = R.rotate(x, small, f, 1.0, interleaved)
    within(got, want, tol, "int32 positions")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=ids)
@pytest.mark.parametrize("tokens", [0, 1, 3, 20011])
def test_rotary_lengths_strides_and_in_place(hc, dtype, tokens):
    heads, dim, rot = 3, 64, 32
    f, _ = hc.rotary_frequencies(rot)
    at = torch.arange(tokens)
    wide = rnd(2, tokens, heads + 2, dim + 8, dtype=dtype).cuda()
    for x in (wide[:, 1:heads + 1, 8:], wide[:, 1:heads + 1, 3:dim + 3],
              wide[:, :heads, :dim].transpose(0, 1).contiguous().transpose(0, 1)):
        want, tol = R.rotate(x.cpu(), at, f.cpu())
        got = hc.rotary(x, at.cuda(), f)
        within(got, want, tol, "strided")
        before = wide.clone()
        hc.rotary(x, at.cuda(), f, out=x)
        assert torch.equal(x, got), "in place"
        if x.data_ptr() >= wide.data_ptr() and tokens and x.stride(0) == wide.stride(0):
            x.copy_(torch.as_strided(before, x.shape, x.stride(), x.storage_offset()))
            assert torch.equal(wide, before), "wrote beside x"


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient(hc, interleaved):
    """The inverse rotation is the gradient: against the formula's transpose, and against differences of the forward (which
    is linear, so that a difference of any width is exact up to the bounds of its two ends)."""
    x, g = rnd(3, 9, 2, 32), rnd(4, 9, 2, 32)
    f, _ = hc.rotary_frequencies(20)
    at = torch.arange(9) * 1000
    grad = hc.rotary(g.cuda(), at.cuda(), f, amplitude=1.5, interleaved=interleaved, inverse=True)
    want, tol = R.rotate(g, at, f.cpu(), 1.5, interleaved, inverse=True)
    within(grad, want, tol, "formula")
    r = random.Random(5)
    y = hc.rotary(x.cuda(), at.cuda(), f, amplitude=1.5, interleaved=interleaved).double()
    _, ty = R.rotate(x, at, f.cpu(), 1.5, interleaved)
    for _ in range(24):
        t, h, d = r.randrange(9), r.randrange(2), r.randrange(32)
        x2 = x.clone()
        x2[t, h, d] += 1.0
        step = float(x2[t, h, d].double() - x[t, h, d].double())
        y2 = hc.rotary(x2.cuda(), at.cuda(), f, amplitude=1.5, interleaved=interleaved).double()
        _, ty2 = R.rotate(x2, at, f.cpu(), 1.5, interleaved)
        change = float(((y2 - y) * g.cuda().double()).sum())
        bound = float(((ty + ty2)[t, h] * g[t, h].abs().double()).sum()) + float(tol[t, h, d])
        assert abs(change - step * float(grad[t, h, d])) <= 1.5 * bound


def test_rotary_frequencies(hc):
    f, a = hc.rotary_frequencies(8, 10000.0, device="cpu")
    assert a == 1.0 and f.tolist() == [1.0, 0.1, 0.01, 0.001]
    g, _ = hc.rotary_frequencies(8, 10000.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(g, f / 4)
    g, _ = hc.rotary_frequencies(8, 10000.0, scaling="base", factor=4.0, device="cpu")
    assert g[0] == 1.0 and abs(float(g[-1] / (f[-1] / 4)) - 1) < 1e-12
    # turns in 1000 tokens: 159, 16, 1.6, 0.16
    g, a = hc.rotary_frequencies(8, 10000.0, scaling="by_parts", factor=4.0, original_length=1000, slow=1.0, fast=32.0,
                                 device="cpu")
    assert abs(a - (0.1 * math.log(4) + 1)) < 1e-12 and g[0] == f[0] and abs(float(g[3] / f[3]) - 0.25) < 1e-12
    keep = (1000 * 0.1 / (2 * math.pi) - 1) / 31
    assert abs(float(g[1]) - 0.1 * (keep + (1 - keep) / 4)) < 1e-12


# -------------------------------------------------------------------------------------- caches and batches --

class Batch:
    """Sequences with (new tokens, tokens in all), their pages scattered over a pool whose unused places hold `stale`."""

    def __init__(self, seed, both, heads, kv_heads, dim, page, dtype, cu=True, layout="token", stale=math.nan, extra=2):
        r = random.Random(seed)
        self.both, self.page, self.dtype = both, page, dtype
        used = [max(0, -(-n // page)) for _, n in both]
        self.width = max(used + [1]) + 1
        pages = sum(used) + extra
        order = list(range(pages))
        r.shuffle(order)
        rows = []
        for u in used:
            # entries past the used ones are wild on purpose: nobody may follow them
            rows.append(order[:u] + [r.choice([-1, -7, pages, 2 ** 31 - 1]) for _ in range(self.width - u)])
            order = order[u:]
        self.table = torch.tensor(rows, dtype=torch.int32).reshape(len(both), self.width)
        self.lens = torch.tensor([n for _, n in both], dtype=torch.int32)
        starts = [0]
        for q, _ in both:
            starts.append(starts[-1] + q)
        self.starts, self.tokens = starts, starts[-1]
        self.cu = torch.tensor(starts, dtype=torch.int32) if cu else None
        self.k = self.pool(rnd(seed + 1, pages, page, kv_heads, dim, dtype=dtype), layout)
        self.v = self.pool(rnd(seed + 2, pages, page, kv_heads, dim, dtype=dtype), layout)
        self.q = rnd(seed + 3, self.tokens, heads, dim, dtype=dtype, scale=1.5)
        held = torch.zeros(pages, page, dtype=torch.bool)
        for row, (_, n) in zip(rows, both):
            for j in range(max(0, n)):
                held[row[j // page], j % page] = True
        self.held = held
        if stale is not None:
            self.k[~held] = stale
            self.v[~held] = stale

    @staticmethod
    def pool(x, layout):
        """The same pool with heads before tokens in memory, or with gaps between the pages."""
        if layout == "head":
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        if layout == "gaps":
            wide = torch.full((x.shape[0], 2, *x.shape[1:]), math.nan, dtype=x.dtype)
            wide[:, 1] = x
            return wide[:, 1]
        return x

    def cuda(self, t):
        """On the GPU with the same strides."""
        if t is None or t.is_contiguous():
            return None if t is None else t.cuda()
        size = 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        g = torch.full((size + t.storage_offset(),), math.nan, dtype=t.dtype, device="cuda")
        y = torch.as_strided(g, t.shape, t.stride(), t.storage_offset())
        y.copy_(t)
        return y

    def run(self, hc, **kw):
        return hc.paged_attention(self.cuda(self.q), self.cuda(self.k), self.cuda(self.v), self.table.cuda(), self.lens.cuda(),
                                  self.cuda(self.cu), return_lse=True, **kw)

    def check(self, hc, what="", **kw):
        ref = {k: v for k, v in kw.items() if k in ("scale", "window", "softcap")}
        out, lse, tol, ltol = R.attention(self.q, self.k, self.v, self.table, self.lens, self.cu, **ref)
        got, glse = self.run(hc, **kw)
        within(got, out, tol, what + " out")
        within(glse, lse, ltol, what + " lse")
        return got, glse


# ---------------------------------------------------------------------------------------------- append --

APPENDS = [  # (both, heads, kv_heads, dim, rot, page)
    ([(1, 1)], 4, 4, 64, 64, 16),
    ([(1, 700), (1, 0), (1, 16), (1, 17)], 20, 4, 128, 128, 16),
    ([(5, 5), (0, 9), (33, 100), (1, 64), (7, 3)], 6, 2, 128, 64, 32),
    ([(3, 11), (2, 2)], 3, 1, 80, 40, 7),
    ([(4, 9), (2, 40)], 2, 2, 10, 6, 1),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"s{len(c[0])}d{c[3]}p{c[5]}")
@pytest.mark.parametrize("layout", ["token", "head", "gaps"])
def test_rotary_append(hc, dtype, interleaved, case, layout):
    both, heads, kv_heads, dim, rot, page = case
    single = all(q == 1 for q, _ in both)
    b = Batch(7, both, heads, kv_heads, dim, page, dtype, cu=not single, layout=layout, stale=None)
    mixed = rnd(11, b.tokens, heads + 2 * kv_heads, dim, dtype=dtype)  # one projection's rows: q, k and v side by side
    q, k, v = mixed.split([heads, kv_heads, kv_heads], 1)
    f, _ = hc.rotary_frequencies(rot)
    kc, vc, g = b.cuda(b.k), b.cuda(b.v), mixed.cuda()
    gq, gk, gv = g.split([heads, kv_heads, kv_heads], 1)
    got = hc.rotary_append(gq, gk, gv, kc, vc, b.table.cuda(), b.lens.cuda(), b.cuda(b.cu), inv_freq=f, amplitude=0.75,
                           interleaved=interleaved)
    at = torch.cat([torch.arange(n - nq, n) for nq, n in both])
    want, tol = R.rotate(q, at, f.cpu(), 0.75, interleaved)
    within(got, want, tol, "q")
    wk, tk = R.rotate(k, at, f.cpu(), 0.75, interleaved)
    ek, ev, et = b.k.double().clone(), b.v.double().clone(), torch.zeros(b.k.shape, dtype=torch.float64)
    for s, (nq, n) in enumerate(both):
        for i in range(nq):
            p, t = n - nq + i, b.starts[s] + i
            if p < 0:
                continue
            place = (int(b.table[s, p // page]), p % page)
            ek[place], ev[place], et[place] = wk[t], v[t].double(), tk[t]
    within(kc, ek, et, "keys")
    assert torch.equal(vc.cpu().double(), ev), "values"
    # in place, q among the columns of the projection's output
    again = hc.rotary_append(gq, gk, gv, kc, vc, b.table.cuda(), b.lens.cuda(), b.cuda(b.cu), inv_freq=f, amplitude=0.75,
                             interleaved=interleaved, out=gq)
    assert again is gq and torch.equal(gq, got)
    assert torch.equal(gk.cpu(), k) and torch.equal(gv.cpu(), v)


def test_append_passes_over_missing_pages(hc):
    b = Batch(3, [(2, 40), (1, 17)], 2, 1, 64, 16, BF16, stale=None)
    b.table[0, 2] = b.k.shape[0]  # outside the pool
    b.table[1, 1] = -1
    kc, vc = b.k.cuda(), b.v.cuda()
    f, _ = hc.rotary_frequencies(64)
    k = rnd(1, 3, 1, 64, dtype=BF16).cuda()
    hc.rotary_append(b.q.cuda(), k, k, kc, vc, b.table.cuda(), b.lens.cuda(), b.cu.cuda(), inv_freq=f)
    assert torch.equal(kc.cpu(), b.k) and torch.equal(vc.cpu(), b.v)


# ------------------------------------------------------------------------------------------- attention --

SINGLES = [  # (lengths, heads, kv_heads, dim, page)
    ([1], 1, 1, 64, 16),
    ([0, 1, 2, 15, 16, 17], 4, 4, 64, 16),
    ([700], 20, 4, 128, 16),
    ([33, 0, 4097, 128, 129, 511], 32, 8, 128, 64),
    ([2000, 31], 8, 1, 64, 128),
    ([100, 257], 16, 1, 128, 32),
    ([300, 77], 20, 1, 128, 16),
    ([130, 9], 40, 1, 64, 16),
    ([65, 200], 5, 5, 128, 7),
    ([45, 3], 6, 2, 80, 5),
    ([260], 2, 1, 256, 16),
    ([90, 31], 3, 3, 40, 1),
    ([19], 2, 2, 5, 3),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("case", SINGLES, ids=lambda c: f"n{max(c[0])}h{c[1]}k{c[2]}d{c[3]}p{c[4]}")
def test_attention_single_tokens(hc, dtype, case):
    lens, heads, kv_heads, dim, page = case
    b = Batch(13, [(1, n) for n in lens], heads, kv_heads, dim, page, dtype, cu=False)
    got, lse = b.check(hc)
    b.check(hc, "hints", max_q=1, max_kv=max(lens))
    again, lse2 = b.run(hc)
    assert torch.equal(got, again) and torch.equal(lse, lse2), "not the same bits twice"
    b.check(hc, "window", window=33)
    b.check(hc, "capped", softcap=5.0, scale=0.3)


CHUNKS = [  # ((new, all), heads, kv_heads, dim, page)
    ([(1, 1), (2, 2), (3, 5)], 2, 2, 64, 16),
    ([(17, 17), (1, 40), (0, 12), (5, 3), (3, 0), (64, 200)], 4, 2, 128, 16),
    ([(129, 400)], 4, 1, 128, 64),
    ([(300, 300), (1, 129), (31, 129)], 5, 1, 64, 32),
    ([(70, 1100), (2, 900)], 8, 2, 128, 128),
    ([(40, 555), (9, 60)], 3, 1, 128, 256),
    ([(130, 131)], 7, 1, 64, 16),
    ([(33, 77), (20, 21)], 2, 1, 96, 16),
    ([(25, 61)], 6, 3, 128, 7),
    ([(12, 30)], 2, 2, 200, 8),
    ([(9, 20)], 40, 1, 64, 16),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: f"q{max(q for q, _ in c[0])}h{c[1]}k{c[2]}d{c[3]}p{c[4]}")
def test_attention_chunks(hc, dtype, case):
    both, heads, kv_heads, dim, page = case
    b = Batch(17, both, heads, kv_heads, dim, page, dtype)
    got, lse = b.check(hc)
    b.check(hc, "hints", max_q=max(q for q, _ in both), max_kv=max(n for _, n in both))
    again, lse2 = b.run(hc)
    assert torch.equal(got, again) and torch.equal(lse, lse2), "not the same bits twice"
    b.check(hc, "window", window=19)
    b.check(hc, "window of one", window=1)
    b.check(hc, "capped", softcap=4.0, scale=0.4, window=100)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [1, 4, 8, 24, 128, 384, 512])
def test_attention_page_sizes(hc, dtype, dim, page):
    """Pages that divide the kernels' blocks of keys, are multiples of them, or neither."""
    Batch(67, [(70, 700), (1, 513), (3, 3)], 4, 2, dim, page, dtype).check(hc, window=300)
    Batch(71, [(1, 700), (1, 513)], 4, 2, dim, page, dtype, cu=False).check(hc)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("layout", ["head", "gaps"])
def test_attention_layouts(hc, dtype, layout):
    Batch(19, [(1, 300), (1, 45)], 8, 2, 128, 16, dtype, cu=False, layout=layout).check(hc)
    Batch(23, [(100, 300), (1, 45)], 8, 2, 64, 32, dtype, layout=layout).check(hc)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids)
def test_attention_strided_and_unaligned_queries(hc, dtype):
    """Queries as columns of a projection's output, once at an odd place (no 16-byte vectors), once read from the last axis
    outwards; out given, with gaps of its own that stay as they are."""
    for both in ([(1, 200), (1, 31)], [(60, 200), (7, 31)]):
        b = Batch(29, both, 4, 2, 64, 16, dtype, cu=both[0][0] > 1)
        want, _, tol, _ = R.attention(b.q, b.k, b.v, b.table, b.lens, b.cu)
        rest = (b.k.cuda(), b.v.cuda(), b.table.cuda(), b.lens.cuda(), b.cuda(b.cu))
        wide = torch.zeros(b.tokens, 4 * 64 + 80, dtype=dtype, device="cuda")
        for at in (8, 3):
            q = wide[:, at:at + 256].view(b.tokens, 4, 64) if at else None
            q.copy_(b.q)
            within(hc.paged_attention(q, *rest), want, tol, f"at {at}")
        q = b.q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        out = torch.full((b.tokens, 4, 100), 7.0, dtype=dtype, device="cuda")
        hc.paged_attention(q, *rest, out=out[:, :, 20:84])
        within(out[:, :, 20:84], want, tol, "out given")
        assert bool((out[:, :, :20] == 7).all() and (out[:, :, 84:] == 7).all())


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_magnitudes(hc, dtype, dim):
    """Scores far apart (one key outweighs the rest, and the largest comes late, so that the running maximum rises by much
    and often), and all alike."""
    for both in ([(1, 1500)], [(140, 1500)]):
        b = Batch(31, both, 4, 1, dim, 16, dtype, cu=both[0][0] > 1)
        rise = torch.linspace(0, 1, 1500)
        for j in range(1500):
            b.k[int(b.table[0, j // 16]), j % 16] *= 4 * float(rise[j])
        b.check(hc, "rising", scale=1.0)
        b.check(hc, "negative scale", scale=-0.2)
        for j in range(1500):
            b.k[int(b.table[0, j // 16]), j % 16] = 0
        b.check(hc, "alike")
        b.check(hc, "no scale", scale=0.0)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("scale", [0.001, 0.02, 0.05, 0.2, 2.0])
def test_attention_caps(hc, dtype, dim, scale):
    """Scores that are small against the cap, near it, beyond it, and in one block all of these."""
    for both in ([(1, 300)], [(140, 700), (9, 20)]):
        b = Batch(83, both, 4, 2, dim, 16, dtype, cu=both[0][0] > 1)
        b.check(hc, "whole", softcap=5.0, scale=scale)
        b.check(hc, "window", softcap=5.0, scale=scale, window=90)
        b.q[::3] *= 0.05
        b.k[:, 5] *= 4
        b.check(hc, "mixed", softcap=5.0, scale=scale)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=ids)
def test_attention_split_and_not_split_agree(hc, dtype):
    """One sequence is split over the GPU, a hundred are not; both within the bound, so the split's joining is exact."""
    one = Batch(37, [(1, 3001)], 8, 2, 128, 16, dtype, cu=False)
    one.check(hc)
    many = Batch(41, [(1, 301 + i) for i in range(100)], 8, 2, 128, 16, dtype, cu=False)
    many.check(hc)
    # a bound on kv_lens that is wrong steers the split, not the result
    one.check(hc, "low bound", max_kv=100)
    Batch(43, [(90, 2000)], 8, 2, 128, 16, dtype).check(hc, "low bounds", max_kv=64, max_q=1)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("hints", [(0, 0), (1, 1), (7, 30), (10 ** 6, 10 ** 9)], ids=lambda h: f"q{h[0]}kv{h[1]}")
def test_attention_wrong_hints(hc, dtype, dim, hints):
    """Bounds that are too low or too high choose the kernel and the split, not the result."""
    kw = dict(max_q=hints[0], max_kv=hints[1])
    Batch(101, [(1, 700), (1, 0), (1, 33)], 8, 2, dim, 16, dtype, cu=False).check(hc, "single", **kw)
    Batch(103, [(1, 700), (40, 600), (0, 9), (5, 5)], 8, 2, dim, 16, dtype).check(hc, "chunks", window=70, **kw)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("both", [[(1, 320), (1, 160)], [(70, 320), (1, 160)]], ids=["single", "chunk"])
def test_attention_lengths_and_pages_out_of_range(hc, dtype, dim, both):
    """A length past what the table's row holds is cut to it; a negative one counts as none; a sequence with pages outside the
    pool disturbs no other."""
    b = Batch(107, both, 8, 2, dim, 16, dtype, cu=both[0][0] > 1)
    b.table = b.table[:, :20].contiguous()
    out, lse, tol, ltol = R.attention(b.q, b.k, b.v, b.table, b.lens, b.cu)
    b.lens = torch.tensor([2 ** 31 - 1, 160], dtype=torch.int32)
    got, glse = b.run(hc)
    within(got, out, tol, "long")
    within(glse, lse, ltol, "long lse")
    b.table[0, 3], b.table[0, 4] = -1, 10 ** 9
    n = both[0][0]
    got, glse = b.run(hc)
    within(got[n:], out[n:], tol[n:], "beside missing pages")
    within(glse[n:], lse[n:], ltol[n:], "beside missing pages, lse")
    b.lens = torch.tensor([-5, 160], dtype=torch.int32)
    got, glse = b.run(hc)
    assert bool((got[:n] == 0).all()) and bool((glse[:n] == -math.inf).all())
    within(got[n:], out[n:], tol[n:], "beside none")
    assert hc.debug_wait_timeouts() == 0


def test_attention_chunk_by_chunk(hc):
    """A prompt read at once and in pieces gives every token the same result, within the bounds of both."""
    f, _ = hc.rotary_frequencies(128)
    n, heads, kv_heads, dim, page = 333, 8, 2, 128, 16
    q, k, v = (rnd(s, n, h, dim, dtype=BF16).cuda() for s, h in ((1, heads), (2, kv_heads), (3, kv_heads)))
    table = torch.randperm(24, generator=torch.Generator().manual_seed(1))[:21].int().view(1, 21)
    kc = torch.full((24, page, kv_heads, dim), math.nan, dtype=BF16, device="cuda")
    vc = kc.clone()
    pieces, qs = [], []
    for a, b in ((0, 100), (100, 101), (101, 130), (130, 131), (131, 333)):
        lens, cu = torch.tensor([b], dtype=torch.int32).cuda(), torch.tensor([0, b - a], dtype=torch.int32).cuda()
        qr = hc.rotary_append(q[a:b], k[a:b], v[a:b], kc, vc, table.cuda(), lens, cu, inv_freq=f)
        pieces.append(hc.paged_attention(qr, kc, vc, table.cuda(), lens, cu))
        qs.append(qr)
    cu = torch.tensor([0, n], dtype=torch.int32)
    lens = torch.tensor([n], dtype=torch.int32)
    want, _, tol, _ = R.attention(torch.cat(qs).cpu(), kc.cpu(), vc.cpu(), table, lens, cu)
    within(torch.cat(pieces), want, tol, "in pieces")


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
def test_attention_nan_reaches_only_its_own(hc, dtype):
    """A NaN in a query stays in its own head; one in a sequence's keys or values leaves other sequences alone."""
    b = Batch(47, [(30, 200), (1, 90), (25, 60)], 4, 2, 128, 16, dtype)
    clean, _ = b.run(hc)
    b.q[3, 2, 5] = math.nan
    got, _ = b.run(hc)
    assert bool(torch.isnan(got[3, 2]).all())
    got[3, 2] = clean[3, 2]
    assert torch.equal(got, clean)
    b.q[3, 2, 5] = 0
    base, _ = b.run(hc)
    b.v[int(b.table[1, 2]), 3, 0, 7] = math.inf  # sequence 1 (one new token, which sees it), key head 0
    got, _ = b.run(hc)
    assert bool(torch.isinf(got[30, :2, 7]).all())
    got[30, :2, 7] = base[30, :2, 7]
    assert torch.equal(got, base)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim,page,flags", [(64, 16, 0), (128, 32, 0), (128, 7, 0), (128, 16, 2)])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_unseen_values_may_be_anything(hc, dtype, dim, page, flags, window):
    """Infinities and NaN in values (and NaN in keys) of tokens that only some of the new tokens see reach those alone: the last
    new tokens' own, and, with a window, some that only the first of them still see. Few new tokens and many."""
    for both, at in (([(5, 60)], [58, 59, 17]), ([(3, 3), (2, 130)], [129]), ([(150, 333)], [330, 300, 250, 190, 150])):
        for what in ("one value", "whole values", "keys"):
            b = Batch(73, both, 4, 2, dim, page, dtype)
            s, n = len(both) - 1, both[-1][1]
            for i, j in enumerate(at):
                place = (int(b.table[s, j // page]), j % page)
                if what == "keys":
                    b.k[place] = math.nan
                elif what == "whole values":
                    b.v[place] = math.nan
                else:
                    b.v[place][i % 2, (7 * i + 3) % dim] = [math.inf, math.nan, -math.inf][i % 3]
            out, lse, tol, ltol = R.attention(b.q, b.k, b.v, b.table, b.lens, b.cu, window=window)
            got, glse = b.run(hc, window=window, flags=flags)
            within(got, out, tol, what)
            within(glse, lse, ltol, what + " lse")


def test_attention_long_offsets(hc):
    """A pool of more than 2^31 elements, its pages far apart: offsets pass 32 bits."""
    page, kv_heads, dim = 16, 1, 64
    far = 2 ** 22 + 3  # elements between pages
    far -= far % 8
    pages = 2 ** 31 // far + 40
    pool = torch.empty(2, pages * far, dtype=BF16, device="cuda")
    views = [torch.as_strided(pool[i], (pages, page, kv_heads, dim), (far, dim, dim, 1)) for i in range(2)]
    for both in ([(1, 500)], [(100, 500)]):
        b = Batch(53, both, 2, kv_heads, dim, page, BF16, cu=both[0][0] > 1)
        n = b.k.shape[0]
        to = torch.arange(n) + pages - n
        for view, src in zip(views, (b.k, b.v)):
            view[pages - n:] = src.cuda()
        out, _, tol, _ = R.attention(b.q, b.k, b.v, b.table, b.lens, b.cu)
        table = b.table.clone()
        used = (b.table >= 0) & (b.table < n)
        table[used] = to[b.table[used].long()].int()
        got = hc.paged_attention(b.q.cuda(), *views, table.cuda(), b.lens.cuda(), b.cuda(b.cu))
        within(got, out, tol, "far pages")


def test_attention_other_stream_and_graph(hc):
    b = Batch(59, [(1, 2000), (1, 35)], 8, 2, 128, 16, BF16, cu=False)
    want, _, tol, _ = R.attention(b.q, b.k, b.v, b.table, b.lens)
    t = [x.cuda() for x in (b.q, b.k, b.v, b.table, b.lens)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [hc.paged_attention(*t, stream=side) for _ in range(20)]
    junk = [torch.full((1 << 20,), math.nan, device="cuda") for _ in range(20)]  # would take over memory freed too early
    torch.cuda.synchronize()
    for g in got:
        within(g, want, tol, "other stream")
    del junk
    ws = torch.empty(hc.paged_attention_workspace_size(*t), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(t[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hc.paged_attention(*t, out=out, workspace=ws)
    t[4].copy_(torch.tensor([1999, 20], dtype=torch.int32))  # lengths are read on the device, at each replay
    ws.fill_(255)  # NaN all over
    graph.replay()
    torch.cuda.synchronize()
    want, _, tol, _ = R.attention(b.q, b.k, b.v, b.table, torch.tensor([1999, 20]))
    within(out, want, tol, "replayed")


# ----------------------------------------------------------------------------------------------- pages --

def pool(seed, planes, pages, *rest, dtype=BF16):
    return rnd(seed, planes, pages, *rest, dtype=dtype)


@pytest.mark.parametrize("dtype,planes,pages,rest", [(BF16, 3, 11, (16, 2, 64)), (F32, 1, 7, (1, 1, 1)), (BF16, 2, 9, (3, 1, 7)),
                                                     (F16, 2, 9, (16, 8, 128)), (torch.uint8, 2, 5, (13,))], ids=str)
def test_page_copy(hc, dtype, planes, pages, rest):
    c = torch.randint(0, 255, (planes, pages, *rest), generator=torch.Generator().manual_seed(1)).to(dtype)
    src = torch.tensor([0, 3, -1, pages, 2], dtype=torch.int32)
    dst = torch.tensor([1, 4, 2, 2, -5], dtype=torch.int32)
    want = c.clone()
    want[:, 1], want[:, 4] = c[:, 0], c[:, 3]
    g = c.cuda()
    assert hc.page_copy(g, src.cuda(), dst.cuda()) is g
    assert torch.equal(g.cpu(), want)
    hc.page_copy(g, src[:0].cuda(), dst[:0].cuda())
    assert torch.equal(g.cpu(), want)


def tables(seed, seqs, width, page, pages, most, wild=True):
    """Sequences that share some of their first pages, lengths from none to full, and counts with a few outside holders."""
    r = random.Random(seed)
    order = list(range(pages))
    r.shuffle(order)
    lens = [r.choice([0, 1, page, page + 1, width * page, r.randint(0, width * page)]) if i % 2 else r.randint(0, width * page)
            for i in range(seqs)]
    rows, refs, first = [], [0] * pages, []
    for i, n in enumerate(lens):
        u = -(-n // page)
        row = (first[: r.randint(0, len(first))] if i % 3 else [])[:u]
        while len(row) < u and len(order) > pages - most:
            row.append(order.pop())
        while len(row) < u:  # the pool is out: a hole in the table
            row.append(-1)
        first = row if i % 3 == 0 else first
        for p in row:
            if p >= 0:
                refs[p] += 1
        tail = [r.choice([-1, pages, -2 ** 31, 5]) if wild else -1 for _ in range(width - u)]
        rows.append(row + tail)
    for p in order[:3]:
        refs[p] += 2  # held by somebody else
    return (torch.tensor(rows, dtype=torch.int32).reshape(seqs, width), torch.tensor(lens, dtype=torch.int32),
            torch.tensor(refs, dtype=torch.int32))


POOLS = [(1, 1, 1, 4, 4), (5, 6, 16, 64, 60), (16, 9, 16, 200, 190), (33, 4, 7, 120, 110), (40, 300, 4, 30000, 20000),
         (3, 2, 1 << 10, 70000, 6), (130, 70, 16, 9500, 9450)]  # (sequences, width, page size, pages, pages in use at most)


@pytest.mark.parametrize("sizes", POOLS, ids=str)
def test_page_fork(hc, sizes):
    seqs, width, page, pages, most = sizes
    table, lens, refs = tables(61, seqs, width, page, pages, most)
    r = random.Random(62)
    for children in (seqs, 0, 2 * seqs + 1):
        parents = [r.choice([-1, r.randrange(seqs), r.randrange(max(1, seqs // 3)), 10 ** 6]) for _ in range(children)]
        c = pool(63, 2, pages, page if page < 100 else 1, 1, 2)
        g = c.cuda()
        t, n, k, missing = hc.page_fork(g, table.cuda(), lens.cuda(), refs.cuda(),
                                        torch.tensor(parents, dtype=torch.int32).cuda(), page_size=page)
        wt, wn, wk, wm, copies = R.Pages(table, lens, refs, page).fork(parents)
        assert torch.equal(t.cpu(), wt) and n.tolist() == wn and k.tolist() == wk and missing.tolist() == [wm]
        for a, b in copies:
            c[:, b] = c[:, a]
        assert torch.equal(g.cpu(), c), "pages"


def test_page_fork_without_free_pages(hc):
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    lens, refs = torch.tensor([20, 25], dtype=torch.int32), torch.tensor([1, 1, 1, 1, 1], dtype=torch.int32)
    parents = [0, 0, 1, 0, 1]
    c = pool(1, 2, 5, 16, 1, 8)
    g = c.cuda()
    t, n, k, missing = hc.page_fork(g, table.cuda(), lens.cuda(), refs.cuda(), torch.tensor(parents, dtype=torch.int32).cuda())
    assert missing.tolist() == [3] and n.tolist() == [20, 20, 25, 20, 25]
    assert t.tolist() == [[0, 1], [0, -1], [2, 3], [0, -1], [2, -1]] and k.tolist() == [3, 1, 2, 1, 1]
    assert torch.equal(g.cpu(), c)


@pytest.mark.parametrize("sizes", POOLS, ids=str)
def test_page_extend_and_release(hc, sizes):
    seqs, width, page, pages, most = sizes
    table, lens, refs = tables(71, seqs, width, page, pages, most)
    r = random.Random(72)
    for top in (1, page, 3 * page, width * page):
        more = [r.choice([0, r.randint(0, top), -3]) for _ in range(seqs)]
        t, n, k, missing = hc.page_extend(table.cuda(), lens.cuda(), refs.cuda(), torch.tensor(more, dtype=torch.int32).cuda(),
                                          page_size=page)
        wt, wn, wk, wm = R.Pages(table, lens, refs, page).extend(more)
        assert torch.equal(t.cpu(), wt) and n.tolist() == wn and k.tolist() == wk and missing.tolist() == [wm]
    drop = [r.random() < 0.5 for _ in range(seqs)]
    t, n, k = hc.page_release(table.cuda(), lens.cuda(), refs.cuda(), torch.tensor(drop).cuda(), page_size=page)
    wt, wn, wk = R.Pages(table, lens, refs, page).release(drop)
    assert torch.equal(t.cpu(), wt) and n.tolist() == wn and k.tolist() == wk


@pytest.mark.parametrize("sizes", POOLS, ids=str)
def test_page_compact(hc, sizes):
    seqs, width, page, pages, most = sizes
    table, lens, refs = tables(81, seqs, width, page, pages, most)
    c = pool(83, 3, pages, page if page < 100 else 1, 1, 8 if page != 7 else 1)
    g = c.cuda()
    t, k, remap, live = hc.page_compact(g, table.cuda(), lens.cuda(), refs.cuda(), page_size=page)
    wt, wk, wr, wl, moves = R.Pages(table, lens, refs, page).compact()
    assert torch.equal(t.cpu(), wt) and k.tolist() == wk and remap.tolist() == wr and live.tolist() == [wl]
    for a, b in moves:
        c[:, b] = c[:, a]
    assert torch.equal(g.cpu(), c), "pages"


@pytest.mark.parametrize("state", ["empty", "full", "front", "back"])
def test_page_compact_extremes(hc, state):
    pages = 9000
    refs = torch.zeros(pages, dtype=torch.int32)
    if state == "full":
        refs += 1
    if state == "front":
        refs[: pages // 2] = 3
    if state == "back":
        refs[pages - pages // 2:] = 2
    table, lens = torch.zeros((0, 4), dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    c = pool(1, 1, pages, 1, 1, 8)
    g = c.cuda()
    t, k, remap, live = hc.page_compact(g, table.cuda(), lens.cuda(), refs.cuda())
    _, wk, wr, wl, moves = R.Pages(table, lens, refs, 1).compact()
    assert t.shape == (0, 4) and k.tolist() == wk and remap.tolist() == wr and live.tolist() == [wl]
    for a, b in moves:
        c[:, b] = c[:, a]
    assert torch.equal(g.cpu(), c)


def test_wrong_tensors_are_refused(hc):
    b = Batch(5, [(1, 30), (1, 9)], 4, 2, 64, 16, BF16, cu=False)
    q, k, v, t, n = b.q.cuda(), b.k.cuda(), b.v.cuda(), b.table.cuda(), b.lens.cuda()
    f, _ = hc.rotary_frequencies(64)
    at = torch.zeros(2, dtype=torch.int64, device="cuda")
    bad = [
        lambda: hc.paged_attention(b.q, k, v, t, n), lambda: hc.paged_attention(q.float(), k, v, t, n),
        lambda: hc.paged_attention(q, k, v[:, :8], t, n), lambda: hc.paged_attention(q, k, v, t.long(), n),
        lambda: hc.paged_attention(q, k, v, t, n[:1]), lambda: hc.paged_attention(q[:1], k, v, t, n),
        lambda: hc.paged_attention(q[:, :3], k, v, t, n), lambda: hc.paged_attention(q[..., :32], k, v, t, n),
        lambda: hc.paged_attention(q, k, v, t, n, n), lambda: hc.paged_attention(q, k, v, t.t(), n),
        lambda: hc.paged_attention(q, k, v, t, n, out=q[:1]), lambda: hc.rotary(q, at.float(), f),
        lambda: hc.rotary(q, at[:1], f), lambda: hc.rotary(q, at, f.float()), lambda: hc.rotary(q[0], at, f),
        lambda: hc.rotary_append(q, q, q, k, v, t, n, inv_freq=f), lambda: hc.page_copy(b.k, n, n),
        lambda: hc.page_copy(k.view(1, *k.shape), n, n[:1]), lambda: hc.page_copy(k.view(1, *k.shape)[:, ::2], n, n),
        lambda: hc.page_fork(k.view(1, *k.shape), t, n, n, n), lambda: hc.page_extend(t, n, n, n[:1], page_size=16),
        lambda: hc.page_extend(t, n, n, n, page_size=0), lambda: hc.page_release(t, n, n, n, page_size=16),
        lambda: hc.rotary_frequencies(3), lambda: hc.rotary_frequencies(8, scaling="no"),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(TypeError):
        hc.rotary(at.view(1, 1, 2), at[:1], f)
    for call in (lambda: hc.paged_attention(q, k, v, t, n, out=q), lambda: hc.paged_attention(q, k, v, t, n, window=-1),
                 lambda: hc.paged_attention(q, k, v, t, n, softcap=-1.0), lambda: hc.rotary(q[..., :62].clone(), at, f),
                 lambda: hc.paged_attention(q, k, v, t, n, flags=8)):
        with pytest.raises(hc.HcError):
            call()
    long = Batch(6, [(1, 3001)], 8, 2, 128, 16, BF16, cu=False)
    with pytest.raises(hc.HcError, match="workspace"):
        long.run(hc, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
