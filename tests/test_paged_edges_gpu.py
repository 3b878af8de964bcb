"""The paged-cache operators at the ends of their ranges, on the GPU: caps of every size, bytes that nobody sees, streams,
bounds that end early, values that are not finite."""
import math
import random

import pytest
import torch

import _paged_ref as R
from test_paged_gpu import BF16, F16, F32, Batch, hc, ids, rnd, within  # noqa: F401 (hc is a fixture)

pytestmark = pytest.mark.gpu

V = 2.0 ** -24


# ---------------------------------------------------------------------------------------------- caps --

def one_feature(dtype, heads, kv_heads, dim, tokens, reach, seed):
    """Queries and keys of one feature each, so that a score is one exact product, and all keys of a head alike: a token that
    sees n of them has lse = s + log(n). Scores from 2^-9 to `reach` of either sign."""
    r = random.Random(seed)
    q = torch.zeros(tokens, heads, dim, dtype=dtype)
    for t in range(tokens):
        for h in range(heads):
            q[t, h, 7] = r.choice([-1, 1]) * 2.0 ** r.uniform(-6, math.log2(reach)) if (t + h) % 5 else 0.0
    k = torch.zeros(kv_heads, dim, dtype=dtype)
    k[:, 7] = torch.tensor([1.0 + 0.25 * (i % 3) for i in range(kv_heads)])
    return q, k


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("cap", [1e-3, 5.0, 50.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e30])
@pytest.mark.parametrize("both", [[(1, 1), (1, 300)], [(20, 20), (40, 300)]], ids=["single", "chunk"])
def test_caps_of_every_size(hc, dtype, dim, cap, both):
    """c tanh(s / c) to a few units of its own size, whatever c is. Bound of lse = F(s) + log(n): the cap's argument, the cap and
    its place in a base-2 exponent round some 16 times in all (16 v |F|), the sum of weights and its logarithm as in _paged_ref."""
    heads, kv_heads, page, scale = 6, 2, 16, 0.125
    b = Batch(3, both, heads, kv_heads, dim, page, dtype, cu=both[0][0] > 1)
    b.q, k = one_feature(dtype, heads, kv_heads, dim, b.tokens, 2.0 ** 14, 5)
    b.k[b.held] = k
    out, lse = b.run(hc, scale=scale, softcap=cap)
    s = b.q.double()[:, :, 7] * k[:, 7].double().repeat_interleave(heads // kv_heads) * scale
    f = cap * torch.tanh(s / cap)
    n = torch.tensor([m - nq + i + 1 for nq, m in both for i in range(nq)], dtype=torch.float64)[:, None]
    want = f + n.log()
    within(lse, want, 16 * V * f.abs() + (n + 16) * V + 2.0 ** -21 + 2 * V * want.abs(), "lse")
    # all weights are alike: the values' mean
    mean, _, tol, _ = R.attention(torch.zeros_like(b.q), b.k, b.v, b.table, b.lens, b.cu)
    within(out, mean, tol, "out")


def cap_bounds(b, out, lse, scale):
    """Bounds as in _paged_ref, with 16 v |s| for the cap in place of 4 v c, and coarser: |s| <= scale |q| |k| for every score,
    and the values' largest for their weighted mean."""
    n, dim, u = max(m for _, m in b.both), b.q.shape[2], R.U[b.dtype]
    big = scale * b.q.double().norm(dim=-1) * b.k[b.held].double().norm(dim=-1).max()
    v = b.v[b.held].double().abs()
    e = (dim + 8 + 16 + 4) * V * big + 2.0 ** -21
    tol = (2 * e + (n + 16) * V)[..., None] * v.max() + u * out.abs()
    if b.dtype != F32:
        tol = tol + u * v.max()
    if b.dtype == F16:
        tol = tol + 2.0 ** -25 * (n * v.max() + 1)
    return tol, e + (n + 16) * V + 2 * V * lse.abs()


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("cap", [20.0, 50.0, 1e3, 1e6, 1e30])
@pytest.mark.parametrize("scale", [0.1, 1.0])
def test_large_caps_over_ordinary_scores(hc, dtype, dim, cap, scale):
    for both in ([(1, 700), (1, 33)], [(70, 700), (1, 33)]):
        b = Batch(211, both, 8, 2, dim, 16, dtype, cu=both[0][0] > 1)
        out, lse, _, _ = R.attention(b.q, b.k, b.v, b.table, b.lens, b.cu, scale=scale, softcap=cap)
        tol, ltol = cap_bounds(b, out, lse, scale)
        got, glse = b.run(hc, scale=scale, softcap=cap)
        within(got, out, tol, "out")
        within(glse, lse, ltol, "lse")


# ------------------------------------------------------------------------------------- what is not seen --

@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("cap", [0.0, 8.0, 30.0])
@pytest.mark.parametrize("both", [[(1, 700), (1, 37)], [(5, 300), (2, 37)], [(140, 700), (9, 37)]], ids=["single", "few", "chunk"])
def test_bits_do_not_follow_what_is_not_seen(hc, dtype, dim, cap, both):
    """The same bits whatever lies in the rest of a sequence's last page, in the pool's other pages, in keys that the window has
    left, and, for a token, in the keys and values of those after it."""
    b = Batch(31, both, 4, 2, dim, 16, dtype, cu=both[0][0] > 1, stale=0.0)
    kw = dict(softcap=cap, scale=0.3, window=100)
    base, lse = b.run(hc, **kw)
    for stale in (0.01, -300.0, 6e4, math.inf, -math.inf, math.nan):
        b.k[~b.held] = stale
        b.v[~b.held] = stale
        got, glse = b.run(hc, **kw)
        assert torch.equal(got, base) and torch.equal(glse, lse), f"stale {stale}"
    places = {(s, j): (int(b.table[s, j // 16]), j % 16) for s, (_, n) in enumerate(both) for j in range(n)}
    for huge in (-300.0, 6e4, math.inf):
        keep = b.k.clone(), b.v.clone()
        for (s, j), place in places.items():
            if j <= both[s][1] - both[s][0] - 100:  # no new token sees it
                b.k[place], b.v[place] = huge, -huge
        got, glse = b.run(hc, **kw)
        assert torch.equal(got, base) and torch.equal(glse, lse), f"left keys {huge}"
        b.k, b.v = keep
    for last in (1, 3):
        if last >= both[0][0]:
            continue
        for key, value in ((3.0, 3.0), (-300.0, 300.0), (6e4, 6e4), (math.nan, math.inf)):
            keep = b.k.clone(), b.v.clone()
            n, nq = both[0][1], both[0][0]
            for j in range(n - last, n):
                b.k[places[0, j]], b.v[places[0, j]] = key, value
            got, glse = b.run(hc, **kw)
            seen = [t for t in range(b.tokens) if not nq - last <= t < nq]
            assert torch.equal(got[seen], base[seen]) and torch.equal(glse[seen], lse[seen]), f"later key {key}"
            b.k, b.v = keep


# -------------------------------------------------------------------------------------------- streams --

def calls_with_streams(hc):
    """Every entry point that takes a stream: (what, call(stream=...)), each giving a tuple of tensors. No call changes its
    inputs in a way that a second one would see."""
    b = Batch(61, [(40, 300), (1, 35)], 8, 2, 128, 16, BF16, stale=0.0)
    f, _ = hc.rotary_frequencies(128)
    q, k, v, table, lens, cu = (x.cuda() for x in (b.q, b.k, b.v, b.table, b.lens, b.cu))
    kv = rnd(5, b.tokens, 2, 128, dtype=BF16).cuda()
    kc, vc = k.clone(), v.clone()
    at = torch.arange(b.tokens, device="cuda")
    pool = torch.stack((k, v))
    refs = torch.zeros(k.shape[0], dtype=torch.int32)
    for row, (_, n) in zip(b.table, b.both):
        refs[row[: -(-n // 16)].long()] += 1
    refs = refs.cuda()
    parents = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    one = torch.ones(2, dtype=torch.int32, device="cuda")
    ids_ = torch.tensor([int(b.table[0, 0])], dtype=torch.int32, device="cuda")
    free = (refs == 0).nonzero()[:1, 0].int()
    tup = lambda x: x if isinstance(x, tuple) else (x,)  # noqa: E731
    rest = (table, lens, cu)
    return [
        ("rotary", lambda **kw: tup(hc.rotary(q, at, f, **kw))),
        ("rotary_append", lambda **kw: tup(hc.rotary_append(q, kv, kv, kc, vc, *rest, inv_freq=f, **kw)) + (kc, vc)),
        ("paged_attention", lambda **kw: hc.paged_attention(q, k, v, *rest, return_lse=True, **kw)),
        ("page_copy", lambda **kw: tup(hc.page_copy(pool, ids_, free, **kw))),
        ("page_fork", lambda **kw: hc.page_fork(pool, table, lens, refs, parents, **kw)),
        ("page_extend", lambda **kw: hc.page_extend(table, lens, refs, one, page_size=16, **kw)),
        ("page_release", lambda **kw: hc.page_release(table, lens, refs, one.byte(), page_size=16, **kw)),
        ("page_compact", lambda **kw: hc.page_compact(pool, table, lens, refs, **kw)),
    ]


def test_other_streams_do_not_take_memory_that_is_still_in_use(hc):
    """Blocks freed on the current stream, whose kernels there have yet to write them, must not hold another stream's results
    or workspace: the current stream is kept busy, and then fills every block that the call might have been handed."""
    for what, call in calls_with_streams(hc):
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        torch.cuda._sleep(200_000_000)  # a tenth of a second
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (4, 64, 500, 2000, 60000, 10 ** 6, 5 * 10 ** 6, 10 ** 8)
                  for _ in range(8)]
        for x in blocks:
            x.fill_(255)
        del blocks, x
        got = call(stream=side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), what


def test_results_of_another_stream_are_not_handed_out_too_early(hc):
    """The caller may free a result on its own stream while that one's kernels still read it."""
    for what, call in calls_with_streams(hc):
        if what == "page_copy":
            continue  # (gives back its input)
        want = call()[0].clone()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(200_000_000)
        kept = got[0].clone()
        del got
        for _ in range(4):
            call(stream=side)
            with torch.cuda.stream(side):
                junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (64, 500, 2000, 60000, 10 ** 6)]
        torch.cuda.synchronize()
        assert torch.equal(kept, want), what
        del junk


# -------------------------------------------------------------------------------------------- devices --

class Elsewhere(torch.Tensor):
    """A tensor that says it lies on another GPU."""

    def get_device(self):
        return 1


def test_tensors_of_different_devices_are_refused(hc):
    b = Batch(61, [(40, 300), (1, 35)], 8, 2, 128, 16, BF16, stale=0.0)
    f, _ = hc.rotary_frequencies(128)
    q, k, v, table, lens, cu = (x.cuda() for x in (b.q, b.k, b.v, b.table, b.lens, b.cu))
    kv = rnd(5, b.tokens, 2, 128, dtype=BF16).cuda()
    at = torch.arange(b.tokens, device="cuda")
    pool = torch.stack((k, v))
    refs = torch.ones(k.shape[0], dtype=torch.int32, device="cuda")
    one = torch.ones(2, dtype=torch.int32, device="cuda")
    ids_ = torch.tensor([0], dtype=torch.int32, device="cuda")
    work = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    calls = [
        (lambda a: hc.rotary(a[0], a[1], a[2], out=a[3]), [q, at, f, torch.empty_like(q)]),
        (lambda a: hc.rotary_append(*a[:8], inv_freq=a[8], out=a[9]), [q, kv, kv.clone(), k, v, table, lens, cu, f, q.clone()]),
        (lambda a: hc.paged_attention(*a[:6], out=a[6], workspace=a[7]), [q, k, v, table, lens, cu, q.clone(), work]),
        (lambda a: hc.paged_attention_workspace_size(*a), [q, k, v, table, lens, cu]),
        (lambda a: hc.page_copy(*a), [pool, ids_, ids_ + 1]),
        (lambda a: hc.page_fork(*a), [pool, table, lens, refs, one]),
        (lambda a: hc.page_extend(*a, page_size=16), [table, lens, refs, one]),
        (lambda a: hc.page_release(*a, page_size=16), [table, lens, refs, one.byte()]),
        (lambda a: hc.page_compact(*a), [pool, table, lens, refs]),
    ]
    for n, (call, args) in enumerate(calls):
        call(args)
        for i in range(len(args)):
            bad = [t.as_subclass(Elsewhere) if j == i else t for j, t in enumerate(args)]
            with pytest.raises(ValueError):
                call(bad)
                pytest.fail(f"call {n}: tensor {i} was taken")


def test_a_stream_of_another_device_is_refused(hc):
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0
    at = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        hc.rotary(torch.zeros(2, 1, 8, device="cuda"), at, hc.rotary_frequencies(8)[0], stream=Stream())


def test_tensors_of_another_device_than_the_current_one(hc, monkeypatch):
    """The call makes the tensors' device the current one (here, where there is but one, the current one is said to be another)."""
    from hyper_connection_rank_gb300 import _paged
    entered = []
    real = torch.cuda.device

    def device(index):
        entered.append(index)
        return real(index)
    for what, call in calls_with_streams(hc):
        want = [t.clone() for t in call()]
        monkeypatch.setattr(_paged, "_current_device", lambda: 3)
        monkeypatch.setattr(torch.cuda, "device", device)
        got = call()
        monkeypatch.undo()
        assert entered and set(entered) == {0}, what
        entered.clear()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), what


# ------------------------------------------------------------------------- rows that no sequence has --

@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pad", [(0, 5), (0, 300), (3, 0), (4, 70)], ids=str)
def test_append_writes_nothing_for_rows_past_the_bounds(hc, dtype, interleaved, pad):
    """cu_q that begins past the first row or ends before the last (a buffer of a fixed size): those rows go nowhere, and the
    others go where they would without them."""
    f, _ = hc.rotary_frequencies(64)
    front, back = pad
    b = Batch(3, [(2, 40), (7, 47), (3, 160)], 2, 1, 64, 16, dtype, stale=None)
    b.table = b.table[:, :10].contiguous()  # the last sequence fills its row: a place further on is past the table
    k, v = (rnd(s, front + b.tokens + back, 1, 64, dtype=dtype).cuda() for s in (1, 2))
    q = rnd(4, front + b.tokens + back, 2, 64, dtype=dtype).cuda()
    rest = (b.table.cuda(), b.lens.cuda())
    want = [b.k.cuda(), b.v.cuda()]
    inner = slice(front, front + b.tokens)
    wq = hc.rotary_append(q[inner], k[inner], v[inner], *want, *rest, b.cu.cuda(), inv_freq=f, interleaved=interleaved)
    got = [b.k.cuda(), b.v.cuda()]
    gq = hc.rotary_append(q, k, v, *got, *rest, (b.cu + front).cuda(), inv_freq=f, interleaved=interleaved)
    assert torch.equal(gq[inner], wq)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool(torch.isfinite(gq.float()).all())
    # bounds that leave no row to any sequence
    none = [b.k.cuda(), b.v.cuda()]
    hc.rotary_append(q, k, v, *none, *rest, torch.zeros_like(b.cu).cuda(), inv_freq=f, interleaved=interleaved)
    assert torch.equal(none[0].cpu(), b.k) and torch.equal(none[1].cpu(), b.v)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("both", [[(1, 700), (2, 30)], [(5, 60), (1, 300)], [(130, 700), (1, 90), (17, 40)]], ids=["few", "some", "chunk"])
@pytest.mark.parametrize("max_q", [None, 1])
def test_attention_gives_zeros_for_rows_past_the_bounds(hc, dtype, dim, both, max_q):
    for front, back in ((0, 1), (0, 333), (2, 0), (150, 40)):
        b = Batch(47, both, 4, 2, dim, 16, dtype)
        want, lse, tol, ltol = R.attention(b.q, b.k, b.v, b.table, b.lens, b.cu)
        n = front + b.tokens + back
        q = torch.full((n, 4, dim), 1.0, dtype=dtype, device="cuda")
        inner = slice(front, front + b.tokens)
        q[inner] = b.q.cuda()
        out = torch.full((n, 4, dim), 7.0, dtype=dtype, device="cuda")
        rest = (b.k.cuda(), b.v.cuda(), b.table.cuda(), b.lens.cuda())
        got, glse = hc.paged_attention(q, *rest, (b.cu + front).cuda(), max_q=max_q, return_lse=True, out=out)
        within(got[inner], want, tol, "out")
        within(glse[inner], lse, ltol, "lse")
        for rows in (slice(0, front), slice(n - back, n)):
            assert bool((got[rows] == 0).all()) and bool((glse[rows] == -math.inf).all()), (front, back)
        got, glse = hc.paged_attention(q, *rest, torch.zeros_like(b.cu).cuda(), max_q=max_q, return_lse=True, out=out)
        assert bool((got == 0).all()) and bool((glse == -math.inf).all())


# ------------------------------------------------------------------------------------------- workspaces --

@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("scale", [None, -0.2, 0.0, 1e-6])
@pytest.mark.parametrize("both", [[(1, 3001)], [(500, 4000), (1, 90)]], ids=["single", "chunk"])
def test_a_workspace_of_the_size_asked_for_suffices(hc, dtype, scale, both):
    b = Batch(37, both, 8, 2, 128, 16, dtype, cu=both[0][0] > 1)
    t = [b.cuda(x) for x in (b.q, b.k, b.v, b.table, b.lens, b.cu)]
    for kw in ({}, dict(window=500), dict(max_q=500, max_kv=4000), dict(flags=hc.HC_FLAG_FORCE_GENERAL)):
        n = hc.paged_attention_workspace_size(*t, scale=scale, **kw)
        work = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")
        got = hc.paged_attention(*t, scale=scale, workspace=work, **kw)
        assert torch.equal(got, hc.paged_attention(*t, scale=scale, **kw))


# ------------------------------------------------------------------------------ values that are not finite --

@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim,page,flags", [(64, 16, 0), (128, 32, 0), (128, 16, 2)])
@pytest.mark.parametrize("window", [0, 40, 200])
def test_many_unseen_values_may_be_anything(hc, dtype, dim, page, flags, window):
    """As many infinities and NaN as a chunk has tokens, one feature each: they reach those features of the tokens that see them,
    and nothing else. With a window, the first tokens still see some that the others have left."""
    for both in ([(150, 333)], [(1, 9), (290, 300), (5, 60)]):
        b = Batch(79, both, 4, 2, dim, page, dtype)
        s = max(range(len(both)), key=lambda i: both[i][0])
        n = both[s][1]
        for i, j in enumerate(range(n - both[s][0] - 60 if n > 320 else 5, n, 3)):
            place = (int(b.table[s, j // page]), j % page)
            b.v[place][i % 2, (11 * i + 3) % dim] = [math.inf, math.nan, -math.inf, math.inf][i % 4]
        out, lse, tol, ltol = R.attention(b.q, b.k, b.v, b.table, b.lens, b.cu, window=window, scale=0.05)
        got, glse = b.run(hc, window=window, flags=flags, scale=0.05)
        within(got, out, tol, "out")
        within(glse, lse, ltol, "lse")


# ---------------------------------------------------------------------------------------------- pages --

@pytest.mark.parametrize("page,old", [(2 ** 30, 2 ** 31 - 5), (2 ** 30, 2 ** 30), (2 ** 29 + 1, 2 ** 31 - 1), (2 ** 31 - 1, 7)])
def test_extend_ends_at_the_longest_length(hc, page, old):
    used = -(-old // page)
    table = torch.full((2, 6), -1, dtype=torch.int32)
    table[0, :used] = torch.arange(used)
    refs = torch.zeros(9, dtype=torch.int32)
    refs[:used] = 1
    most = 2 ** 31 - 1
    for more in (0, 100, most):
        n = min(old + more, most)
        want = -(-n // page)
        t, lens, k, missing = hc.page_extend(table.cuda(), torch.tensor([old, 0], dtype=torch.int32).cuda(), refs.cuda(),
                                             torch.tensor([more, 1], dtype=torch.int32).cuda(), page_size=page)
        assert lens.tolist() == [n, 1] and missing.tolist() == [0]
        assert t.tolist() == [list(range(want)) + [-1] * (6 - want), [want] + [-1] * 5]
        assert k.tolist() == [1] * (want + 1) + [0] * (9 - want - 1)


# -------------------------------------------------------------------------------------------- weights --

@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("both,heads,kv_heads", [([(1, 40)], 4, 1), ([(1, 700), (1, 33)], 20, 4), ([(1, 4001)], 8, 1),
                                                 ([(1, 100 + i) for i in range(60)], 8, 8), ([(5, 60), (3, 9)], 2, 2),
                                                 ([(2, 500), (1, 20)], 8, 2)], ids=lambda v: str(len(v)) if isinstance(v, list) else None)
def test_weights_of_up_to_eight_rows_keep_their_precision(hc, dtype, dim, both, heads, kv_heads):
    """Values of 1 and -1, whose weighted mean nearly vanishes, so that what rounding takes off a weight shows: with up to eight
    rows to a key head a weight goes into the product as two numbers of T, 2^-16 of it lost at most (in float16 what lies below
    2^-25 of the largest too, as _paged_ref has it), where it is rounded to T else."""
    b = Batch(89, both, heads, kv_heads, dim, 16, dtype, cu=any(q > 1 for q, _ in both))
    b.v[b.held] = b.v[b.held].sign()
    out, lse, tol, ltol = R.attention(b.q, b.k, b.v, b.table, b.lens, b.cu, scale=0.1)
    if dtype != F32:
        tol = tol - R.U[dtype] + 2.0 ** -16  # (the sum of weights times |values| is 1)
    got, glse = b.run(hc, scale=0.1, max_q=max(q for q, _ in both))
    within(got, out, tol, "out")
    within(glse, lse, ltol, "lse")
