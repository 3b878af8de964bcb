"""The operators of a serving layer's paged key/value cache, as cases to be measured.

Between two hyper-connection blocks of a decoder sits an attention layer whose keys and values live in
pages of a pool. Its operators are

  rotary           rotation of query or key heads by their positions (and back, which is its gradient)
  rotary_append    the same for the new tokens of a batch, the keys and values written into their pages
  paged_attention  softmax attention of the new tokens over the pages of their sequences
  page_copy, page_fork, page_compact   the pool's upkeep: copies, beams that go on from others, defragmentation

``run`` computes them in elementary torch operations (``own`` false) or through the framework (``own`` true).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases --

def listed():
    return [
        # one user's next token: 20 heads of 128 (the 2560-wide layer), the smallest call a decode loop makes
        dict(name="append_one", op="append", dtype="bf16", seqs=1, q=1, past=699, empty=0, heads=20, kv_heads=4, dim=128,
             rot=128, interleaved=False, page=16),
        # prompts of several users arrive together: about 8000 tokens of ragged chunks, 32 query and 8 key heads
        dict(name="append_prompts", op="append", dtype="bf16", seqs=8, q=2047, past=4001, empty=0, heads=32, kv_heads=8,
             dim=128, rot=128, interleaved=False, page=64),
        # the gradient of a rotation in training: float32, pairs side by side, half of each head left as it is
        dict(name="rotate_back_f32", op="rotary", dtype="f32", tokens=4099, heads=20, dim=128, rot=64, interleaved=True,
             inverse=True, reach=131071),
        # one user's next token over a short context, the smallest attention call
        dict(name="decode_one", op="attention", dtype="bf16", seqs=1, q=1, past=699, empty=0, heads=20, kv_heads=4, dim=128,
             page=16, window=0, softcap=0.0),
        # a serving batch: 64 slots of ragged contexts, three of them empty
        dict(name="decode_batch", op="attention", dtype="bf16", seqs=64, q=1, past=8191, empty=3, heads=32, kv_heads=8,
             dim=128, page=64, window=0, softcap=0.0),
        # two users with very long contexts
        dict(name="decode_long", op="attention", dtype="f16", seqs=2, q=1, past=130001, empty=0, heads=32, kv_heads=8,
             dim=128, page=128, window=0, softcap=0.0),
        # a long prompt read in chunks: 2047 new tokens behind 28001 cached ones (the largest product here)
        dict(name="chunk_long", op="attention", dtype="bf16", seqs=1, q=2047, past=28001, empty=0, heads=32, kv_heads=8,
             dim=128, page=64, window=0, softcap=0.0),
        # continuous batching on the 1280-wide layer (20 heads of 64): single tokens and chunks mixed, sliding window,
        # capped scores, small pages
        dict(name="chunk_mixed", op="attention", dtype="f16", seqs=17, q=301, past=2501, empty=0, heads=20, kv_heads=4,
             dim=64, page=16, window=1000, softcap=30.0),
        # float32 all through, as a model is checked before it is quantised
        dict(name="chunk_f32", op="attention", dtype="f32", seqs=3, q=131, past=901, empty=0, heads=20, kv_heads=4, dim=128,
             page=16, window=0, softcap=0.0),
        # pages of a prompt copied for a second user of the pool, across 48 layers' keys and values
        dict(name="copy_prompt", op="copy", dtype="bf16", planes=96, pages=301, page=16, kv_heads=4, dim=128, seqs=1,
             tokens=1601),
        # beam search goes on from the chosen beams: a few pages copied, tables and counts rewritten
        dict(name="fork_beams", op="fork", dtype="bf16", planes=8, pages=1021, page=16, kv_heads=4, dim=128, seqs=16,
             tokens=701),
        # a fragmented pool is moved together: 24 layers' keys and values, a third of the pages live
        dict(name="compact_pool", op="compact", dtype="bf16", planes=48, pages=1501, page=16, kv_heads=8, dim=128, seqs=24,
             tokens=601),
    ]


def spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm and odd (unless it is a bound)."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) | 1))


def draw(rng):
    op = rng.choice(["append", "rotary", "decode", "decode", "chunk", "chunk", "copy", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    dim = rng.choice([64, 128, 128])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotary":
        return dict(op=op, dtype=dtype, tokens=spread(rng, 1, 8192), heads=spread(rng, 1, 33), dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5,
                    reach=spread(rng, 100, 500000))
    if op == "append":
        return dict(op=op, dtype=dtype, seqs=spread(rng, 1, 33), q=spread(rng, 1, 301), past=spread(rng, 1, 4001), empty=0,
                    heads=kv_heads * group, kv_heads=kv_heads, dim=dim, rot=rng.choice([dim, dim // 2]),
                    interleaved=rng.random() < 0.5, page=page)
    if op in ("decode", "chunk"):
        seqs = spread(rng, 1, 65 if op == "decode" else 9)
        # the longest context is one whose keys and values all sequences together keep within a few GB
        past = spread(rng, 1, min(65537, 2 ** 28 // (seqs * kv_heads * dim)))
        q = 1
        if op == "chunk":
            past, q = min(past, 16385), spread(rng, 2, 2 ** 11 - 1)
            # within the largest listed product, and in float32, where chunks are short, a part of that
            most = 1.9e9 if dtype != "f32" else 5e7
            q = max(2, min(q, int(most / (seqs * kv_heads * group * (past + q)))))
        return dict(op="attention", dtype=dtype, seqs=seqs, q=q, past=past, empty=rng.choice([0, 1]) if seqs > 2 and q == 1 else 0,
                    heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page,
                    window=rng.choice([0, 0, spread(rng, 16, 4001)]), softcap=rng.choice([0.0, 0.0, 30.0]))
    planes, seqs = 2 * spread(rng, 1, 25), spread(rng, 2, 33)
    # one sequence's share of a pool of at most 1 GB
    tokens = spread(rng, page, max(page, min(4001, 2 ** 30 // (planes * kv_heads * dim * SIZES[dtype] * 3 * seqs))))
    pages = 3 * seqs * -(-tokens // page) + 2 * seqs
    return dict(op=op, dtype=dtype, planes=planes, pages=pages, page=page, kv_heads=kv_heads, dim=dim, seqs=seqs, tokens=tokens)


def lengths(case):
    """(new tokens, tokens in the cache with them) of every sequence. They go by the case's sizes alone."""
    r = random.Random("%(seqs)d %(q)d %(past)d" % case)
    got = []
    for i in range(case["seqs"]):
        full = i == 0
        # a mixed batch: every third sequence of a batch of chunks is at its next single token
        q = case["q"] if full else 1 if i % 3 == 1 and case["seqs"] > 8 else r.randint((case["q"] + 1) // 2, case["q"])
        past = case["past"] if full else r.randint(case["past"] // 4, case["past"])
        got.append((q, past + q))
    for i in range(case["empty"]):
        got[1 + i] = (got[1 + i][0], 0)  # a slot of the batch that nobody uses
    return got


def fork_plan(case):
    """Lengths of the old sequences and the parents of the new ones."""
    r = random.Random("%(seqs)d %(tokens)d" % case)
    lens = [r.randint(max(1, case["tokens"] // 2), case["tokens"]) for _ in range(case["seqs"])]
    some = r.sample(range(case["seqs"]), max(1, case["seqs"] // 2))
    return lens, [r.choice(some) for _ in range(case["seqs"])]


# --------------------------------------------------------------------------------------------- prepare --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    def pool(*shape):
        """A pool's bytes: values of every page, those that nobody uses among them."""
        x = torch.empty(*shape, device="cuda", dtype=dt)
        return x.normal_(generator=g)

    def ints(v, d=torch.int32):
        return torch.tensor(v, dtype=d, device="cuda")

    s = dict(case)
    if case["op"] == "rotary":
        s["x"] = normal(case["tokens"], case["heads"], case["dim"])
        s["positions"] = ints([r.randint(0, case["reach"]) for _ in range(case["tokens"])], torch.int64)
        s.update(angles(case["rot"], case["reach"] + 1))
        return s
    if case["op"] in ("append", "attention"):
        both = lengths(case)
        order = list(range(len(both)))
        r.shuffle(order)
        both = [both[i] for i in order]
        qs, ns = [b[0] for b in both], [b[1] for b in both]
        page = case["page"]
        used = [-(-n // page) for n in ns]
        width = max(used) + 1
        total = sum(used) + 3
        ids = list(range(total))
        r.shuffle(ids)
        table = []
        for u in used:
            table.append(ids[:u] + [-1] * (width - u))
            ids = ids[u:]
        cu = [0]
        for q in qs:
            cu.append(cu[-1] + q)
        s["table"], s["lens"], s["cu"] = ints(table), ints(ns), None if case["q"] == 1 else ints(cu)
        s["tokens"], s["max_q"], s["max_kv"] = cu[-1], max(qs), max(ns)
        s["k_cache"] = pool(total, page, case["kv_heads"], case["dim"])
        s["v_cache"] = pool(total, page, case["kv_heads"], case["dim"])
        # queries as the projection leaves them, a little longer than normal, as trained ones are
        s["q"] = (1.5 * torch.randn(cu[-1], case["heads"], case["dim"], generator=g, device="cuda")).to(dt)
        if case["op"] == "append":
            # the projections' output as one matrix: keys and values are parts of its rows
            kv = normal(cu[-1], 2, case["kv_heads"], case["dim"])
            s["k"], s["v"] = kv[:, 0], kv[:, 1]
            s.update(angles(case["rot"], s["max_kv"]))
        return s
    # the pool's upkeep
    cache = pool(case["planes"], case["pages"], case["page"], case["kv_heads"], case["dim"])
    s["cache"] = cache
    page, pages, seqs = case["page"], case["pages"], case["seqs"]
    if case["op"] == "copy":
        ids = r.sample(range(pages), 2 * (pages // 3))
        s["src"], s["dst"] = ints(ids[: pages // 3]), ints(ids[pages // 3:])
        return s
    if case["op"] == "fork":
        lens, parents = fork_plan(case)
        r.shuffle(parents)
        ids = r.sample(range(pages), sum(-(-n // page) for n in lens))
        table, shared = [], []
        s["parents"] = ints(parents)
    else:
        # sequences in fours go on from one prompt, whose full pages they share
        lens = [case["tokens"]] * seqs
        table, shared = [], []
        n = -(-case["tokens"] // page)
        half = n // 2
        live = sum(half * (i % 4 == 0) + n - half for i in range(seqs))
        # a share of the live pages lies behind the place where a compact pool would end
        behind = min(live // 2, pages - live)
        ids = r.sample(range(live), live - behind) + r.sample(range(live, pages), behind)
        r.shuffle(ids)
    width = -(-case["tokens"] // page) + 2
    refs = [0] * pages
    for i, n in enumerate(lens):
        u = -(-n // page)
        k = u // 2 if case["op"] == "compact" else 0
        if i % 4 == 0:
            shared, ids = ids[:k], ids[k:]
        row = shared[:k] + ids[: u - k]
        ids = ids[u - k:]
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (width - u))
    s["table"], s["lens"], s["refs"] = ints(table), ints(lens), ints(refs)
    return s


def angles(rot, reach):
    """The frequencies of a rotation, and the table of its cosines and sines that a program without the framework keeps."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(reach, dtype=torch.float64, device="cuda")[:, None] * f
    return dict(freq=f, cos=a.cos().float(), sin=a.sin().float())


# ------------------------------------------------------------------------------------------------- run --

def run(s):
    return run_own(s) if own else PLAIN[s["op"]](s)


def run_own(s):
    import hyper_connection_rank_gb300 as hc
    if s["op"] == "rotary":
        return hc.rotary(s["x"], s["positions"], s["freq"], interleaved=s["interleaved"], inverse=s["inverse"])
    if s["op"] == "append":
        q = hc.rotary_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                             inv_freq=s["freq"], interleaved=s["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    if s["op"] == "attention":
        return hc.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], window=s["window"],
                                  softcap=s["softcap"], max_q=s["max_q"], max_kv=s["max_kv"])
    if s["op"] == "copy":
        return hc.page_copy(s["cache"], s["src"], s["dst"])
    if s["op"] == "fork":
        return hc.page_fork(s["cache"], s["table"], s["lens"], s["refs"], s["parents"]) + (s["cache"],)
    return hc.page_compact(s["cache"], s["table"], s["lens"], s["refs"]) + (s["cache"],)


def rotate(x, cos, sin, s, inverse=False):
    """x (tokens, heads, dim) in float32, its first `rot` features rotated in pairs."""
    x = x.float()
    rot = s["rot"]
    cos, sin = cos[:, None], sin[:, None]
    sin = -sin if inverse else sin
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def where(s):
    """For every new token its sequence and its position there."""
    lens = s["lens"].long()
    t = torch.arange(s["tokens"], device="cuda")
    if s["cu"] is None:
        return t, lens - 1
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, lens[seq] - (cu[seq + 1] - t)


def plain_rotary(s):
    at = s["positions"]
    return rotate(s["x"], s["cos"][at], s["sin"][at], s, s["inverse"]).to(s["x"].dtype)


def plain_append(s):
    seq, at = where(s)
    cos, sin = s["cos"][at], s["sin"][at]
    slot = s["table"][seq, at // s["page"]].long() * s["page"] + at % s["page"]
    s["k_cache"].flatten(0, 1)[slot] = rotate(s["k"], cos, sin, s).to(s["k"].dtype)
    s["v_cache"].flatten(0, 1)[slot] = s["v"]
    return rotate(s["q"], cos, sin, s).to(s["q"].dtype), s["k_cache"], s["v_cache"]


def plain_attention(s):
    """All sequences padded to the longest, one product for the scores and one for the values."""
    seqs, heads, kv, dim = s["lens"].numel(), s["heads"], s["kv_heads"], s["dim"]
    seq, at = where(s)
    nq, n = s["max_q"], s["max_kv"]
    first = torch.arange(seqs, device="cuda") if s["cu"] is None else s["cu"][:-1].long()
    row = torch.arange(s["tokens"], device="cuda") - first[seq]
    q = torch.zeros(seqs, nq, heads, dim, device="cuda")
    q[seq, row] = s["q"].float()
    place = torch.full((seqs, nq), -1, device="cuda")
    place[seq, row] = at
    q = q.view(seqs, nq, kv, heads // kv, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, dim)
    pages = s["table"][:, : -(-n // s["page"])].clamp(min=0).long()
    k = s["k_cache"][pages].flatten(1, 2)[:, :n].float().transpose(1, 2)
    v = s["v_cache"][pages].flatten(1, 2)[:, :n].float().transpose(1, 2)
    score = (q @ k.transpose(2, 3)) * (1 / math.sqrt(dim))
    if s["softcap"]:
        score = s["softcap"] * torch.tanh(score / s["softcap"])
    j = torch.arange(n, device="cuda")
    seen = (j <= place[:, :, None]) & (j < s["lens"][:, None, None])
    if s["window"]:
        seen &= j > place[:, :, None] - s["window"]
    score = score.view(seqs, kv, heads // kv, nq, n).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(seqs, kv, -1, n) @ v).view(seqs, kv, heads // kv, nq, dim) / torch.where(total > 0, total, 1.0)
    return out.permute(0, 3, 1, 2, 4).reshape(seqs, nq, heads, dim)[seq, row].to(s["q"].dtype)


def plain_copy(s):
    s["cache"][:, s["dst"].long()] = s["cache"][:, s["src"].long()]
    return s["cache"]


def plain_fork(s):
    """Full pages are shared; of a page that is not full the first child keeps the original, the others get copies."""
    table, refs, parents, page = s["table"].long(), s["refs"], s["parents"].long(), s["page"]
    used = lambda n: torch.arange(table.shape[1], device="cuda") < (n[:, None] + page - 1) // page  # noqa: E731
    lens = torch.where(parents >= 0, s["lens"][parents.clamp(min=0)], 0)
    new = torch.where(used(lens), table[parents.clamp(min=0)], -1)
    earlier = (parents[:, None] == parents[None]).tril(-1).any(1)
    need = earlier & (lens % page != 0)
    last = ((lens + page - 1) // page - 1).long()
    src = new[need, last[need]]
    new[need, last[need]] = -1
    refs = refs - torch.bincount(table[used(s["lens"])], minlength=refs.numel())
    refs = refs + torch.bincount(new[new >= 0], minlength=refs.numel())
    free = (refs <= 0).nonzero()[:, 0]
    dst = free[: src.numel()]
    got = need.nonzero()[: dst.numel(), 0]
    new[got, last[got]] = dst
    refs[dst] = 1
    s["cache"][:, dst] = s["cache"][:, src[: dst.numel()]]
    return new.int(), lens.int(), refs.int(), torch.full((1,), src.numel() - dst.numel(), dtype=torch.int32, device="cuda"), s["cache"]


def plain_compact(s):
    """The live pages behind the place where a compact pool ends move into the holes before it, in order."""
    table, refs, page = s["table"].long(), s["refs"], s["page"]
    live = refs > 0
    i = torch.arange(refs.numel(), device="cuda")
    end = live.sum()
    src, dst = (live & (i >= end)).nonzero()[:, 0], (~live & (i < end)).nonzero()[:, 0]
    to = torch.where(live, i, -1)
    to[src] = dst
    used = torch.arange(table.shape[1], device="cuda") < (s["lens"][:, None] + page - 1) // page
    new = torch.where(used, to[table.clamp(min=0)], -1)
    count = torch.zeros_like(refs)
    count[to[live]] = refs[live]
    s["cache"][:, dst] = s["cache"][:, src]
    return new.int(), count, to.int(), end.int().view(1), s["cache"]


PLAIN = dict(rotary=plain_rotary, append=plain_append, attention=plain_attention, copy=plain_copy, fork=plain_fork,
             compact=plain_compact)


# ------------------------------------------------------------------------------------------------ work --

def work(case):
    size = SIZES[case["dtype"]]
    if case["op"] == "rotary":
        n = case["tokens"] * case["heads"]
        return dict(bytes=2 * n * case["dim"] * size + 8 * case["tokens"] + 4 * case["rot"], flops=3 * n * case["rot"])
    if case["op"] == "append":
        tokens = sum(q for q, _ in lengths(case))
        n = tokens * (case["heads"] + 2 * case["kv_heads"])
        return dict(bytes=2 * n * case["dim"] * size + 8 * case["seqs"] + 4 * case["rot"],
                    flops=3 * tokens * (case["heads"] + case["kv_heads"]) * case["rot"])
    if case["op"] == "attention":
        read = pairs = tokens = 0
        for q, n in lengths(case):
            tokens += q
            w = case["window"] or n + 1
            lo = max(0, n - q + 1 - w)  # the first key that the first new token sees
            read += max(0, n - lo)
            pairs += sum(min(n - q + 1 + i, w) for i in range(q) if n - q + 1 + i > 0)
        return dict(bytes=2 * read * case["kv_heads"] * case["dim"] * size + 2 * tokens * case["heads"] * case["dim"] * size
                    + 4 * read // case["page"] + 4 * case["seqs"], flops=4 * case["dim"] * case["heads"] * pairs)
    one = 2 * case["planes"] * case["page"] * case["kv_heads"] * case["dim"] * size  # a page read and written
    if case["op"] == "copy":
        return dict(bytes=case["pages"] // 3 * (one + 8), flops=0)
    u = -(-case["tokens"] // case["page"])
    meta = 2 * 4 * (case["seqs"] * u + case["pages"])
    if case["op"] == "fork":
        lens, parents = fork_plan(case)
        copies = sum((parents.count(p) - 1) * (lens[p] % case["page"] != 0) for p in set(parents))
        return dict(bytes=copies * one + meta, flops=0)
    live = sum(u // 2 * (i % 4 == 0) + u - u // 2 for i in range(case["seqs"]))
    return dict(bytes=min(live // 2, case["pages"] - live) * one + meta + 4 * case["pages"], flops=0)


# ----------------------------------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return turn(s["x"], s["positions"].double()[:, None] * s["freq"], s, -1.0 if s["inverse"] else 1.0)
    if case["op"] in ("append", "attention"):
        lens = s["lens"].tolist()
        cu = list(range(len(lens) + 1)) if s["cu"] is None else s["cu"].tolist()
        table = s["table"].tolist()
    if case["op"] == "append":
        at = torch.cat([torch.arange(n - (cu[i + 1] - cu[i]), n) for i, n in enumerate(lens)]).cuda()
        angle = at.double()[:, None] * s["freq"]
        k, v = turn(s["k"], angle, s, 1.0), s["v"].double()
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        for i in range(len(lens)):
            p = at[cu[i]: cu[i + 1]]
            page = s["table"][i, (p // s["page"])].long()
            k_cache[page, p % s["page"]] = k[cu[i]: cu[i + 1]]
            v_cache[page, p % s["page"]] = v[cu[i]: cu[i + 1]]
        return turn(s["q"], angle, s, 1.0), k_cache, v_cache
    if case["op"] == "attention":
        group = s["heads"] // s["kv_heads"]
        out = torch.zeros(s["tokens"], s["heads"], s["dim"], dtype=torch.float64, device="cuda")
        for i, n in enumerate(lens):
            if n == 0:
                continue
            pages = torch.tensor(table[i][: -(-n // s["page"])], device="cuda")
            k = s["k_cache"][pages].flatten(0, 1)[:n].double()
            v = s["v_cache"][pages].flatten(0, 1)[:n].double()
            for b in range(cu[i], cu[i + 1], 512):  # so many tokens at a time that their scores fit
                e = min(b + 512, cu[i + 1])
                at = torch.arange(n - (cu[i + 1] - b), n - (cu[i + 1] - e), device="cuda")[:, None]
                j = torch.arange(n, device="cuda")
                hidden = j > at
                if s["window"]:
                    hidden |= j <= at - s["window"]
                for h in range(s["heads"]):
                    z = s["q"][b:e, h].double() @ k[:, h // group].T / math.sqrt(s["dim"])
                    if s["softcap"]:
                        z = torch.tanh(z / s["softcap"]) * s["softcap"]
                    out[b:e, h] = torch.softmax(z.masked_fill(hidden, -math.inf), 1) @ v[:, h // group]
        return out
    # whole pages and whole numbers: a pool moves page by page, on lists
    cache = s["cache"]
    if case["op"] == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            cache[:, b] = cache[:, a]
        return cache
    page, refs = s["page"], s["refs"].tolist()
    rows = [row[: -(-n // page)] for row, n in zip(s["table"].tolist(), s["lens"].tolist())]
    width = s["table"].shape[1]
    as_table = lambda rows: torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32)  # noqa: E731
    if case["op"] == "fork":
        new, lens, copies, seen = [], [], [], set()
        for i, p in enumerate(s["parents"].tolist()):
            lens.append(int(s["lens"][p]))
            new.append(list(rows[p]))
            if p in seen and lens[-1] % page:
                copies.append((i, new[-1][-1]))
                new[-1][-1] = None
            seen.add(p)
        for row in rows:
            for p in row:
                refs[p] -= 1
        for row in new:
            for p in row:
                if p is not None:
                    refs[p] += 1
        free = [p for p, c in enumerate(refs) if c <= 0]
        missing = max(0, len(copies) - len(free))
        for (i, a), b in zip(copies, free):
            cache[:, b] = cache[:, a]
            new[i][-1] = b
            refs[b] = 1
        new = [[-1 if p is None else p for p in row] for row in new]
        return as_table(new), torch.tensor(lens, dtype=torch.int32), torch.tensor(refs, dtype=torch.int32), \
            torch.tensor([missing], dtype=torch.int32), cache
    end = sum(c > 0 for c in refs)
    holes = [p for p, c in enumerate(refs) if c <= 0 and p < end]
    to = [p if c > 0 else -1 for p, c in enumerate(refs)]
    for a, b in zip([p for p, c in enumerate(refs) if c > 0 and p >= end], holes):
        cache[:, b] = cache[:, a]
        to[a] = b
    count = [0] * len(refs)
    for p, c in enumerate(refs):
        if c > 0:
            count[to[p]] = c
    return as_table([[to[p] for p in row] for row in rows]), torch.tensor(count, dtype=torch.int32), \
        torch.tensor(to, dtype=torch.int32), torch.tensor([end], dtype=torch.int32), cache


def turn(x, angle, s, sign):
    """x in 64 bits with its pairs turned by the angle, as a product of complex numbers."""
    x = x.double()
    rot = s["rot"]
    head = x[..., :rot]
    pair = head.unflatten(-1, (rot // 2, 2)) if s["interleaved"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(angle), sign * angle)[:, None]
    pair = torch.view_as_real(z)
    pair = pair if s["interleaved"] else pair.transpose(-1, -2)
    return torch.cat((pair.flatten(-2), x[..., rot:]), -1)
