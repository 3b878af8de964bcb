"""What a decoder of hyper-connection blocks runs besides attention when it serves, as cases to be measured.

  expert_route  scores of a router turned into experts and weights for every token
  expert_mlp    the feed-forward layer between two blocks whose weights belong to experts: the chosen experts' products
  token_sample  the next tokens, drawn from the logits with given random numbers

``run`` computes them in elementary torch operations (``own`` false) or through the framework (``own`` true).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases --

def listed():
    return [
        # one user's next token, the smallest call a decode loop makes
        dict(name="route_one", op="route", dtype="bf16", tokens=1, experts=128, k=8, scoring="softmax", bias=False, groups=1,
             top_groups=1, best=1, renormalise=True, scale=1.0, unused=0),
        # prompts of several users: 8191 tokens, scores by sigmoid with a bias for balance, four of eight groups
        dict(name="route_prompts", op="route", dtype="f32", tokens=8191, experts=256, k=8, scoring="sigmoid", bias=True, groups=8,
             top_groups=4, best=2, renormalise=True, scale=2.5, unused=0),
        # a mixed batch in a buffer of a fixed size, a number of experts that no power of two divides, weights as they are
        dict(name="route_mixed", op="route", dtype="f16", tokens=1027, experts=60, k=6, scoring="softmax", bias=True, groups=1,
             top_groups=1, best=1, renormalise=False, scale=1.0, unused=100),
        # one user's next token through the 2560-wide layer: eight experts' weights are read
        dict(name="mlp_one", op="mlp", dtype="bf16", tokens=1, experts=64, k=8, hidden=2560, inner=640, rows_out=False, unused=0),
        # a serving batch of single tokens: every expert is hit by a few
        dict(name="mlp_batch", op="mlp", dtype="bf16", tokens=61, experts=64, k=6, hidden=2560, inner=640, rows_out=False,
             unused=3),
        # prompts read in one call (the largest product here)
        dict(name="mlp_prompts", op="mlp", dtype="bf16", tokens=8191, experts=64, k=8, hidden=2560, inner=640, rows_out=False,
             unused=0),
        # few large experts on the 1280-wide layer, weights as checkpoints keep them (outputs first, inputs contiguous)
        dict(name="mlp_wide", op="mlp", dtype="f16", tokens=1301, experts=16, k=2, hidden=1280, inner=2560, rows_out=True,
             unused=0),
        # float32 all through, as a model is checked before it is quantised
        dict(name="mlp_f32", op="mlp", dtype="f32", tokens=131, experts=12, k=3, hidden=1280, inner=704, rows_out=False, unused=0),
        # one user's next token
        dict(name="sample_one", op="sample", dtype="bf16", rows=1, vocab=131072, spread=3.0, temperature=True, top_k=0, top_p=True,
             min_p=False),
        # a serving batch whose users choose for themselves
        dict(name="sample_batch", op="sample", dtype="f32", rows=64, vocab=131072, spread=3.0, temperature=True, top_k=100,
             top_p=True, min_p=True),
        # a few users of a smaller vocabulary, of an odd size
        dict(name="sample_few", op="sample", dtype="f16", rows=7, vocab=50001, spread=2.0, temperature=True, top_k=0, top_p=False,
             min_p=True),
        # many continuations of one prompt, drawn from the whole distribution
        dict(name="sample_plain", op="sample", dtype="f32", rows=256, vocab=200003, spread=2.0, temperature=False, top_k=0,
             top_p=False, min_p=False),
    ]


def spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm and odd (unless it is a bound)."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) | 1))


def draw(rng):
    op = rng.choice(["route", "mlp", "mlp", "mlp", "sample", "sample"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        each = spread(rng, 2, 257 // groups)
        top_groups = rng.randint(1, groups)
        return dict(op=op, dtype=dtype, tokens=spread(rng, 1, 8191), experts=groups * each, k=rng.randint(1, min(12, top_groups * each)),
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups, top_groups=top_groups,
                    best=rng.choice([1, 2]), renormalise=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    unused=rng.choice([0, 0, 1]))
    if op == "mlp":
        experts = spread(rng, 2, 129)
        k = rng.randint(1, min(8, experts))
        # most layers are multiples of 64 wide, some of 8, a few of nothing
        step = rng.choice([64, 64, 64, 8, 1])
        hidden, inner = max(step, spread(rng, 128, 2560) // step * step), max(step, spread(rng, 64, 2560) // step * step)
        experts = max(k, min(experts, int(6.4e8 / (3 * hidden * inner * SIZES[dtype]))))
        # within the largest listed product, and where there are no tensor cores for it, a part of that
        most = 6.4e11 if dtype != "f32" and step > 1 else 2e10
        tokens = spread(rng, 1, max(1, min(8191, int(most / (6 * k * hidden * inner)))))
        return dict(op=op, dtype=dtype, tokens=tokens, experts=experts, k=k, hidden=hidden, inner=inner,
                    rows_out=rng.random() < 0.5, unused=rng.choice([0, 0, tokens // 5]))
    rows = spread(rng, 1, 257)
    return dict(op=op, dtype=dtype, rows=rows, vocab=spread(rng, 101, min(262145, int(5.1e7 / rows))), spread=rng.choice([1.0, 2.0, 4.0]),
                temperature=rng.random() < 0.7, top_k=rng.choice([0, 0, 1, 20, 100, 1001]), top_p=rng.random() < 0.5,
                min_p=rng.random() < 0.3)


# --------------------------------------------------------------------------------------------- prepare --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(n, lo=0.0, hi=1.0):
        return torch.rand(n, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case)
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        # some experts are more popular than others; the bias works against that
        popular = normal(e)
        s["logits"] = (normal(t, e) + popular).to(dt)
        s["bias"] = -0.1 * popular if case["bias"] else None
        s["live"] = torch.tensor([t - case["unused"]], dtype=torch.int32, device="cuda") if case["unused"] else None
        return s
    if case["op"] == "mlp":
        t, e, h, i = case["tokens"], case["experts"], case["hidden"], case["inner"]

        def weight(rows, cols):
            """(experts, rows, cols), whose products with normal inputs are normal."""
            shape = (e, cols, rows) if case["rows_out"] else (e, rows, cols)
            w = torch.empty(*shape, device="cuda", dtype=dt).normal_(0.0, rows ** -0.5, generator=g)
            return w.transpose(1, 2) if case["rows_out"] else w

        s["x"] = normal(t, h).to(dt)
        s["gate_w"], s["up_w"], s["down_w"] = weight(h, i), weight(h, i), weight(i, h)
        # as a router leaves them: distinct experts, some of them popular, weights that add up to one
        best, ids = (normal(t, e) + 0.5 * normal(e)).topk(case["k"])
        s["ids"], s["weights"] = ids.int(), torch.softmax(best, -1)
        if case["unused"]:
            # rows at the end of a buffer of a fixed size that are nobody's
            s["ids"][t - case["unused"]:] = -1
            s["weights"][t - case["unused"]:] = 0.0
        return s
    n, v = case["rows"], case["vocab"]
    # a few words stand out, as they do after training
    x = normal(n, v) * case["spread"]
    x.scatter_add_(1, torch.randint(v, (n, 20), generator=g, device="cuda"), 4.0 * normal(n, 20).abs() + case["spread"])
    s["logits"] = x.to(dt)
    # random numbers come in steps of 2^-24, as most generators make them
    s["uniform"] = torch.rand(n, generator=g, device="cuda")
    s["t"] = uniform(n, 0.5, 1.2) if case["temperature"] else None
    s["k"] = torch.randint(1, case["top_k"] + 1, (n,), generator=g, device="cuda", dtype=torch.int32) if case["top_k"] else None
    s["p"] = uniform(n, 0.5, 1.0) if case["top_p"] else None
    s["m"] = uniform(n, 0.01, 0.2) if case["min_p"] else None
    return s


# ------------------------------------------------------------------------------------------------- run --

def run(s):
    return run_own(s) if own else PLAIN[s["op"]](s)


def run_own(s):
    import hyper_connection_rank_gb300 as hc
    if s["op"] == "route":
        return hc.expert_route(s["logits"], s["k"], bias=s["bias"], scoring=s["scoring"], groups=s["groups"],
                               top_groups=s["top_groups"], group_best=s["best"], renormalise=s["renormalise"], scale=s["scale"],
                               live=s["live"])
    if s["op"] == "mlp":
        return hc.expert_mlp(s["x"], s["gate_w"], s["up_w"], s["down_w"], s["ids"], s["weights"])
    return hc.token_sample(s["logits"], s["uniform"], temperature=1.0 if s["t"] is None else s["t"],
                           top_k=0 if s["k"] is None else s["k"], top_p=1.0 if s["p"] is None else s["p"],
                           min_p=0.0 if s["m"] is None else s["m"], return_logprob=True)


def plain_route(s):
    """Scores and their comparison in float64, since which of two close scores is the larger is what counts."""
    x = s["logits"].double()
    t, e = x.shape
    if s["scoring"] == "softmax":
        score = (x - x.amax(-1, keepdim=True)).exp()
        score = score / score.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + (-x).exp())
    choice = score if s["bias"] is None else score + s["bias"].double()
    if s["groups"] > 1:
        each = choice.view(t, s["groups"], -1)
        value = each.sort(dim=-1, descending=True).values[..., : s["best"]].sum(-1)
        chosen = value.sort(dim=-1, descending=True, stable=True).indices[:, : s["top_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, chosen, True)
        choice = each.masked_fill(~kept[..., None], -math.inf).view(t, e)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, : s["k"]]
    w = score.gather(1, ids)
    if s["renormalise"]:
        w = w / w.sum(-1, keepdim=True)
    w = (w * s["scale"]).float()
    ids = ids.int()
    if s["live"] is not None:
        dead = torch.arange(t, device=x.device)[:, None] >= s["live"]
        ids, w = ids.masked_fill(dead, -1), w.masked_fill(dead, 0.0)
    return ids, w


def plain_mlp(s):
    """The tokens' rows sorted by expert, one expert after the other."""
    x, ids, e = s["x"].float(), s["ids"].flatten().long(), s["experts"]
    k = s["k"]
    order = ids.argsort(stable=True)
    counts = torch.bincount(ids + 1, minlength=e + 1).tolist()
    at = counts[0]
    each = torch.zeros(ids.numel(), x.shape[1], device=x.device)
    for i, n in enumerate(counts[1:]):
        if n:
            rows = order[at: at + n]
            r = x[rows // k]
            g, u = r @ s["gate_w"][i].float(), r @ s["up_w"][i].float()
            each[rows] = (g / (1 + (-g).exp()) * u) @ s["down_w"][i].float()
        at += n
    return (each.view(-1, k, x.shape[1]) * s["weights"][..., None]).sum(1).to(s["x"].dtype)


def plain_sample(s):
    """Weights, their order and their sums in float64: a token's place in the cumulated weights is compared with a number."""
    x = s["logits"].double()
    w = x - x.amax(-1, keepdim=True)
    w = (w if s["t"] is None else w / s["t"].double()[:, None]).exp()
    if s["k"] is not None or s["p"] is not None:
        w = best_weights(x, w, s)
    if s["m"] is not None:
        w = w * (w >= s["m"].double()[:, None])
    below = w.cumsum(-1)
    total = below[:, -1:]
    token = (below > s["uniform"].double()[:, None] * total).byte().argmax(-1, keepdim=True)
    return token[:, 0].int(), (w.gather(1, token) / total).log()[:, 0].float()


def best_weights(x, w, s):
    """The weights with zeros where top_k and top_p leave a token out."""
    at = x.sort(dim=-1, descending=True, stable=True).indices
    w = w.gather(1, at)
    if s["k"] is not None:
        w = w * (torch.arange(w.shape[1], device=w.device) < s["k"][:, None])
    if s["p"] is not None:
        before = w.cumsum(-1) - w
        keep = before < s["p"].double()[:, None] * w.sum(-1, keepdim=True)
        keep[:, 0] = True
        w = w * keep
    return torch.zeros_like(w).scatter_(1, at, w)


PLAIN = dict(route=plain_route, mlp=plain_mlp, sample=plain_sample)


# ----------------------------------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return exact_route(s)
    if case["op"] == "mlp":
        return exact_mlp(s)
    return exact_sample(s)


def exact_route(s):
    x = s["logits"].double().cpu().numpy()
    bias = np.zeros(x.shape[1]) if s["bias"] is None else s["bias"].double().cpu().numpy()
    live = len(x) - s["unused"]
    ids, w = np.full((len(x), s["k"]), -1, np.int32), np.zeros((len(x), s["k"]))
    for t in range(live):
        if s["scoring"] == "softmax":
            score = np.exp(x[t] - x[t].max())
            score /= math.fsum(score)
        else:
            score = 1 / (1 + np.exp(-x[t]))
        choice = score + bias
        members = choice.reshape(s["groups"], -1)
        value = np.sort(members, 1)[:, ::-1][:, : s["best"]].sum(1)
        groups = np.argsort(-value, kind="stable")[: s["top_groups"]]
        allowed = np.repeat(np.isin(np.arange(s["groups"]), groups), members.shape[1])
        order = [e for e in np.argsort(-choice, kind="stable") if allowed[e]][: s["k"]]
        ids[t] = order
        w[t] = score[order] * s["scale"] / (score[order].sum() if s["renormalise"] else 1.0)
    return torch.from_numpy(ids), torch.from_numpy(w)


def exact_mlp(s):
    x, y = s["x"].double(), torch.zeros_like(s["x"], dtype=torch.float64)
    for e in range(s["experts"]):
        token, place = torch.nonzero(s["ids"] == e, as_tuple=True)
        if token.numel():
            row = x[token]
            up = torch.einsum("th,hi->ti", row, s["up_w"][e].double())
            gate = torch.einsum("th,hi->ti", row, s["gate_w"][e].double())
            inner = up * gate * torch.sigmoid(gate) * s["weights"][token, place].double()[:, None]
            y.index_add_(0, token, torch.einsum("ti,ih->th", inner, s["down_w"][e].double()))
    return y


def exact_sample(s):
    x = s["logits"].double().cpu().numpy()
    get = lambda name: None if s[name] is None else s[name].double().cpu().numpy()  # noqa: E731
    u, t, k, p, m = get("uniform"), get("t"), get("k"), get("p"), get("m")
    tokens, logs = np.zeros(len(x), np.int32), np.zeros(len(x))
    for r in range(len(x)):
        w = np.exp((x[r] - x[r].max()) / (1.0 if t is None else t[r]))
        if k is not None or p is not None:
            n = len(w) if k is None else min(int(k[r]), len(w))
            # only the candidates are sorted: those that reach the n-th largest value
            least = np.partition(x[r], len(w) - n)[len(w) - n]
            some = np.flatnonzero(x[r] >= least)
            some = some[np.argsort(-x[r][some], kind="stable")][:n]
            if p is not None:
                mass = np.cumsum(w[some])
                n = max(1, int(np.count_nonzero(mass - w[some] < p[r] * mass[-1])))
                some = some[:n]
            kept = np.zeros_like(w)
            kept[some] = w[some]
            w = kept
        if m is not None:
            w = np.where(w >= m[r], w, 0.0)
        total = np.cumsum(w)
        tokens[r] = np.searchsorted(total, u[r] * total[-1], side="right")
        logs[r] = math.log(w[tokens[r]] / total[-1])
    return torch.from_numpy(tokens), torch.from_numpy(logs)


# ------------------------------------------------------------------------------------------------ work --

def work(case):
    size = SIZES[case["dtype"]]
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        # a score and its comparisons: about ten operations an expert
        return dict(bytes=(t - case["unused"]) * e * size + t * k * 8 + (4 * e if case["bias"] else 0), flops=10 * t * e)
    if case["op"] == "mlp":
        t, h, i = case["tokens"] - case["unused"], case["hidden"], case["inner"]
        # every expert that some token chose is read once
        hit = case["experts"] * (1 - (1 - case["k"] / case["experts"]) ** t)
        return dict(bytes=int(3 * hit * h * i * size) + (t + case["tokens"]) * h * size + case["tokens"] * case["k"] * 8,
                    flops=6 * t * case["k"] * h * i)
    return dict(bytes=case["rows"] * (case["vocab"] * size + 12), flops=10 * case["rows"] * case["vocab"])
