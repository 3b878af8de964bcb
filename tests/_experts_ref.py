"""Plain float64 forms of routing, the experts' layer and the choice of tokens, on the CPU, and the error bounds that the tests
hold the kernels to. Written from the definitions in include/hc_experts.h and include/hc_sample.h; nothing here uses the
library.

Bounds. u is the unit roundoff of the tensors' type T (2^-24, 2^-11, 2^-8), v = 2^-24 that of float32.

Routing. The order is exact. A weight of a renormalised softmax or sigmoid is a quotient of exp(.) by a sum of top_k <= 32 of
them: exp is off by 2 ulp (4 v), its argument's rounding is carried as a second part (or is at most |x| v), a sigmoid's sum and
quotient add 2 v, the sum 32 + 8 v, the quotient and the scale 2 v: 64 v of the weight, and for arguments of sigmoids |x| v.
Over a whole softmax of n experts the sum has ceil(n / 32) + 5 roundings, and its terms' arguments round: (n / 32 + 64) v.

Experts. A sum of n products in float32 is off by at most 2 (n + 8) v S, S the sum of the products' magnitudes (the tensor
cores may cut off where they add, which is twice a rounding). With e_g and e_u those errors of the two inner products: silu's
slope is at most 1.1, and the approximate exponential and quotient are off by 2^-20, so silu(g) is off by
e_s = 1.1 e_g + 2^-20 |silu(g)| and h = silu(g) u by e_h = e_s (|u| + e_u) + |silu(g)| e_u + 2 v |h|; 16-bit kernels round it
to T: u |h| more (and in float16 2^-25). o = h down: e_o = sum e_h |down| + 2 (inner + 8) v sum |h| |down|, and where 16-bit
kernels keep it as integers of 16 bits with one exponent to sixteen, half a unit more: with the largest of them in 2^(e - 1) ..
2^e the unit is 2^(e - 15) / (1 - 2^-14), so at most 2^-15 (1 + 2^-13) of the largest (2^-126 where all are below 2^-110). The sum over the chosen: sum |w| e_o + (top_k + 2) v sum |w o|, and the store: u |y| (2^-25).

Tokens. A kernel's weight is off by 2^-37 of itself at most, so is each sum; where a comparison in the reference is closer than
2^-35 the test would not tell anything, and the reference says so. Log-probabilities: a quotient of two integers rounded to
float32 and log1p, 4 roundings on a value that moves by its own relative error: 8 v (1 + |log p|) of it, and 8 v.
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
V = 2.0 ** -24


def route(logits, top_k, bias=None, scoring="softmax", groups=1, top_groups=None, group_best=1, renormalise=True, scale=1.0,
          live=None):
    """(ids, weights, bound of the weights)"""
    x = logits.double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    n, e = x.shape
    top_groups = groups if top_groups is None else top_groups
    ids = torch.full((n, top_k), -1, dtype=torch.int32)
    weights, tol = torch.zeros(n, top_k, dtype=torch.float64), torch.zeros(n, top_k, dtype=torch.float64)
    for t in range(n if live is None else min(n, live)):
        r = x[t]
        if scoring == "sigmoid":
            s = torch.sigmoid(r)
        else:
            m = r.max()
            d = torch.where(r == m, 0.0, r - m)
            p = torch.exp(d) if m > -math.inf else torch.zeros_like(r)
            s = p / p.sum() if m > -math.inf else p
        # without a bias the scores' order is the logits'
        c = r if bias is None else s + bias.double()
        c = torch.where(torch.isnan(c), -math.inf, c)
        allowed = torch.ones(e, dtype=torch.bool)
        if top_groups < groups:
            # (scores rise with logits, so that of one score to a group the order is theirs, too, where float64 has 1 for several)
            g = (s if bias is None and group_best == 2 else c).view(groups, -1)
            value = g.sort(-1, descending=True).values[:, :group_best].sum(-1)
            best = sorted(range(groups), key=lambda i: (-value[i].item(), i))[:top_groups]
            allowed = torch.zeros(groups, dtype=torch.bool).index_fill_(0, torch.tensor(best), True).repeat_interleave(e // groups)
        order = sorted((i for i in range(e) if allowed[i]), key=lambda i: (-c[i].item(), i))[:top_k]
        ids[t] = torch.tensor(order)
        w = s[order]
        lost = 64.0 + (0.0 if renormalise else e / 32)
        if renormalise:
            # the same quotient from logits, where the scores themselves are too small for any type
            xs = r[order]
            if xs.max() == -math.inf:
                w = torch.zeros_like(xs)
            elif scoring == "softmax":
                d = torch.where(xs == xs.max(), 0.0, xs - xs.max())
                w = torch.softmax(d, -1)
            else:
                lift = max(-xs.max().item(), 0.0)
                a = torch.exp(xs.clamp(max=0) + lift) / (1 + torch.exp(-xs.abs()))
                w = a / a.sum()
        # (a sigmoid's argument is added to the lift before the exponential, at a cost of half an ulp of the sum)
        slack = 4 * r[order].abs().clamp(max=200.0) if scoring == "sigmoid" else 0.0
        weights[t] = w * scale
        tol[t] = (weights[t].abs() * (lost + slack)) * V + 1e-37
    return ids, weights, tol


def experts(x, gate, up, down, ids, w, rounded=True, stored=True):
    """(y, bound). rounded: h is rounded to T; stored: each expert's result is kept in 16 bits with an exponent."""
    dt = x.dtype
    u = U[dt] if dt != torch.float32 else 0.0
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    x = x.double()
    n, hidden = x.shape
    inner = gate.shape[2]
    y, tol = torch.zeros(n, hidden, dtype=torch.float64), torch.zeros(n, hidden, dtype=torch.float64)
    size = torch.zeros(n, hidden, dtype=torch.float64)
    k = ids.shape[1]
    for j in range(k):
        for e in range(gate.shape[0]):
            rows = torch.nonzero(ids[:, j] == e).flatten()
            if not rows.numel():
                continue
            r, g, p, d = x[rows], gate[e].double(), up[e].double(), down[e].double()
            a, b = r @ g, r @ p
            ea, eb = 2 * (hidden + 8) * V * (r.abs() @ g.abs()), 2 * (hidden + 8) * V * (r.abs() @ p.abs())
            s = a * torch.sigmoid(a)
            h = s * b
            es = 1.1 * ea + 2.0 ** -20 * s.abs()
            eh = es * (b.abs() + eb) + s.abs() * eb + 2 * V * h.abs()
            if rounded:
                eh = eh + u * (h.abs() + eh) + tiny
            o = h @ d
            eo = eh @ d.abs() + 2 * (inner + 8) * V * (h.abs() @ d.abs())
            if stored and dt != torch.float32:
                most = torch.nn.functional.pad(o.abs() + eo, (0, -hidden % 16)).view(len(rows), -1, 16).amax(-1, keepdim=True)
                eo = eo + (2.0 ** -15 * (1 + 2.0 ** -13) * most + 2.0 ** -126).expand(-1, -1, 16).flatten(1)[:, :hidden]
            c = w[rows, j].double()[:, None]
            y[rows] += c * o
            tol[rows] += c.abs() * eo
            size[rows] += (c * o).abs()
    tol += (k + 2) * V * size
    return y, tol + U[dt] * (y.abs() + tol) + tiny


def sample(logits, uniform, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(tokens, log-probabilities, bound, whether the definition decides within 2^-35) as lists over the rows."""
    rows, vocab = logits.shape

    def each(v):
        # (numbers reach the kernel as float32; 0.7 instead of its float32 would move sums by 1e-9 of themselves)
        v = v if isinstance(v, (torch.Tensor, int)) else torch.full((rows,), v)
        return v.tolist() if isinstance(v, torch.Tensor) else [v] * rows

    got = []
    for x, u, t, k, p, m in zip(logits.double(), uniform.double().tolist(), each(temperature), each(top_k), each(top_p), each(min_p)):
        x = torch.where(torch.isnan(x), -math.inf, x)
        top = x.max()
        if top == -math.inf:
            got.append((-1, -math.inf, 0.0, True))
            continue
        first = int(torch.nonzero(x == top)[0])
        if not t > 0:
            got.append((first, 0.0, 0.0, True))
            continue
        w = torch.where(x == top, 1.0, torch.exp((x - top) / t))
        w = torch.where(x == -math.inf, 0.0, w)
        sure = True
        order = x.sort(descending=True, stable=True).indices
        if k > 0:
            order = order[:k]
        if p <= 0.0:
            order = order[:1]
        elif p < 1.0:
            ws = w[order]
            before = ws.cumsum(0) - ws
            goal = p * ws.sum()
            keep = before < goal
            keep[0] = True
            # (sums of few equal weights are exact on both sides)
            sure &= bool(((before - goal).abs() > 2.0 ** -35 * ws.sum()).all()) or bool((ws == ws.round()).all())
            order = order[keep]
        if m > 0:
            least = min(m, 1.0)
            # (the largest weight is 1 on both sides)
            sure &= bool((((w[order] - least).abs() > 2.0 ** -35) | (w[order] == 1.0)).all())
            order = order[w[order] >= least]
        kept = torch.zeros_like(w)
        kept[order] = w[order]
        total = kept.cumsum(0)
        u = min(max(u, 0.0), 1.0) if u == u else 0.0
        goal = u * total[-1]
        sure &= bool(((total - goal).abs() > 2.0 ** -35 * total[-1]).all()) or bool((kept == kept.round()).all())
        over = torch.nonzero(total > goal).flatten()
        token = int(over[0]) if over.numel() else int(torch.nonzero(kept).flatten()[-1])
        log = math.log(kept[token] / total[-1])
        got.append((token, log, 8 * V * (1 + abs(log)) * (1 + abs(log)), sure))
    return list(zip(*got))
