"""Plain float64 forms of the paged-cache operators, on lists and dense tensors, and the error bounds that the tests hold the
kernels to. Written from the definitions in include/hc_paged.h; nothing here uses the library.

Bounds. u is the unit roundoff of the tensors' type T (2^-24, 2^-11, 2^-8), v = 2^-24 that of float32.

Rotation: y = a cos - b sin with amplitude A. The half turns are rounded to float32 (angle off by pi 2^-25 at most), sine and
cosine are off by 2 v, three roundings follow: |y - y*| <= A (|a| + |b|) 8 v + u |y*|. The 64-bit fraction of a turn (and the
float64 angle here) carry 2^-53 of the angle each: |position * frequency| 2^-51 more.

Attention: a score is a sum of dim products, then scaled (and capped: tanh has slope at most 1, and its own error is
below 4 v times the cap): ds = (dim + 8) v A, A = scale * sum_d |q_d k_d| at its largest over the row's keys, plus 4 v cap.
Base-2 exponents round once more, their power is off by 2^-21 at most: a weight is off by the factor 1 + e with
e = ds + 4 v |s| + 2^-21. Weights, their sum and the sum of values: |o - o*| <= (2 e + (n + 16) v) W with
W = sum_j p_j |v_j| and n keys. The 16-bit kernels round each weight to T: u W more, and in float16 where weights
below 2^-14 of the largest lose more, 2^-25 sum_j |v_j|. The store rounds once: u |o*|. lse: e + (n + 16) v + 2 v |lse|.
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
V = 2.0 ** -24


def rotate(x, positions, inv_freq, amplitude=1.0, interleaved=False, inverse=False):
    """x (tokens, heads, dim): the rotated heads in float64, and the bound of their error."""
    u = U[x.dtype]
    x = x.double()
    f = inv_freq.double()
    half = f.numel()
    angle = positions.double()[:, None] * f
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None] * (-1 if inverse else 1)
    y, tol = x.clone(), torch.zeros_like(x)
    ia = torch.arange(half) * 2 if interleaved else torch.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = amplitude * (a * c - b * s)
    y[..., ib] = amplitude * (b * c + a * s)
    t = abs(amplitude) * (a.abs() + b.abs()) * (8 * V + angle.abs()[:, None] * 2.0 ** -51)
    tol[..., ia] = t + u * y[..., ia].abs()
    tol[..., ib] = t + u * y[..., ib].abs()
    # (float16 below its normal range rounds to multiples of 2^-24)
    return y, tol + (2.0 ** -25 if u == 2.0 ** -11 else 0.0)


def attention(q, k_cache, v_cache, table, lens, cu=None, scale=None, window=0, softcap=0.0):
    """(out, lse, bound of out, bound of lse) in float64; q etc. on the CPU."""
    u = U[q.dtype]
    tokens, heads, dim = q.shape
    page, kv_heads = k_cache.shape[1:3]
    group = heads // kv_heads
    scale = 1 / math.sqrt(dim) if scale is None else scale
    seqs = table.shape[0]
    cu = list(range(seqs + 1)) if cu is None else cu.tolist()
    out = torch.zeros(tokens, heads, dim, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    ltol = torch.zeros_like(lse)
    for s in range(seqs):
        n, nq = min(int(lens[s]), table.shape[1] * page), cu[s + 1] - cu[s]
        if n <= 0 or nq == 0:
            continue
        ids = table[s, : -(-n // page)].long()
        k = k_cache[ids].flatten(0, 1)[:n].double()
        v = v_cache[ids].flatten(0, 1)[:n].double()
        for i in range(nq):
            p = n - nq + i
            lo = max(0, p - window + 1) if window else 0
            if p < 0:
                continue
            for g in range(kv_heads):
                x = q[cu[s] + i, g * group:(g + 1) * group].double()
                kk, vv = k[lo:p + 1, g], v[lo:p + 1, g]
                z = x @ kk.T * scale
                big = (x.abs() @ kk.abs().T).amax(1, keepdim=True) * abs(scale)
                ds = (dim + 8) * V * big
                if softcap:
                    z = softcap * torch.tanh(z / softcap)
                    ds = ds + 4 * V * softcap
                e = ds + 4 * V * z.abs().amax(1, keepdim=True) + 2.0 ** -21
                m = torch.logsumexp(z, 1, keepdim=True)
                w = torch.exp(z - m)
                o = w @ vv
                W = w @ vv.abs()
                t = (2 * e + (p + 1 - lo + 16) * V) * W + u * o.abs()
                if q.dtype != torch.float32:
                    t = t + u * W
                if q.dtype == torch.float16:
                    t = t + 2.0 ** -25 * vv.abs().sum(0) + 2.0 ** -25
                h = slice(g * group, (g + 1) * group)
                out[cu[s] + i, h], tol[cu[s] + i, h] = o, t
                lse[cu[s] + i, h] = m[:, 0]
                ltol[cu[s] + i, h] = (e + (p + 1 - lo + 16) * V + 2 * V * m.abs())[:, 0]
    return out, lse, tol, ltol


class Pages:
    """A pool's tables and counts as lists, one page at a time."""

    def __init__(self, table, lens, refs, page):
        self.page, self.width = page, table.shape[1]
        self.refs = refs.tolist()
        cap = self.width * page
        self.lens = [max(0, n) for n in lens.tolist()]
        self.rows = [row[: -(-min(n, cap) // page)] for row, n in zip(table.tolist(), self.lens)]
        self.ok = lambda p: 0 <= p < len(self.refs)

    def free(self):
        return [p for p, c in enumerate(self.refs) if c <= 0]

    def table(self, rows):
        rows = [[p if self.ok(p) else -1 for p in r] for r in rows]
        return torch.tensor([r + [-1] * (self.width - len(r)) for r in rows], dtype=torch.int32).reshape(-1, self.width)

    def fork(self, parents):
        """(table, lens, refs, missing, copies) after it."""
        for row in self.rows:
            for p in row:
                if self.ok(p):
                    self.refs[p] -= 1
        new, lens, want, seen = [], [], [], set()
        for i, parent in enumerate(parents):
            known = 0 <= parent < len(self.rows)
            row = list(self.rows[parent]) if known else []
            n = min(self.lens[parent], self.width * self.page) if known else 0
            if parent in seen and n % self.page:
                if self.ok(row[-1]):
                    want.append((i, row[-1]))
                row[-1] = -1
            seen.add(parent)
            for p in row:
                if self.ok(p):
                    self.refs[p] += 1
            new.append(row)
            lens.append(n)
        free, copies = self.free(), []
        for (i, a), b in zip(want, free):
            new[i][-1] = b
            self.refs[b] = 1
            copies.append((a, b))
        return self.table(new), lens, self.refs, len(want) - len(copies), copies

    def extend(self, more):
        new, lens, missing = [], [], 0
        free = self.free()
        for row, n, m in zip(self.rows, self.lens, more):
            row, m = list(row), max(0, m)
            need = -(-(n + m) // self.page) - -(-n // self.page)
            for _ in range(need):
                if len(row) < self.width and free:
                    b = free.pop(0)
                    self.refs[b] = 1
                    row.append(b)
                else:
                    missing += 1
            new.append(row)
            lens.append(min(n + m, len(row) * self.page))
        return self.table(new), lens, self.refs, missing

    def release(self, drop):
        for row, d in zip(self.rows, drop):
            for p in row:
                if d and self.ok(p):
                    self.refs[p] -= 1
        return self.table([[] if d else r for r, d in zip(self.rows, drop)]), \
            [0 if d else n for n, d in zip(self.lens, drop)], self.refs

    def compact(self):
        """(table, refs, remap, live, moves)"""
        live = sum(c > 0 for c in self.refs)
        holes = [p for p in self.free() if p < live]
        movers = [p for p, c in enumerate(self.refs) if c > 0 and p >= live]
        remap = [p if c > 0 else -1 for p, c in enumerate(self.refs)]
        for a, b in zip(movers, holes):
            remap[a] = b
        refs = [0] * len(self.refs)
        for p, c in enumerate(self.refs):
            if c > 0:
                refs[remap[p]] = c
        rows = [[remap[p] if self.ok(p) else -1 for p in row] for row in self.rows]
        return self.table(rows), refs, remap, live, list(zip(movers, holes))
