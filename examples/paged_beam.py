"""Beam search with a small random decoder: hyper-connection mixes around attention over a paged key/value cache.

Each layer is a low-rank mix (``lowrank_mix``), whose output feeds the layer's projections; the new queries and keys are
rotated and the keys and values written into pages (``rotary_append``), ``paged_attention`` reads them back, and the
projected result goes into the next mix with its gate. The pool of pages serves all layers: planes 2l and 2l + 1 are the
keys and values of layer l. Sequences grow by ``page_extend``, beams go on from one another by ``page_fork``, and
``page_compact`` moves a fragmented pool together between two steps.

    python examples/paged_beam.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import hyper_connection_rank_gb300 as hc  # noqa: E402


class Cache:
    """A pool of pages, and the sequences that live in it."""

    def __init__(self, layers, pages, page, kv_heads, dim, dtype, seqs, width):
        self.pool = torch.zeros(2 * layers, pages, page, kv_heads, dim, dtype=dtype, device="cuda")
        self.page = page
        ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.lens, self.refs = ints(seqs, width) - 1, ints(seqs), ints(pages)

    def layer(self, i):
        return self.pool[2 * i], self.pool[2 * i + 1]

    def grow(self, new_tokens):
        self.table, self.lens, self.refs, missing = hc.page_extend(self.table, self.lens, self.refs, new_tokens,
                                                                   page_size=self.page)
        return missing

    def fork(self, parents):
        self.table, self.lens, self.refs, missing = hc.page_fork(self.pool, self.table, self.lens, self.refs, parents)
        return missing

    def compact(self):
        self.table, self.refs, _, live = hc.page_compact(self.pool, self.table, self.lens, self.refs)
        return live


class Decoder:
    """A decoder of hyper-connected attention layers with random weights."""

    def __init__(self, seed=0, vocab=101, layers=3, branches=4, hidden=256, rank=64, heads=8, kv_heads=2, dim=64, window=0,
                 dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda rows, *cols: (torch.randn(rows, *cols, generator=g, device="cuda") / rows ** 0.5).to(dtype)  # noqa: E731
        self.branches, self.heads, self.kv_heads, self.dim, self.window, self.dtype = branches, heads, kv_heads, dim, window, dtype
        wide = branches * hidden
        self.embed = w(hidden, vocab).t().contiguous() * hidden ** 0.5
        self.mixes = [dict(norm_scale=torch.ones(wide, dtype=dtype, device="cuda"), down_w=w(wide, rank), up_w=w(rank, wide),
                           inject_w=w(wide, branches)) for _ in range(layers + 1)]
        self.qkv = [w(hidden, (heads + 2 * kv_heads) * dim) for _ in range(layers)]
        self.out = [w(heads * dim, hidden) for _ in range(layers)]
        self.head = w(hidden, vocab)
        self.inv_freq, self.amplitude = hc.rotary_frequencies(dim)

    def mix(self, i, streams, prev_out, prev_gate):
        return hc.lowrank_mix(streams, prev_out=prev_out, prev_gate=prev_gate, num_branches=self.branches,
                              reduction_scale=1.0 / self.branches, gate_mul=2.0, **self.mixes[i])

    def __call__(self, cache, tokens, cu_q=None, max_q=None):
        """Logits of the new tokens, whose pages the cache already has. cu_q bounds each sequence's; None: one each."""
        streams = self.embed[tokens].repeat(1, self.branches)
        prev_out = prev_gate = None
        h, k = self.heads, self.kv_heads
        for i, (qkv, proj) in enumerate(zip(self.qkv, self.out)):
            x, gate, streams = self.mix(i, streams, prev_out, prev_gate)
            q, key, value = (x @ qkv).view(-1, h + 2 * k, self.dim).split([h, k, k], 1)
            keys, values = cache.layer(i)
            q = hc.rotary_append(q, key, value, keys, values, cache.table, cache.lens, cu_q, inv_freq=self.inv_freq,
                                 amplitude=self.amplitude)
            y = hc.paged_attention(q, keys, values, cache.table, cache.lens, cu_q, window=self.window, max_q=max_q)
            prev_out, prev_gate = y.flatten(1) @ proj, gate
        x, _, _ = self.mix(len(self.qkv), streams, prev_out, prev_gate)
        return (x @ self.head).float()


def beam_search(model, prompt, beams=4, steps=12, page=16, pages=None, compact_at=None):
    """The best sequences that go on from a prompt: (tokens (beams, steps), their log-probabilities, logits of the last step)."""
    n = prompt.numel()
    width = (n + steps) // page + 1
    cache = Cache(len(model.qkv), pages or 2 * beams * width, page, model.kv_heads, model.dim, model.dtype, 1, width)
    cache.grow(torch.tensor([n], dtype=torch.int32, device="cuda"))
    logits = model(cache, prompt, torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n)[-1:]
    scores = torch.zeros(1, device="cuda")
    path = torch.zeros(1, 0, dtype=torch.int64, device="cuda")
    for step in range(steps):
        total = (scores[:, None] + torch.log_softmax(logits, -1)).flatten()
        scores, best = total.topk(beams)
        parents, token = best // logits.shape[1], best % logits.shape[1]
        path = torch.cat((path[parents], token[:, None]), 1)
        cache.fork(parents.int())
        if step == compact_at:
            cache.compact()
        if step + 1 < steps:
            cache.grow(torch.ones(beams, dtype=torch.int32, device="cuda"))
            logits = model(cache, token)
    return path, scores, logits


def main():
    model = Decoder()
    prompt = torch.randint(0, 101, (150,), generator=torch.Generator().manual_seed(1)).cuda()
    path, scores, _ = beam_search(model, prompt, compact_at=5)
    for p, s in zip(path.tolist(), scores.tolist()):
        print(f"{s:8.3f}  {p}")


if __name__ == "__main__":
    main()
