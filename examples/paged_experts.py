"""Serving with a small random decoder whose feed-forward layers belong to experts: chunks of prompts, then single tokens.

Each layer is attention over a paged cache and an experts' layer, a hyper-connection mix before either: the router's logits
choose experts for every token (``expert_route``), ``expert_mlp`` runs them, and its result goes into the next mix with that
mix's gate. ``token_sample`` draws the next tokens from the last logits. A batch has a fixed number of places: those behind the
last sequence are no sequence's (``live``), so that one captured graph serves any number of them.

    python examples/paged_experts.py
"""
import torch

import paged_beam
from paged_beam import Cache

import hyper_connection_rank_gb300 as hc


class ExpertDecoder(paged_beam.Decoder):
    """The decoder of paged_beam.py with an experts' layer behind every attention layer."""

    def __init__(self, seed=0, layers=3, hidden=256, experts=16, chosen=4, inner=128, groups=4, top_groups=2, dtype=torch.bfloat16,
                 **kw):
        super().__init__(seed=seed, layers=layers, hidden=hidden, dtype=dtype, **kw)
        extra = paged_beam.Decoder(seed=seed + 1, layers=layers, hidden=hidden, dtype=dtype, **kw)
        self.mixes += extra.mixes[1:]
        g = torch.Generator(device="cuda").manual_seed(seed + 2)

        def w(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") / shape[-2] ** 0.5).to(dtype)

        self.routers = [w(hidden, experts) for _ in range(layers)]
        self.biases = [0.1 * torch.randn(experts, generator=g, device="cuda") for _ in range(layers)]
        # gate and up lie side by side
        self.inner = [w(experts, hidden, 2 * inner).split(inner, -1) for _ in range(layers)]
        self.outer = [w(experts, inner, hidden) for _ in range(layers)]
        self.choose = dict(top_k=chosen, scoring="sigmoid", groups=groups, top_groups=top_groups, group_best=2, scale=1.5)

    def feed_forward(self, i, x, live=None):
        experts, weights = hc.expert_route(x @ self.routers[i], bias=self.biases[i], live=live, **self.choose)
        return hc.expert_mlp(x, *self.inner[i], self.outer[i], experts, weights)

    def __call__(self, cache, tokens, cu_q=None, max_q=None, live=None):
        """Logits of the new tokens, as in paged_beam.py. live: (1,) int32, how many rows are tokens."""
        streams = self.embed[tokens].repeat(1, self.branches)
        prev_out = prev_gate = None
        h, k = self.heads, self.kv_heads
        for i, (qkv, proj) in enumerate(zip(self.qkv, self.out)):
            x, gate, streams = self.mix(2 * i, streams, prev_out, prev_gate)
            q, key, value = (x @ qkv).view(-1, h + 2 * k, self.dim).split([h, k, k], 1)
            keys, values = cache.layer(i)
            q = hc.rotary_append(q, key, value, keys, values, cache.table, cache.lens, cu_q, inv_freq=self.inv_freq,
                                 amplitude=self.amplitude)
            y = hc.paged_attention(q, keys, values, cache.table, cache.lens, cu_q, window=self.window, max_q=max_q)
            x, gate, streams = self.mix(2 * i + 1, streams, y.flatten(1) @ proj, gate)
            prev_out, prev_gate = self.feed_forward(i, x, live), gate
        x, _, _ = self.mix(2 * len(self.qkv), streams, prev_out, prev_gate)
        return x @ self.head


def generate(model, prompts, steps, seed=0, page=16, places=None, **filters):
    """`steps` tokens behind each prompt (a list of token tensors): (tokens (prompts, steps), their log-probabilities). The
    prompts are read as one batch of chunks, then single tokens by a captured graph over `places` rows."""
    n, lens = len(prompts), [p.numel() for p in prompts]
    places = places or n
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    width = (max(lens) + steps) // page + 1
    cache = Cache(len(model.qkv), places * width, page, model.kv_heads, model.dim, model.dtype, places, width)
    rand = torch.rand(steps, places, generator=torch.Generator().manual_seed(seed)).cuda()
    cu = ints([0] * (places + 1))
    cu[1:n + 1] = ints(lens).cumsum(0)
    cu[n + 1:] = cu[n]
    cache.grow(cu.diff())
    logits = model(cache, torch.cat(prompts), cu, max_q=max(lens))
    token, logprob = torch.zeros(places, dtype=torch.int32, device="cuda"), torch.zeros(places, device="cuda")
    token[:n], logprob[:n] = hc.token_sample(logits[cu[1:n + 1].long() - 1], rand[0, :n], return_logprob=True, **filters)
    path, logs = [token[:n].clone()], [logprob[:n].clone()]
    live, draw = ints([n]), rand[0].clone()
    one = ints([1] * n + [0] * (places - n))
    bounds = ints([min(i, n) for i in range(places + 1)])  # a token for each sequence, none for the other places

    def step():
        y = model(cache, token.long(), bounds, max_q=1, live=live)
        return hc.token_sample(y, draw, return_logprob=True, **filters)

    graph = None
    for i in range(1, steps):
        cache.grow(one)
        draw.copy_(rand[i])
        if graph is None:
            # (the calls before a capture, on another stream; what they write is written again)
            table, kv = cache.table, cache.lens
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                result = step()
        else:
            table.copy_(cache.table)
            kv.copy_(cache.lens)
            cache.table, cache.lens = table, kv
        graph.replay()
        token.copy_(result[0])
        path.append(token[:n].clone())
        logs.append(result[1][:n].clone())
        token.clamp_(min=0)
    return torch.stack(path, 1), torch.stack(logs, 1)


def main():
    model = ExpertDecoder()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 101, (n,), generator=g).cuda() for n in (150, 7, 61)]
    path, logs = generate(model, prompts, 12, places=8, temperature=0.8, top_k=40, top_p=0.95)
    for p, s in zip(path.tolist(), logs.sum(1).tolist()):
        print(f"{s:8.3f}  {p}")


if __name__ == "__main__":
    main()
