"""The entry points of the experts' layer and of the choice of tokens (include/hc_experts.h, include/hc_sample.h) reject bad
arguments on the host before any launch (CPU only; no compute calls)."""
import os
import re

import pytest
import torch

import hyper_connection_rank_gb300 as hc
from hyper_connection_rank_gb300 import _binding as B
from hyper_connection_rank_gb300 import _experts as E
from hyper_connection_rank_gb300 import build as gpu_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORMAT = {"hc_expert_route_t": E._ROUTE, "hc_expert_mlp_t": E._MLP, "hc_token_sample_t": E._SAMPLE}
CODES = {"int64_t": "q", "int32_t": "i", "uint32_t": "I", "float": "f", "size_t": "N"}


@pytest.fixture(scope="module")
def L():
    gpu_build.build()
    return B.load_library()


def fields(struct_name):
    """(name, type, whether it is a pointer) of a struct's fields in the headers, in order."""
    text = "".join(open(os.path.join(ROOT, "include", h)).read() for h in ("hc_experts.h", "hc_sample.h"))
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + struct_name + ";", text).group(1)
    got = []
    for decl in body.split(";"):
        words = decl.replace("const ", "").strip()
        if words:
            kind, rest = words.split(None, 1)
            got += [(name.strip(" *\n"), kind, "*" in name or "*" in kind) for name in rest.split(",")]
    return got


def pack(name, **values):
    have = fields(name)
    assert set(values) <= {f for f, _, _ in have}, set(values) - {f for f, _, _ in have}
    return FORMAT[name].pack(*[values.get(f, 0.0 if kind == "float" and not ptr else 0) for f, kind, ptr in have])


@pytest.mark.parametrize("name", sorted(FORMAT))
def test_packed_structs_have_the_header_s_fields(name):
    """Field by field: pointers and 8-byte integers are 8 bytes, the others 4, in the header's order."""
    codes = re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), FORMAT[name].format.lstrip("@").replace("0q", ""))
    assert codes == "".join("P" if ptr else CODES[kind] for _, kind, ptr in fields(name))


ROUTE = dict(logits=0x1000000, bias=0x2000000, live=0x2100000, experts_out=0x3000000, weights_out=0x4000000, tokens=5,
             logits_stride=64, experts=64, top_k=6, groups=8, top_groups=3, group_best=2, renormalise=1, dtype=B.HC_BF16, scale=1.0)


@pytest.mark.parametrize("over", [
    dict(logits=0), dict(experts_out=0), dict(weights_out=0), dict(tokens=-1), dict(experts=0), dict(groups=0), dict(groups=7),
    dict(top_groups=0), dict(top_groups=9), dict(group_best=0), dict(group_best=3), dict(top_k=0), dict(top_k=25), dict(dtype=4),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(logits_stride=-1), dict(logits=0x1000001), dict(bias=0x2000002),
    dict(live=0x2100001), dict(experts_out=ROUTE["logits"] + 64), dict(weights_out=ROUTE["experts_out"] + 8),
    dict(weights_out=ROUTE["bias"])], ids=str)
def test_route_rejects(L, over):
    assert L.hc_expert_route(pack("hc_expert_route_t", **{**ROUTE, **over}), None) == B.HC_ERR_INVALID_ARG
    assert L.hc_last_error()


@pytest.mark.parametrize("over", [dict(experts=1028, groups=4, logits_stride=1028), dict(groups=64, top_groups=64), dict(top_k=33, top_groups=8),
                                  dict(tokens=2 ** 31)], ids=str)
def test_route_limits(L, over):
    assert L.hc_expert_route(pack("hc_expert_route_t", **{**ROUTE, **over}), None) == B.HC_ERR_UNSUPPORTED


MLP = dict(x=0x10000000, gate=0x20000000, up=0x30000000, down=0x40000000, experts=0x50000000, weights=0x50100000, out=0x60000000,
           workspace=0x70000000, workspace_bytes=1 << 30, tokens=5, x_stride=128, out_stride=128, up_expert_stride=128 * 64,
           up_in_stride=64, up_out_stride=1, down_expert_stride=128 * 64, down_in_stride=128, down_out_stride=1, num_experts=4,
           top_k=2, hidden=128, inner=64, dtype=B.HC_BF16)


@pytest.mark.parametrize("over", [
    dict(x=0), dict(gate=0), dict(up=0), dict(down=0), dict(experts=0), dict(weights=0), dict(out=0), dict(x=0x10000001),
    dict(experts=0x50000002), dict(weights=0x50100001)], ids=str)
def test_mlp_rejects_pointers(L, over):
    assert L.hc_expert_mlp(pack("hc_expert_mlp_t", **{**MLP, **over}), None) == B.HC_ERR_INVALID_ARG
    assert L.hc_last_error()


@pytest.mark.parametrize("over", [
    dict(tokens=-1), dict(num_experts=0), dict(top_k=0), dict(hidden=0), dict(inner=0), dict(dtype=3), dict(flags=1 << 20),
    dict(x_stride=-128), dict(out_stride=127), dict(up_in_stride=63), dict(up_out_stride=2), dict(up_in_stride=1, up_out_stride=127),
    dict(down_in_stride=127), dict(down_out_stride=0), dict(up_expert_stride=-1), dict(down_expert_stride=-8)], ids=str)
def test_mlp_rejects_sizes(L, over):
    args = pack("hc_expert_mlp_t", **{**MLP, **over})
    assert L.hc_expert_mlp(args, None) == B.HC_ERR_INVALID_ARG
    assert L.hc_last_error()
    assert L.hc_expert_mlp_workspace_size(args) == 0


@pytest.mark.parametrize("over", [
    dict(num_experts=1025), dict(top_k=33), dict(hidden=65537, x_stride=65537, out_stride=65537, up_expert_stride=65537 * 64,
                                                 down_in_stride=65537, down_expert_stride=65537 * 64),
    dict(tokens=2 ** 23), dict(tokens=2 ** 40), dict(up_expert_stride=2 ** 45)], ids=lambda v: str(min(v)))
def test_mlp_limits(L, over):
    args = pack("hc_expert_mlp_t", **{**MLP, **over})
    assert L.hc_expert_mlp(args, None) == B.HC_ERR_UNSUPPORTED
    assert L.hc_expert_mlp_workspace_size(args) == 0


SAMPLE = dict(logits=0x1000000, uniform=0x2000000, temperatures=0x2100000, top_ps=0x2200000, min_ps=0x2300000, top_ks=0x2400000,
              tokens_out=0x3000000, logprobs_out=0x4000000, rows=3, logits_stride=1000, vocab=1000, dtype=B.HC_F16)


@pytest.mark.parametrize("over", [
    dict(logits=0), dict(uniform=0), dict(tokens_out=0), dict(rows=-1), dict(vocab=0), dict(dtype=-1), dict(logits_stride=-1),
    dict(logits=0x1000001), dict(uniform=0x2000001), dict(top_ks=0x2400002), dict(logprobs_out=0x4000003),
    dict(tokens_out=SAMPLE["logits"] + 2000), dict(logprobs_out=SAMPLE["tokens_out"] + 8), dict(tokens_out=SAMPLE["top_ks"])],
    ids=str)
def test_sample_rejects(L, over):
    assert L.hc_token_sample(pack("hc_token_sample_t", **{**SAMPLE, **over}), None) == B.HC_ERR_INVALID_ARG
    assert L.hc_last_error()


@pytest.mark.parametrize("over", [dict(vocab=409601, logits_stride=409601), dict(rows=2 ** 24), dict(rows=100, logits_stride=2 ** 40)], ids=str)
def test_sample_limits(L, over):
    assert L.hc_token_sample(pack("hc_token_sample_t", **{**SAMPLE, **over}), None) == B.HC_ERR_UNSUPPORTED


def test_nothing_to_do(L):
    """No rows: fine, whatever the pointers; no arguments: not."""
    assert L.hc_expert_route(pack("hc_expert_route_t", **{**ROUTE, "tokens": 0, "logits": 0}), None) == B.HC_OK
    assert L.hc_expert_mlp(pack("hc_expert_mlp_t", **{**MLP, "tokens": 0, "x": 0, "workspace": 0}), None) == B.HC_OK
    assert L.hc_token_sample(pack("hc_token_sample_t", **{**SAMPLE, "rows": 0, "logits": 0}), None) == B.HC_OK
    for f in (L.hc_expert_route, L.hc_expert_mlp, L.hc_token_sample):
        assert f(None, None) == B.HC_ERR_INVALID_ARG
    assert L.hc_expert_mlp_workspace_size(None) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are nobody's")
def test_good_arguments_reach_the_device(L):
    """Without one there is an error of another kind."""
    for f, args in ((L.hc_expert_route, pack("hc_expert_route_t", **ROUTE)), (L.hc_expert_mlp, pack("hc_expert_mlp_t", **MLP)),
                    (L.hc_token_sample, pack("hc_token_sample_t", **SAMPLE))):
        assert f(args, None) in (B.HC_ERR_CUDA, B.HC_ERR_UNSUPPORTED)


def test_cpu_tensors_are_refused():
    x, w = torch.zeros(2, 8), torch.zeros(4, 8, 8)
    e, r = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    for call in (lambda: hc.expert_route(x, 2), lambda: hc.expert_mlp(x, w, w, w, e, r), lambda: hc.token_sample(x, x[:, 0]),
                 lambda: hc.expert_mlp_workspace_size(x, w, w, w, e, r)):
        with pytest.raises((ValueError, TypeError)):
            call()
