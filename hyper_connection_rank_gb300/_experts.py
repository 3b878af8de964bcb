"""Binding of the experts' layer (include/hc_experts.h) and of the choice of tokens (include/hc_sample.h).

Argument checks and marshalling only, as in _binding.py: every step runs in
the CUDA kernels of libhc_lowrank_mix.so, PyTorch supplies memory and streams.
All calls are asynchronous and may be captured in a CUDA graph; ``stream=`` runs
a call, and allocates, on another stream than the current one.
"""
from __future__ import annotations

import struct

import torch

from ._binding import check, lib
from ._paged import _current_device, _current_stream, _device, _dtype_code, _launch, _on_stream, _sized

__all__ = ["expert_route", "expert_mlp", "expert_mlp_workspace_size", "token_sample"]

# The argument structs of the headers, field by field ("0q": padded to 8 bytes as in C).
_ROUTE = struct.Struct("@5P2q5i2iif0q")
_MLP = struct.Struct("@7PPN3q3q3q4iiI0q")
_SAMPLE = struct.Struct("@2P3PP2P2qii3fi0q")

_SCORING = {"softmax": 0, "sigmoid": 1}


def _rows(name, t, dtype, device):
    """A matrix with contiguous rows: (rows, columns, elements from row to row)."""
    if t.dtype is not dtype or t.get_device() != device or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-dimensional CUDA tensor of dtype {dtype} on device {device}")
    (rows, cols), (step, inner) = t.shape, t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return rows, cols, step if rows > 1 else cols


def _dense(name, t, shape, dtype, device):
    """The address of a contiguous tensor of this shape."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of shape {shape} and dtype {dtype} on device {device}")
    return t.data_ptr()


def expert_route(logits, top_k, *, bias=None, scoring="softmax", groups=1, top_groups=None, group_best=1, renormalise=True,
                 scale=1.0, live=None, stream=None):
    """Experts for every token (hc_expert_route). logits: (tokens, experts), float32, float16 or bfloat16, any row stride;
    scoring: "softmax" or "sigmoid"; bias: (experts,) float32, added to the scores for the choice but not to the weights.
    groups > 1: only the experts of the top_groups best runs of experts / groups are chosen from, a run counting as the sum of
    its group_best (1 or 2) best. Equal values go to the lower index. The weights are the chosen scores, divided by their sum
    with ``renormalise``, times ``scale``. live: (1,) int32, how many rows are tokens; the others get experts of -1 and
    weights of 0. Returns (experts (tokens, top_k) int32, best first, weights (tokens, top_k) float32)."""
    if stream is not None:
        return _on_stream(stream, expert_route, logits, top_k, bias=bias, scoring=scoring, groups=groups, top_groups=top_groups,
                          group_best=group_best, renormalise=renormalise, scale=scale, live=live)
    code, device = _dtype_code(logits), _device(logits)
    tokens, experts, step = _rows("logits", logits, logits.dtype, device)
    if scoring not in _SCORING:
        raise ValueError(f"unknown scoring {scoring!r}")
    bias_at = 0 if bias is None else _dense("bias", bias, (experts,), torch.float32, device)
    live_at = 0 if live is None else _dense("live", live, (1,), torch.int32, device)
    ids = logits.new_empty((tokens, max(top_k, 0)), dtype=torch.int32)
    weights = logits.new_empty((tokens, max(top_k, 0)), dtype=torch.float32)
    args = _ROUTE.pack(logits.data_ptr(), bias_at, live_at, ids.data_ptr(), weights.data_ptr(), tokens, step, experts, top_k,
                       groups, groups if top_groups is None else top_groups, group_best, _SCORING[scoring], bool(renormalise),
                       code, scale)
    _launch(device, lib().hc_expert_route, args)
    return ids, weights


def _weight(name, t, dtype, device):
    """(shape, strides) of a weight of (experts, inputs, outputs)."""
    if t.dtype is not dtype or t.get_device() != device or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-dimensional CUDA tensor of dtype {dtype} on device {device}")
    shape, (es, i, o) = tuple(t.shape), t.stride()
    # (the stride of an axis of one element says nothing)
    if shape[2] == 1 and i != 1:
        o = 1
    if shape[1] == 1 and o != 1:
        i = 1
    if i == 1 and o == 1:
        i, o = (max(shape[2], 1), 1) if shape[1] == 1 else (1, max(shape[1], 1))
    return shape, (es if shape[0] > 1 else 0, i, o)


def _mlp_args(x, gate_w, up_w, down_w, experts, weights, flags, out, out_step, work, size, device):
    dtype = x.dtype
    code = _dtype_code(x)
    tokens, hidden, step = _rows("x", x, dtype, device)
    shape, us = _weight("gate_w", gate_w, dtype, device)
    ushape, us2 = _weight("up_w", up_w, dtype, device)
    dshape, ds = _weight("down_w", down_w, dtype, device)
    n, _, inner = shape
    if ushape != shape or us2 != us:
        raise ValueError("gate_w and up_w must have the same shape and strides")
    if shape[1] != hidden or dshape != (n, inner, hidden):
        raise ValueError("gate_w and up_w must be (experts, hidden, inner), down_w (experts, inner, hidden), with the hidden of x")
    if experts.dim() != 2:
        raise ValueError("experts must be (tokens, top_k)")
    top_k = experts.shape[1]
    ids_at = _dense("experts", experts, (tokens, top_k), torch.int32, device)
    weights_at = _dense("weights", weights, (tokens, top_k), torch.float32, device)
    return _MLP.pack(x.data_ptr(), gate_w.data_ptr(), up_w.data_ptr(), down_w.data_ptr(), ids_at, weights_at, out, work, size,
                     tokens, step, out_step, *us, *ds, n, top_k, hidden, inner, code, flags)


def expert_mlp_workspace_size(x, gate_w, up_w, down_w, experts, weights, *, flags=0):
    """Bytes of workspace that ``expert_mlp`` needs for these tensors (their contents do not matter)."""
    device = _device(x)
    args = _mlp_args(x, gate_w, up_w, down_w, experts, weights, flags, 0, x.shape[1], 0, 0, device)
    return _sized(device, lib().hc_expert_mlp_workspace_size, args)


def expert_mlp(x, gate_w, up_w, down_w, experts, weights, *, out=None, workspace=None, flags=0, stream=None):
    """The feed-forward layer of chosen experts (hc_expert_mlp): for every token the sum over j of weights[:, j] *
    (silu(x @ gate_w[e]) * (x @ up_w[e])) @ down_w[e] with e = experts[:, j]. x: (tokens, hidden), any row stride; gate_w,
    up_w: (num_experts, hidden, inner) and down_w: (num_experts, inner, hidden), whose last or second axis is contiguous
    (``w.transpose(1, 2)`` of weights kept outputs first); experts: (tokens, top_k) int32 and weights: (tokens, top_k)
    float32, as ``expert_route`` gives them. Experts outside 0 .. num_experts - 1 take no part; a row without any gets zeros.
    ``workspace``: a CUDA tensor of at least ``expert_mlp_workspace_size`` bytes, allocated here if omitted."""
    if stream is not None:
        return _on_stream(stream, expert_mlp, x, gate_w, up_w, down_w, experts, weights, out=out, workspace=workspace,
                          flags=flags)
    device = _device(x)
    if out is None:
        out = x.new_empty(x.shape)
    elif out.shape != x.shape:
        raise ValueError("out must have the shape of x")
    out_step = _rows("out", out, x.dtype, device)[2]
    L = lib()
    args = _mlp_args(x, gate_w, up_w, down_w, experts, weights, flags, out.data_ptr(), out_step, 0, 0, device)
    if workspace is not None:
        if workspace.get_device() != device:
            raise ValueError(f"workspace must be a CUDA tensor on device {device}")
        _launch(device, L.hc_expert_mlp, _with(args, workspace.data_ptr(), workspace.numel() * workspace.element_size()))
    elif device == _current_device():
        _mlp_in_scratch(L, device, args)
    else:
        with torch.cuda.device(device):
            _mlp_in_scratch(L, device, args)
    return out


# A block of the current stream's memory without a tensor around it, where this build of torch has that (a third of the time).
_alloc, _free = (getattr(torch._C, "_cuda_cudaCachingAllocator_raw_" + n, None) for n in ("alloc", "delete"))


def _with(args, workspace, size):
    """_MLP's fields with this workspace."""
    return args[:56] + struct.pack("@PN", workspace, size) + args[72:]


def _mlp_in_scratch(L, device, args):
    """The call on the current device and stream, with a workspace that goes back to the allocator right behind it."""
    size, stream = L.hc_expert_mlp_workspace_size(args), _current_stream(device)
    if not size:  # (no rows, or an error that the call reports)
        check(L.hc_expert_mlp(args, stream))
    elif _alloc is None or _free is None:
        work = torch.empty(size, dtype=torch.uint8, device=device)
        check(L.hc_expert_mlp(_with(args, work.data_ptr(), size), stream))
    else:
        work = _alloc(size, stream)
        try:
            check(L.hc_expert_mlp(_with(args, work, size), stream))
        finally:
            _free(work)


def _choice(name, v, rows, dtype, device):
    """(address, number) of a parameter that is a tensor (rows,) or a number."""
    return (_dense(name, v, (rows,), dtype, device), 0) if isinstance(v, torch.Tensor) else (0, v)


def token_sample(logits, uniform, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, return_logprob=False, stream=None):
    """Draw every row's next token (hc_token_sample). logits: (rows, vocab), float32, float16 or bfloat16, any row stride;
    uniform: (rows,) float32 random numbers in [0, 1). temperature, top_p, min_p (float32) and top_k (int32): a number for all
    rows or a tensor (rows,). Of the tokens in the order of falling logits the first top_k stay (0: all), of those the first
    whose probabilities reach top_p, of those the ones at least min_p times as probable as the first. A temperature of 0
    takes the largest logit. Returns tokens (rows,) int32, -1 for a row that has nothing to choose from, and with
    return_logprob also their log-probabilities (rows,) float32 among what stayed."""
    if stream is not None:
        return _on_stream(stream, token_sample, logits, uniform, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p,
                          return_logprob=return_logprob)
    code, device = _dtype_code(logits), _device(logits)
    rows, vocab, step = _rows("logits", logits, logits.dtype, device)
    t_at, t = _choice("temperature", temperature, rows, torch.float32, device)
    k_at, k = _choice("top_k", top_k, rows, torch.int32, device)
    p_at, p = _choice("top_p", top_p, rows, torch.float32, device)
    m_at, m = _choice("min_p", min_p, rows, torch.float32, device)
    tokens = logits.new_empty((rows,), dtype=torch.int32)
    logprobs = logits.new_empty((rows,), dtype=torch.float32) if return_logprob else None
    args = _SAMPLE.pack(logits.data_ptr(), _dense("uniform", uniform, (rows,), torch.float32, device), t_at, p_at, m_at, k_at,
                        tokens.data_ptr(), logprobs.data_ptr() if return_logprob else 0, rows, step, vocab, k, t, p, m, code)
    _launch(device, lib().hc_token_sample, args)
    return (tokens, logprobs) if return_logprob else tokens
