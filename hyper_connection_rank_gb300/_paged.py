"""Binding of the paged-cache operators (include/hc_paged.h).

Argument checks and marshalling only, as in _binding.py: every step runs in
the CUDA kernels of libhc_lowrank_mix.so, PyTorch supplies memory and streams.

Tensors of a batch, in all functions that take one:

  page_table (seqs, max_pages) int32, kv_lens (seqs,) int32, cu_q (seqs + 1,) int32 or None,
  k_cache, v_cache (num_pages, page_size, kv_heads, head_dim), any strides but a contiguous last axis

``kv_lens`` counts the new tokens of the call too. ``cu_q`` bounds each sequence's rows of q; None means one new token
for every sequence. All calls are asynchronous and may be captured in a CUDA graph.
"""
from __future__ import annotations

import math
import struct

import torch

from ._binding import DTYPE_CODES, check, lib

__all__ = ["rotary_frequencies", "rotary", "rotary_append", "paged_attention", "paged_attention_workspace_size",
           "page_copy", "page_fork", "page_extend", "page_release", "page_compact"]

# The argument structs of include/hc_paged.h, field by field ("0q": padded to 8 bytes as in C).
_ROTARY = struct.Struct("@4P5q7if0q")
_APPEND = struct.Struct("@10P3q6q2q3q3i4iiif0q")
_ATTENTION = struct.Struct("@9PN3q4q3q3i3i2iiiI2f0q")
# (in three parts, of which the middle one, workspace and its size, is known last)
_ATTENTION_FRONT, _ATTENTION_WORK, _ATTENTION_BACK = struct.Struct("@8P"), struct.Struct("@PN"), struct.Struct("@3q4q3q3i3i2iiiI2f0q")
_NO_WORK = _ATTENTION_WORK.pack(0, 0)
_PAGES = struct.Struct("@6P2q3i0q")


# (A call costs the host as much as a small kernel costs the GPU, so the checks below ask each tensor for as little as they
# can; what the library checks itself is left to it.)

def _device(t):
    """The index of the GPU that a call's first tensor lies on, which all the others must share."""
    device = t.get_device()
    if device < 0:
        raise ValueError("expected CUDA tensors")
    return device


def _heads(name, t, dtype, device):
    """A tensor of rows of heads, the last axis contiguous: (shape, strides)."""
    if t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor of dtype {dtype} on device {device}")
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or (strides[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name} must have three axes, the last one contiguous")
    return shape, strides


def _flat(name, t, dtype, device):
    if t.dtype is not dtype or t.get_device() != device or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-dimensional CUDA tensor of dtype {dtype} on device {device}")
    return t.shape[0]


def _dtype_code(t):
    code = DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _table(t, device):
    """(sequences, columns, entries from one row to the next)"""
    if t.dtype is not torch.int32 or t.get_device() != device or t.dim() != 2:
        raise ValueError(f"page_table must be a 2-dimensional CUDA tensor of dtype torch.int32 on device {device}")
    (seqs, width), (step, inner) = t.shape, t.stride()
    if width < 1 or (inner != 1 and width > 1):
        raise ValueError("page_table needs at least one column, and contiguous rows")
    return seqs, width, step if seqs > 1 else max(step, width)


def _batch(page_table, kv_lens, cu_q, tokens, device):
    """(sequences, columns, row step of the table, address of cu_q)"""
    seqs, width, step = _table(page_table, device)
    if _flat("kv_lens", kv_lens, torch.int32, device) != seqs:
        raise ValueError("kv_lens and page_table differ in sequences")
    if cu_q is None:
        if tokens != seqs:
            raise ValueError("without cu_q every sequence has one new token")
        return seqs, width, step, 0
    if _flat("cu_q", cu_q, torch.int32, device) != seqs + 1:
        raise ValueError("cu_q must have one entry more than there are sequences")
    return seqs, width, step, cu_q.data_ptr()


def _caches(k_cache, v_cache, dtype, device):
    """(shape, strides) of both."""
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype or k_cache.get_device() != device or \
            v_cache.get_device() != device:
        raise ValueError(f"k_cache and v_cache must be CUDA tensors of dtype {dtype} on device {device}")
    shape, strides = k_cache.shape, k_cache.stride()
    if shape != v_cache.shape or strides != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    if len(shape) != 4 or (strides[3] != 1 and shape[3] > 1):
        raise ValueError("the caches must have four axes, the last one contiguous")
    return shape, strides


def _out(out, like, name, device):
    """(out, its strides): the one given, or a new one of the shape of `like`."""
    if out is None:
        out = torch.empty_like(like)
        return out, out.stride()
    if out.shape != like.shape or out.dtype is not like.dtype:
        raise ValueError(f"out must have the shape and dtype of {name}")
    return out, _heads("out", out, like.dtype, device)[1]


# The current stream's handle and device without Python objects around them, where this build of torch has that.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(device, f, *args):
    """A library call on the current stream of a device, which the library takes to be the current one."""
    if device == _current_device():
        check(f(*args, _current_stream(device)))
    else:
        with torch.cuda.device(device):
            check(f(*args, _current_stream(device)))


def _sized(device, f, *args):
    """A size that the library gives for the current device."""
    if device == _current_device():
        return f(*args)
    with torch.cuda.device(device):
        return f(*args)


def _on_stream(stream, f, *args, out=None, workspace=None, **kw):
    """f's call with another stream as the current one, so that what it allocates comes from that stream's memory: a block that
    was freed on this stream may still be in use by kernels queued here. Results are the caller's, who may free them on this
    stream; memory that the caller gave, inputs among it (another call's results may have no other reference), is not handed out
    again before the other stream is done with it."""
    if stream.device.index != args[0].get_device():
        raise ValueError("the stream and the tensors are on different devices")
    kw.update((name, t) for name, t in (("out", out), ("workspace", workspace)) if t is not None)
    for t in (*args, *kw.values()):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        got = f(*args, **kw)
    for t in got if isinstance(got, tuple) else (got,):
        t.record_stream(here)
    return got


def rotary_frequencies(rot_dim, theta=10000.0, *, scaling=None, factor=1.0, original_length=None, slow=1.0, fast=32.0,
                       device="cuda"):
    """The frequencies of a rotation, radians per token, and the amplitude that goes with them: (inv_freq, amplitude) for
    ``rotary`` and ``rotary_append``. inv_freq[i] = theta ** (-2 i / rot_dim), and for contexts ``factor`` times as long as
    those of ``original_length`` tokens that a model was trained with

      scaling="linear"    every frequency divided by factor (positions are interpolated)
      scaling="base"      theta multiplied by factor ** (rot_dim / (rot_dim - 2)): the slowest pair is interpolated, the
                          fastest is left as it is
      scaling="by_parts"  pairs that make fewer than ``slow`` turns in original_length are interpolated, those that make
                          more than ``fast`` are left, those between go over from one to the other linearly in their turns;
                          amplitude 0.1 ln(factor) + 1 (Peng et al., "YaRN: Efficient Context Window Extension of Large
                          Language Models", section 3.2 and 3.4, whose temperature is 1 / amplitude^2)
    """
    if rot_dim < 2 or rot_dim % 2 or not theta > 0 or not factor >= 1:
        raise ValueError("rot_dim must be even and positive, theta positive, factor at least 1")
    exponent = torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim
    amplitude = 1.0
    if scaling == "base":
        if rot_dim == 2:
            raise ValueError("a single pair has no base to scale")
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    f = theta ** -exponent
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        if original_length is None or not 0 < slow < fast:
            raise ValueError("by_parts needs original_length and 0 < slow < fast")
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device), amplitude


def rotary(x, positions, inv_freq, *, amplitude=1.0, interleaved=False, inverse=False, out=None, stream=None):
    """Rotate heads by their positions (hc_rotary). x: (tokens, heads, head_dim), float32, float16 or bfloat16, any token and
    head stride; positions: (tokens,) int64 or int32; inv_freq: (rot_dim / 2,) float64 from ``rotary_frequencies``. Features
    from rot_dim on are copied. ``inverse=True`` turns back, which also takes the gradient of the result to that of x.
    ``out`` may be x itself."""
    if stream is not None:
        return _on_stream(stream, rotary, x, positions, inv_freq, amplitude=amplitude, interleaved=interleaved, inverse=inverse,
                          out=out)
    code, device = _dtype_code(x), _device(x)
    (tokens, heads, dim), xs = _heads("x", x, x.dtype, device)
    half = _flat("inv_freq", inv_freq, torch.float64, device)
    narrow = positions.dtype is torch.int32
    if _flat("positions", positions, torch.int32 if narrow else torch.int64, device) != tokens:
        raise ValueError("positions and x differ in tokens")
    out, os = _out(out, x, "x", device)
    args = _ROTARY.pack(x.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), out.data_ptr(), tokens, xs[0], xs[1], os[0],
                        os[1], heads, dim, 2 * half, bool(interleaved), bool(inverse), narrow, code, amplitude)
    _launch(device, lib().hc_rotary, args)
    return out


def rotary_append(q, k, v, k_cache, v_cache, page_table, kv_lens, cu_q=None, *, inv_freq, amplitude=1.0, interleaved=False,
                  out=None, stream=None):
    """Rotate a batch's new queries, and rotate its new keys and write them with the values into the cache
    (hc_rotary_append). q: (tokens, heads, head_dim); k, v: (tokens, kv_heads, head_dim), which may be parts of one matrix.
    Positions follow from kv_lens and cu_q. Returns the rotated queries (``out``, which may be q itself)."""
    if stream is not None:
        return _on_stream(stream, rotary_append, q, k, v, k_cache, v_cache, page_table, kv_lens, cu_q, inv_freq=inv_freq,
                          amplitude=amplitude, interleaved=interleaved, out=out)
    code, dtype, device = _dtype_code(q), q.dtype, _device(q)
    (tokens, heads, dim), qs = _heads("q", q, dtype, device)
    kshape, ks = _heads("k", k, dtype, device)
    vshape, vs = _heads("v", v, dtype, device)
    (pages, page, kv_heads, cdim), cs = _caches(k_cache, v_cache, dtype, device)
    half = _flat("inv_freq", inv_freq, torch.float64, device)
    if kshape != vshape or kshape != (tokens, kv_heads, dim) or cdim != dim:
        raise ValueError("q, k, v and the caches differ in tokens, kv_heads or head_dim")
    seqs, width, step, cu = _batch(page_table, kv_lens, cu_q, tokens, device)
    out, os = _out(out, q, "q", device)
    args = _APPEND.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                        inv_freq.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(), cu, tokens, pages, step, qs[0], qs[1],
                        ks[0], ks[1], vs[0], vs[1], os[0], os[1], cs[0], cs[1], cs[2], seqs, width, page, heads, kv_heads, dim,
                        2 * half, bool(interleaved), code, amplitude)
    _launch(device, lib().hc_rotary_append, args)
    return out


def _attention_args(q, k_cache, v_cache, page_table, kv_lens, cu_q, scale, window, softcap, max_q, max_kv, flags, out, lse, os,
                    device):
    """The packed arguments before the workspace, and those after."""
    code = _dtype_code(q)
    (tokens, heads, dim), qs = _heads("q", q, q.dtype, device)
    (pages, page, kv_heads, cdim), cs = _caches(k_cache, v_cache, q.dtype, device)
    if cdim != dim or kv_heads < 1 or heads % kv_heads:
        raise ValueError("heads must be a multiple of kv_heads, and head_dim that of the caches")
    seqs, width, step, cu = _batch(page_table, kv_lens, cu_q, tokens, device)
    front = _ATTENTION_FRONT.pack(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                                  kv_lens.data_ptr(), cu, out, lse)
    back = _ATTENTION_BACK.pack(tokens, pages, step, qs[0], qs[1], os[0], os[1], cs[0], cs[1], cs[2], seqs, width, page, heads,
                                kv_heads, dim, max_q or 0, max_kv or 0, window or 0, code, flags,
                                1.0 / math.sqrt(dim) if scale is None else scale, softcap or 0.0)
    return front, back


def paged_attention_workspace_size(q, k_cache, v_cache, page_table, kv_lens, cu_q=None, *, scale=None, max_q=None, max_kv=None,
                                   window=0, flags=0):
    """Bytes of workspace that ``paged_attention`` needs for these tensors (their contents do not matter) and these arguments,
    which steer the choice of kernels: give those of the call."""
    heads, dim = q.shape[1:]
    device = _device(q)
    front, back = _attention_args(q, k_cache, v_cache, page_table, kv_lens, cu_q, scale, window, 0.0, max_q, max_kv, flags, 0, 0,
                                  (heads * dim, dim), device)
    return _sized(device, lib().hc_paged_attention_workspace_size, front + _NO_WORK + back)


def paged_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q=None, *, scale=None, window=0, softcap=0.0, max_q=None,
                    max_kv=None, return_lse=False, out=None, workspace=None, flags=0, stream=None):
    """Causal attention of a batch's new tokens over their sequences in the cache (hc_paged_attention). q: (tokens, heads,
    head_dim), any token and head stride. scale: 1 / sqrt(head_dim) by default; window > 0: only the last ``window``
    positions are seen; softcap > 0: scores go through softcap * tanh(score / softcap). max_q, max_kv: upper bounds of the
    new tokens of a sequence and of kv_lens, if known; they only steer speed. Returns out (tokens, heads, head_dim), and with
    return_lse also the float32 logarithms (tokens, heads) of the sums of weights. A token that sees nothing gets zeros, and
    minus infinity. ``workspace``: a CUDA tensor of at least ``paged_attention_workspace_size`` bytes, allocated here if
    omitted."""
    if stream is not None:
        return _on_stream(stream, paged_attention, q, k_cache, v_cache, page_table, kv_lens, cu_q, scale=scale, window=window,
                          softcap=softcap, max_q=max_q, max_kv=max_kv, return_lse=return_lse, out=out, workspace=workspace,
                          flags=flags)
    device = _device(q)
    out, os = _out(out, q, "q", device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if return_lse else None
    front, back = _attention_args(q, k_cache, v_cache, page_table, kv_lens, cu_q, scale, window, softcap, max_q, max_kv, flags,
                                  out.data_ptr(), 0 if lse is None else lse.data_ptr(), os, device)
    L = lib()
    work = _NO_WORK
    if workspace is None:
        size = _sized(device, L.hc_paged_attention_workspace_size, front + _NO_WORK + back)
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
            work = _ATTENTION_WORK.pack(workspace.data_ptr(), size)
    else:
        if workspace.get_device() != device:
            raise ValueError(f"workspace must be a CUDA tensor on device {device}")
        work = _ATTENTION_WORK.pack(workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _launch(device, L.hc_paged_attention, front + work + back)
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------------------------------------ pages --

def _pool(cache):
    """(planes, pages, bytes of a page, device) of a pool (planes, num_pages, ...)."""
    if not isinstance(cache, torch.Tensor) or not cache.is_cuda or cache.dim() < 3 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous CUDA tensor (planes, num_pages, ...)")
    planes, pages = cache.shape[:2]
    if cache.numel() == 0:
        raise ValueError("cache is empty")
    return planes, pages, cache.numel() // (planes * pages) * cache.element_size(), cache.get_device()


def _pages(page_table, lens, refs, page_size, seqs_out, index, need_lens=True):
    """The new tables and counts, and the packed arguments."""
    seqs, width, step = _table(page_table, index)
    pages = _flat("refs", refs, torch.int32, index)
    if _flat("lens", lens, torch.int32, index) != seqs:
        raise ValueError("lens and page_table differ in sequences")
    if page_size < 1:
        raise ValueError("page_size must be positive")
    device = refs.device
    table_out = torch.empty((seqs_out, width), dtype=torch.int32, device=device)
    lens_out = torch.empty(seqs_out, dtype=torch.int32, device=device) if need_lens else None
    refs_out = torch.empty_like(refs)
    args = _PAGES.pack(page_table.data_ptr(), lens.data_ptr(), refs.data_ptr(), table_out.data_ptr(),
                       lens_out.data_ptr() if need_lens else 0, refs_out.data_ptr(), pages, step, seqs, width, page_size)
    return args, table_out, lens_out, refs_out


def _pages_workspace(refs, seqs):
    n = lib().hc_pages_workspace_size(refs.shape[0], seqs)
    return torch.empty(n, dtype=torch.uint8, device=refs.device), n


def page_copy(cache, src, dst, *, stream=None):
    """Copy pages within a pool (hc_page_copy): cache[:, dst[i]] = cache[:, src[i]]. cache: (planes, num_pages, ...), where
    the planes are the layers' keys and values; src, dst: int32. The dst are distinct and none is a src; entries outside the
    pool are passed over. Returns cache."""
    if stream is not None:
        return _on_stream(stream, page_copy, cache, src, dst)
    planes, pages, size, device = _pool(cache)
    _flat("src", src, torch.int32, device)
    _flat("dst", dst, torch.int32, device)
    if src.shape != dst.shape:
        raise ValueError("src and dst differ in length")
    _launch(device, lib().hc_page_copy, cache.data_ptr(), planes, pages, size, src.data_ptr(), dst.data_ptr(), src.shape[0])
    return cache


def page_fork(cache, page_table, lens, refs, parents, *, page_size=None, stream=None):
    """New sequences that go on from others, as after a step of beam search (hc_page_fork): new sequence i continues
    parents[i] (-1: it is empty), the old ones are given up. Full pages are shared; of a last page that is not full every
    child but the first gets a copy. refs (num_pages,) int32 counts the tables' entries and whoever else holds a page.
    Returns (page_table, lens, refs, missing), all new; missing (1,) counts the children that no free page was left for."""
    if stream is not None:
        return _on_stream(stream, page_fork, cache, page_table, lens, refs, parents, page_size=page_size)
    planes, pages, size, device = _pool(cache)
    _flat("parents", parents, torch.int32, device)
    n = parents.shape[0]
    args, table_out, lens_out, refs_out = _pages(page_table, lens, refs, cache.shape[2] if page_size is None else page_size, n,
                                                 device)
    if refs.shape[0] != pages:
        raise ValueError("refs must have an entry for every page of cache")
    missing = torch.empty(1, dtype=torch.int32, device=refs.device)
    ws, bytes_ = _pages_workspace(refs, max(n, page_table.shape[0]))
    _launch(device, lib().hc_page_fork, args, parents.data_ptr(), n, missing.data_ptr(), cache.data_ptr(), planes, size,
            ws.data_ptr(), bytes_)
    return table_out, lens_out, refs_out, missing


def page_extend(page_table, lens, refs, new_tokens, *, page_size, stream=None):
    """Pages for new_tokens[s] more tokens of every sequence (hc_page_extend). Returns (page_table, lens, refs, missing)."""
    if stream is not None:
        return _on_stream(stream, page_extend, page_table, lens, refs, new_tokens, page_size=page_size)
    device = _device(refs)
    _flat("new_tokens", new_tokens, torch.int32, device)
    seqs = page_table.shape[0]
    if new_tokens.shape[0] != seqs:
        raise ValueError("new_tokens and page_table differ in sequences")
    args, table_out, lens_out, refs_out = _pages(page_table, lens, refs, page_size, seqs, device)
    missing = torch.empty(1, dtype=torch.int32, device=refs.device)
    ws, bytes_ = _pages_workspace(refs, seqs)
    _launch(device, lib().hc_page_extend, args, new_tokens.data_ptr(), missing.data_ptr(), ws.data_ptr(), bytes_)
    return table_out, lens_out, refs_out, missing


def page_release(page_table, lens, refs, drop, *, page_size, stream=None):
    """Sequences with drop[s] (uint8 or bool) give up their pages (hc_page_release). Returns (page_table, lens, refs)."""
    if stream is not None:
        return _on_stream(stream, page_release, page_table, lens, refs, drop, page_size=page_size)
    device = _device(refs)
    _flat("drop", drop, torch.bool if drop.dtype == torch.bool else torch.uint8, device)
    seqs = page_table.shape[0]
    if drop.shape[0] != seqs:
        raise ValueError("drop and page_table differ in sequences")
    args, table_out, lens_out, refs_out = _pages(page_table, lens, refs, page_size, seqs, device)
    _launch(device, lib().hc_page_release, args, drop.data_ptr())
    return table_out, lens_out, refs_out


def page_compact(cache, page_table, lens, refs, *, page_size=None, stream=None):
    """Move the live pages of a pool to its front (hc_page_compact). Returns (page_table, refs, remap, live): the new tables
    and counts, where each page went (-1: nowhere), and the number of live pages."""
    if stream is not None:
        return _on_stream(stream, page_compact, cache, page_table, lens, refs, page_size=page_size)
    planes, pages, size, device = _pool(cache)
    seqs = page_table.shape[0]
    args, table_out, _, refs_out = _pages(page_table, lens, refs, cache.shape[2] if page_size is None else page_size, seqs,
                                          device, need_lens=False)
    if refs.shape[0] != pages:
        raise ValueError("refs must have an entry for every page of cache")
    remap = torch.empty_like(refs)
    live = torch.empty(1, dtype=torch.int32, device=refs.device)
    ws, bytes_ = _pages_workspace(refs, seqs)
    _launch(device, lib().hc_page_compact, args, remap.data_ptr(), live.data_ptr(), cache.data_ptr(), planes, size, ws.data_ptr(),
            bytes_)
    return table_out, refs_out, remap, live
