"""The paged cache around the codec: append new keys and values to it, and
attend over it.

A layer's cache is two tensors of pages, ``k_pages`` and ``v_pages``, indexed
[page, head, token, channel].  Any strides do, as long as channels lie next to
one another: a pool stored [page, token, head, channel] or [page, 2, head,
token, channel] is passed as the permuted or indexed view.  ``page_table``
(int32 [requests, pages]) lists each request's pages, ``q_begin`` (int32
[requests + 1]) its rows among the new tokens and ``kv_len`` (int32
[requests]) the tokens it has cached once they are in; all three live on the
device and may change between replays of a captured call.

Pages of a contiguous [page, head, token, channel] pool are pages of
``BatchPlan(..., page_elems=heads * page_tokens * head_dim)``.

Both calls run on the current stream of the tensors' device, or on ``stream``
(their new tensors are then allocated on it), never synchronise, and return a
status tensor with one word per request.  Neither has a gradient.
"""
from __future__ import annotations

import functools
import math
import struct

_KV = struct.Struct("<9Q4I4Q2IQ")  # sz_paged_kv
_APPEND = struct.Struct("<18Q4I2f")  # sz_append_args
_ATTENTION = struct.Struct("<7Q3If")  # sz_attention_args

# What every call needs, set by the first one.  A decode step makes these
# calls per layer, so their host side is kept to a few microseconds: one
# packed struct instead of a ctypes structure's fields, device ordinals
# instead of device objects.
_T = None        # torch
_TYPES: dict = {}
_LIB = None
_STREAM = None   # device ordinal -> raw handle of its current stream


def _load():
    global _T, _LIB, _STREAM
    import torch

    from . import lib
    _LIB = lib()
    _TYPES[torch.bfloat16] = 1
    _TYPES[torch.float16] = 2
    _STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
    _T = torch
    return torch


def _ints(name, t, ndim, torch):
    if t.dtype is not torch.int32 or t.dim() != ndim or t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("%s must be an int32 tensor of %d dimension(s) with entries side by side" % (name, ndim))


def _rows(name, t, dtype, tokens, dim):
    """Heads of rows [tokens, heads, dim] and their strides."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 3 or shape[0] != tokens or shape[2] != dim:
        raise ValueError("%s must be %s [%d tokens, heads, %d], got %s %s" % (name, dtype, tokens, dim, t.dtype, tuple(shape)))
    s = t.stride()
    if s[2] != 1:
        raise ValueError("%s needs its channels side by side" % name)
    if t.requires_grad:
        raise ValueError("%s requires a gradient, and this operator has none" % name)
    return shape[1], s[0], s[1]


def _pack_kv(torch, k_pages, v_pages, shape, page_table, q_begin, kv_len, tokens):
    code = _TYPES.get(k_pages.dtype)
    if code is None or v_pages.dtype is not k_pages.dtype:
        raise TypeError("pages are bfloat16 or float16, the same for keys and values; got %s and %s" % (k_pages.dtype, v_pages.dtype))
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("pages are two tensors [pages, heads, page tokens, channels] of one shape")
    k0, k1, k2, k3 = k_pages.stride()
    v0, v1, v2, v3 = v_pages.stride()
    if k3 != 1 or v3 != 1:
        raise ValueError("pages need their channels side by side")
    _ints("page_table", page_table, 2, torch)
    _ints("q_begin", q_begin, 1, torch)
    _ints("kv_len", kv_len, 1, torch)
    reqs, max_pages = page_table.shape
    if q_begin.shape[0] != reqs + 1 or kv_len.shape[0] != reqs:
        raise ValueError("%d requests in page_table, %d in q_begin, %d in kv_len" % (reqs, q_begin.shape[0] - 1, kv_len.shape[0]))
    return _KV.pack(k_pages.data_ptr(), v_pages.data_ptr(), k0, k1, k2, v0, v1, v2, shape[0], shape[1], shape[3], shape[2], code,
                    page_table.data_ptr(), page_table.stride(0) if reqs > 1 else max_pages, q_begin.data_ptr(), kv_len.data_ptr(), reqs,
                    max_pages, tokens)


def _device(tensors):
    """The one CUDA device of all tensors (None among them skipped)."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors on %s and %s" % (tensors[0].device, t.device))
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device, not on %s" % tensors[0].device)
    return dev


def _elsewhere(call, dev, stream):
    """``call`` with another device or stream made current, or None where the
    current ones serve already."""
    torch = _T
    if stream is None and torch.cuda.current_device() == dev:
        return None
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    if stream is not None and stream.device.index != dev:
        raise ValueError("a stream of %s for tensors on cuda:%d" % (stream.device, dev))
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return call()


def append_kv(k, v, k_pages, v_pages, page_table, q_begin, kv_len, *, q=None, q_out=None, rope_freqs=None,
              rope_interleaved=False, rope_scale=1.0, positions=None, q_norm=None, k_norm=None, eps=1e-6,
              hists=None, hist_rows=None, stream=None):
    """Write the new tokens' keys and values (``k``, ``v``: [tokens, heads,
    channels]) into their pages; ``sz_append_kv``.

    ``q`` [tokens, query heads, channels] goes through the same norm and
    rotation into ``q_out`` (a new tensor if not given; ``q`` itself is fine).
    ``rope_freqs``: float64 [R/2] radians per position of the R rotated
    channels, as ``rope_frequencies`` gives them; half layout (t, t + R/2), or
    adjacent pairs with ``rope_interleaved``.  ``positions`` (int64 [tokens])
    replaces the place in the cache as the angle's position.  ``q_norm``,
    ``k_norm``: weights of the per-head norm, in the pages' type.  ``hists``
    (32-bit [rows, 256]) gains the exponent counts of what is written: request
    r's keys in row hist_rows[r], its values in row hist_rows[requests + r]
    (rows r and requests + r without ``hist_rows``).

    Returns (q_out or None, status int32 [requests])."""
    torch = _T or _load()
    shape, dtype = k_pages.shape, k_pages.dtype
    tokens, dim = k.shape[0], shape[-1]
    kv = _pack_kv(torch, k_pages, v_pages, shape, page_table, q_begin, kv_len, tokens)
    hk, k0, k1 = _rows("k", k, dtype, tokens, dim)
    hv, v0, v1 = _rows("v", v, dtype, tokens, dim)
    if hk != shape[1] or hv != shape[1]:
        raise ValueError("pages of %d heads, k of %d, v of %d" % (shape[1], hk, hv))
    q_heads = q0 = q1 = rot_dim = n_hists = 0
    if q is not None:
        q_heads, q0, q1 = _rows("q", q, dtype, tokens, dim)
        if q_out is not None and q_out.shape != q.shape:
            raise ValueError("q_out of shape %s for q of %s" % (tuple(q_out.shape), tuple(q.shape)))
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm need q")
    if rope_freqs is not None:
        if rope_freqs.dtype is not torch.float64 or rope_freqs.dim() != 1 or not rope_freqs.is_contiguous():
            raise ValueError("rope_freqs must be a contiguous float64 vector")
        rot_dim = 2 * rope_freqs.shape[0]
    if positions is not None and (positions.dtype is not torch.int64 or positions.shape != (tokens,) or not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous int64 tensor [%d]" % tokens)
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None and (w.dtype is not dtype or w.shape != (dim,) or not w.is_contiguous()):
            raise ValueError("%s must be a contiguous %s tensor [%d]" % (name, dtype, dim))
    if hists is not None:
        if hists.dtype not in (torch.int32, torch.uint32) or hists.shape[-1] != 256 or not hists.is_contiguous():
            raise ValueError("hists must be a contiguous 32-bit tensor of rows of 256 counts")
        n_hists = hists.numel() // 256
    if hist_rows is not None:
        if hists is None:
            raise ValueError("hist_rows needs hists")
        if hist_rows.dtype not in (torch.int32, torch.uint32) or hist_rows.numel() != 2 * kv_len.shape[0] or not hist_rows.is_contiguous():
            raise ValueError("hist_rows must be a contiguous 32-bit tensor of %d rows" % (2 * kv_len.shape[0]))
    dev = _device((k_pages, v_pages, k, v, page_table, q_begin, kv_len, q, q_out, rope_freqs, positions, q_norm, k_norm, hists, hist_rows))

    def call():
        status = torch.empty_like(kv_len)
        out, o0, o1 = q_out, 0, 0
        if q is not None:
            if out is None:
                out = torch.empty_like(q)
            _, o0, o1 = _rows("q_out", out, dtype, tokens, dim)
        args = _APPEND.pack(k.data_ptr(), v.data_ptr(), k0, k1, v0, v1, _at(q), _at(out), q0, q1, o0, o1, _at(q_norm), _at(k_norm),
                            _at(rope_freqs), _at(positions), _at(hists), _at(hist_rows), q_heads, rot_dim, 1 if rope_interleaved else 0,
                            n_hists, rope_scale, eps)
        st = _LIB.sz_append_kv(kv, args, status.data_ptr(), _STREAM(dev))
        if st:
            _fail(st, "sz_append_kv")
        return out, status

    return _elsewhere(call, dev, stream) or call()


def _at(t):
    return 0 if t is None else t.data_ptr()


def _fail(st, where):
    from . import SzError
    raise SzError(st, where)


def paged_attention(q, k_pages, v_pages, page_table, q_begin, kv_len, *, scale=None, causal=True, window=0, out=None,
                    return_lse=False, workspace=None, stream=None):
    """Attention of the new tokens' queries (``q``: [tokens, query heads,
    channels]) over the paged cache; ``sz_paged_attention``.

    ``scale`` is 1/sqrt(channels) unless given.  ``causal``: a query sees the
    keys up to its own position; ``window`` > 0: only the last ``window`` of
    them.  A query that sees none gets zeros.  ``out`` may be ``q``; rows that
    belong to no request are left as they were.

    Returns (out, lse float32 [tokens, query heads] or None, status int32
    [requests])."""
    torch = _T or _load()
    shape, dtype = k_pages.shape, k_pages.dtype
    tokens, dim = q.shape[0], shape[-1]
    kv = _pack_kv(torch, k_pages, v_pages, shape, page_table, q_begin, kv_len, tokens)
    q_heads, q0, q1 = _rows("q", q, dtype, tokens, dim)
    if out is not None and out.shape != q.shape:
        raise ValueError("out of shape %s for q of %s" % (tuple(out.shape), tuple(q.shape)))
    if scale is None:
        scale = 1.0 / math.sqrt(dim)
    if window < 0 or window >= 1 << 32:
        raise ValueError("window must be 0 (none) or a number of keys below 2^32")
    dev = _device((k_pages, v_pages, q, page_table, q_begin, kv_len, out))

    def call():
        need = _attention_bytes(dim)
        ws = workspace
        if ws is None:
            ws = q.new_empty((need,), dtype=torch.uint8)
        else:
            from . import _workspace
            _workspace(ws, need, q.device)
        status = torch.empty_like(kv_len)
        o = torch.empty_like(q) if out is None else out
        _, o0, o1 = _rows("out", o, dtype, tokens, dim)
        lse = q.new_empty((tokens, q_heads), dtype=torch.float32) if return_lse else None
        args = _ATTENTION.pack(q.data_ptr(), o.data_ptr(), q0, q1, o0, o1, _at(lse), q_heads, 1 if causal else 0, window, scale)
        st = _LIB.sz_paged_attention(kv, args, status.data_ptr(), ws.data_ptr(), ws.nbytes, _STREAM(dev))
        if st:
            _fail(st, "sz_paged_attention")
        return o, lse, status

    return _elsewhere(call, dev, stream) or call()


@functools.lru_cache(maxsize=None)
def _attention_bytes(dim):
    from . import sz_plan_attention
    return sz_plan_attention(dim)


def rope_frequencies(rot_dim, base=10000.0, *, scaling=None, factor=1.0, trained_len=None, low_turns=1.0, high_turns=4.0, device=None):
    """Radians per position of each rotated pair, float64 [rot_dim / 2]:
    base^(-2t/rot_dim), and for contexts ``factor`` times the trained length

    * ``scaling="linear"``: every frequency divided by factor;
    * ``scaling="base"``: the base raised to base * factor^(R / (R - 2)), so
      that the slowest pair is divided by factor and the fastest kept;
    * ``scaling="bands"``: pairs that make fewer than low_turns turns over
      ``trained_len`` positions are divided by factor, pairs with more than
      high_turns are kept, and those between blend linearly in their turns."""
    import torch
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    t = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    if scaling == "base":
        if rot_dim <= 2:
            raise ValueError("scaling='base' needs more than one pair")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freqs = torch.pow(torch.tensor(float(base), dtype=torch.float64), -t / rot_dim)
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "bands":
        if trained_len is None:
            raise ValueError("scaling='bands' needs trained_len")
        turns = freqs * (trained_len / (2 * math.pi))
        keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0.0, 1.0)
        freqs = freqs * (keep + (1 - keep) / factor)
    elif scaling not in (None, "base"):
        raise ValueError("scaling is None, 'linear', 'base' or 'bands', got %r" % (scaling,))
    return freqs.to(device) if device is not None else freqs
