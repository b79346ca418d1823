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

import math
import struct

_KV = struct.Struct("<9Q4I4Q2IQ")  # sz_paged_kv
_APPEND = struct.Struct("<18Q4I2f")  # sz_append_args
_ATTENTION = struct.Struct("<7Q3If")  # sz_attention_args

_TYPES: dict = {}


def _torch():
    import torch
    if not _TYPES:
        _TYPES[torch.bfloat16] = 1
        _TYPES[torch.float16] = 2
    return torch


def _ints(name, t, ndim, torch):
    if t.dtype != torch.int32 or t.dim() != ndim or t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("%s must be an int32 tensor of %d dimension(s) with entries side by side" % (name, ndim))
    return t


def _rows(name, t, dtype, tokens, dim):
    if t.dtype != dtype or t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != dim:
        raise ValueError("%s must be %s [%d tokens, heads, %d], got %s %s" % (name, dtype, tokens, dim, t.dtype, tuple(t.shape)))
    s = t.stride()
    if s[2] != 1:
        raise ValueError("%s needs its channels side by side" % name)
    if t.requires_grad:
        raise ValueError("%s requires a gradient, and this operator has none" % name)
    return s


def _pack_kv(torch, k_pages, v_pages, page_table, q_begin, kv_len, tokens):
    code = _TYPES.get(k_pages.dtype)
    if code is None or v_pages.dtype != k_pages.dtype:
        raise TypeError("pages are bfloat16 or float16, the same for keys and values; got %s and %s" % (k_pages.dtype, v_pages.dtype))
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("pages are two tensors [pages, heads, page tokens, channels] of one shape")
    ks, vs = k_pages.stride(), v_pages.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("pages need their channels side by side")
    _ints("page_table", page_table, 2, torch)
    _ints("q_begin", q_begin, 1, torch)
    _ints("kv_len", kv_len, 1, torch)
    reqs, max_pages = page_table.shape
    if q_begin.shape[0] != reqs + 1 or kv_len.shape[0] != reqs:
        raise ValueError("%d requests in page_table, %d in q_begin, %d in kv_len" % (reqs, q_begin.shape[0] - 1, kv_len.shape[0]))
    return _KV.pack(k_pages.data_ptr(), v_pages.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], shape[0], shape[1], shape[3],
                    shape[2], code, page_table.data_ptr(), page_table.stride(0) if reqs > 1 else max_pages, q_begin.data_ptr(),
                    kv_len.data_ptr(), reqs, max_pages, tokens)


class _On:
    """The device and stream of one call: the tensors' device made current,
    and the given stream, if any."""

    def __init__(self, torch, tensors, stream):
        dev = tensors[0].device
        for t in tensors:
            if t is not None and t.device != dev:
                raise ValueError("tensors on %s and %s" % (dev, t.device))
        if dev.type != "cuda":
            raise ValueError("the tensors must be on a CUDA device, not on %s" % dev)
        self.guards = []
        if torch.cuda.current_device() != dev.index:
            self.guards.append(torch.cuda.device(dev))
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=dev)
            if stream.device != dev:
                raise ValueError("a stream of %s for tensors on %s" % (stream.device, dev))
            self.guards.append(torch.cuda.stream(stream))
        self.stream = stream
        self.dev = dev
        self.torch = torch

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self.dev, (self.stream or self.torch.cuda.current_stream(self.dev)).cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


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
    torch = _torch()
    tokens, dim, dtype = k.shape[0], k_pages.shape[-1], k_pages.dtype
    kv = _pack_kv(torch, k_pages, v_pages, page_table, q_begin, kv_len, tokens)
    ks, vs = _rows("k", k, dtype, tokens, dim), _rows("v", v, dtype, tokens, dim)
    if k.shape[1] != k_pages.shape[1] or v.shape[1] != k_pages.shape[1]:
        raise ValueError("pages of %d heads, k of %d, v of %d" % (k_pages.shape[1], k.shape[1], v.shape[1]))
    qs, q_heads = (0, 0, 0), 0
    if q is not None:
        qs, q_heads = _rows("q", q, dtype, tokens, dim), q.shape[1]
        if q_out is not None and q_out.shape != q.shape:
            raise ValueError("q_out of shape %s for q of %s" % (tuple(q_out.shape), tuple(q.shape)))
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm need q")
    rot_dim = 0
    if rope_freqs is not None:
        if rope_freqs.dtype != torch.float64 or rope_freqs.dim() != 1 or not rope_freqs.is_contiguous():
            raise ValueError("rope_freqs must be a contiguous float64 vector")
        rot_dim = 2 * rope_freqs.shape[0]
    if positions is not None and (positions.dtype != torch.int64 or positions.shape != (tokens,) or not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous int64 tensor [%d]" % tokens)
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None and (w.dtype != dtype or w.shape != (dim,) or not w.is_contiguous()):
            raise ValueError("%s must be a contiguous %s tensor [%d]" % (name, dtype, dim))
    n_hists = 0
    if hists is not None:
        if hists.dtype not in (torch.int32, torch.uint32) or hists.shape[-1] != 256 or not hists.is_contiguous():
            raise ValueError("hists must be a contiguous 32-bit tensor of rows of 256 counts")
        n_hists = hists.numel() // 256
    if hist_rows is not None:
        if hists is None:
            raise ValueError("hist_rows needs hists")
        if hist_rows.dtype not in (torch.int32, torch.uint32) or hist_rows.numel() != 2 * kv_len.shape[0] or not hist_rows.is_contiguous():
            raise ValueError("hist_rows must be a contiguous 32-bit tensor of %d rows" % (2 * kv_len.shape[0]))
    from . import _check, lib
    with _On(torch, (k_pages, v_pages, k, v, page_table, q_begin, kv_len, q, q_out, rope_freqs, positions, q_norm, k_norm, hists,
                     hist_rows), stream) as (dev, s):
        status = torch.empty(kv_len.shape[0], dtype=torch.int32, device=dev)
        qos = (0, 0, 0)
        if q is not None:
            if q_out is None:
                q_out = torch.empty((tokens, q_heads, dim), dtype=dtype, device=dev)
            qos = _rows("q_out", q_out, dtype, tokens, dim)

        def at(t):
            return 0 if t is None else t.data_ptr()

        args = _APPEND.pack(k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1], at(q), at(q_out), qs[0], qs[1], qos[0], qos[1],
                            at(q_norm), at(k_norm), at(rope_freqs), at(positions), at(hists), at(hist_rows), q_heads, rot_dim,
                            1 if rope_interleaved else 0, n_hists, rope_scale, eps)
        _check(lib().sz_append_kv(kv, args, status.data_ptr(), s), "sz_append_kv")
    return q_out, status


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
    torch = _torch()
    tokens, dim, dtype = q.shape[0], k_pages.shape[-1], k_pages.dtype
    kv = _pack_kv(torch, k_pages, v_pages, page_table, q_begin, kv_len, tokens)
    qs, q_heads = _rows("q", q, dtype, tokens, dim), q.shape[1]
    if out is not None and out.shape != q.shape:
        raise ValueError("out of shape %s for q of %s" % (tuple(out.shape), tuple(q.shape)))
    if scale is None:
        scale = 1.0 / math.sqrt(dim)
    if window < 0 or window >= 1 << 32:
        raise ValueError("window must be 0 (none) or a number of keys below 2^32")
    from . import _check, _nbytes, _workspace, lib, sz_plan_attention
    with _On(torch, (k_pages, v_pages, q, page_table, q_begin, kv_len, out), stream) as (dev, s):
        ws = _workspace(workspace, sz_plan_attention(dim), dev)
        status = torch.empty(kv_len.shape[0], dtype=torch.int32, device=dev)
        if out is None:
            out = torch.empty((tokens, q_heads, dim), dtype=dtype, device=dev)
        os_ = _rows("out", out, dtype, tokens, dim)
        lse = torch.empty((tokens, q_heads), dtype=torch.float32, device=dev) if return_lse else None
        args = _ATTENTION.pack(q.data_ptr(), out.data_ptr(), qs[0], qs[1], os_[0], os_[1], lse.data_ptr() if return_lse else 0, q_heads,
                               1 if causal else 0, window, scale)
        _check(lib().sz_paged_attention(kv, args, status.data_ptr(), ws.data_ptr(), _nbytes(ws), s), "sz_paged_attention")
    return out, lse, status


def rope_frequencies(rot_dim, base=10000.0, *, scaling=None, factor=1.0, trained_len=None, low_turns=1.0, high_turns=4.0, device=None):
    """Radians per position of each rotated pair, float64 [rot_dim / 2]:
    base^(-2t/rot_dim), and for contexts ``factor`` times the trained length

    * ``scaling="linear"``: every frequency divided by factor;
    * ``scaling="base"``: the base raised to base * factor^(R / (R - 2)), so
      that the slowest pair is divided by factor and the fastest kept;
    * ``scaling="bands"``: pairs that make fewer than low_turns turns over
      ``trained_len`` positions are divided by factor, pairs with more than
      high_turns are kept, and those between blend linearly in their turns."""
    torch = _torch()
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
