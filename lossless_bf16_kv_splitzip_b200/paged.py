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
status tensor with one word per request.  Neither has a gradient: where
gradients are recorded, tensors that require one are refused, and tensors that
carry a tangent everywhere.
"""
from __future__ import annotations

import functools
import math
import threading

_BINDING = None
_LOADING = threading.Lock()


def binding():
    """The compiled part (csrc/sz_binding.cpp), which checks the arguments,
    allocates the results and calls the library; built in-tree if missing."""
    global _BINDING
    with _LOADING:
        if _BINDING is None:
            import ctypes

            import torch  # noqa: F401  its libraries come first

            from . import lib
            from ._build import build_binding
            build_binding()
            from . import _binding
            loaded = lib()
            _binding.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (loaded.sz_append_kv, loaded.sz_paged_attention)))
            _BINDING = _binding
    return _BINDING


def _raise(status, where):
    from . import SzError
    raise SzError(status, where)


def _handle(stream, tensor):
    """The raw handle of a stream argument."""
    if isinstance(stream, int):
        return stream
    if stream.device != tensor.device:
        raise ValueError("a stream of %s for tensors on %s" % (stream.device, tensor.device))
    return stream.cuda_stream


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
    st, out, status = (_BINDING or binding()).append_kv(
        k, v, k_pages, v_pages, page_table, q_begin, kv_len, q, q_out, rope_freqs, rope_interleaved, rope_scale, positions, q_norm, k_norm,
        eps, hists, hist_rows, stream if stream is None else _handle(stream, k))
    if st:
        _raise(st, "sz_append_kv")
    return out, status


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
    st, o, lse, status = (_BINDING or binding()).paged_attention(
        q, k_pages, v_pages, page_table, q_begin, kv_len, scale, causal, window, out, return_lse, workspace,
        _attention_bytes(k_pages.shape[-1]), stream if stream is None else _handle(stream, q))
    if st:
        _raise(st, "sz_paged_attention")
    return o, lse, status


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
