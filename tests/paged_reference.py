"""Plain 64-bit definitions of the paged-cache operators, on the CPU, with
the error bounds that their 32-bit and 16-bit steps allow."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # rounding of a result, relative: eps / 2 of 2^-7, 2^-10
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half a step among the subnormals


def gather(pages, table_row, n):
    """Token-major [n, heads, dim] float64 of one request."""
    P = pages.shape[2]
    out = torch.zeros((n, pages.shape[1], pages.shape[3]), dtype=torch.float64)
    for j in range(n):
        out[j] = pages[int(table_row[j // P]), :, j % P].double()
    return out


def attention(q, k_pages, v_pages, table, q_begin, kv_len, scale, causal=True, window=0):
    """-> (out, lse, tol_out, tol_lse), float64.  Rows of no request: NaN in
    out and tol (not to be compared).

    Bounds, with u = 2^-24.  A score is a sum of D products in 32 bits, in
    some order and possibly truncated: off by at most 2 D u sum|q k| scale,
    then multiplied by two factors and reduced by the maximum (3 u |s| each
    side); the exponential adds 4 u.  So a weight is off by the factor
    1 + d, d = 2 u (2 D A + 6 A + 4), A the row's largest scale * sum |q k|.
    Weights meet the values in 16 bits (half a step h each, or half a
    subnormal step against a sum of at least 1/2^8); sum and numerator each
    carry d, the accumulators n u: |do| <= (h + 2 d + 2 n u) sum w|v| +
    2^8 tiny sum|v|, and the result is rounded once more."""
    h, tiny, u = HALF_STEP[q.dtype], TINY[q.dtype], 2.0 ** -24
    N, Hq, D = q.shape
    Hk = k_pages.shape[1]
    G = Hq // Hk
    out = torch.full((N, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((N, Hq), math.nan, dtype=torch.float64)
    tol, tol_l = torch.full_like(out, math.nan), torch.full_like(lse, math.nan)
    for r in range(len(kv_len)):
        a, b, L = int(q_begin[r]), int(q_begin[r + 1]), int(kv_len[r])
        n = b - a
        if n == 0:
            continue
        lo = max(0, L - n + 1 - window) if window else 0
        K, V = torch.zeros((L, Hk, D), dtype=torch.float64), torch.zeros((L, Hk, D), dtype=torch.float64)
        P = k_pages.shape[2]
        for j in range(lo, L):
            K[j], V[j] = k_pages[int(table[r, j // P]), :, j % P].double(), v_pages[int(table[r, j // P]), :, j % P].double()
        p = torch.arange(L - n, L)[:, None]
        j = torch.arange(L)[None]
        seen = torch.ones((n, L), dtype=torch.bool)
        if causal:
            seen &= j <= p
        if window:
            seen &= j > p - window
        some = seen.any(1)
        for hq in range(Hq):
            x = q[a:b, hq].double()
            s = (x @ K[:, hq // G].T) * scale
            mag = (x.abs() @ K[:, hq // G].abs().T) * abs(scale)
            s = s.masked_fill(~seen, -math.inf)
            A = mag.masked_fill(~seen, 0.0).amax(1) if L else torch.zeros(n, dtype=torch.float64)
            l = torch.logsumexp(s, 1) if L else torch.full((n,), -math.inf, dtype=torch.float64)
            w = torch.exp(s - l[:, None])
            w = torch.where(seen, w, 0.0)
            o = w @ V[:, hq // G]
            wv = w @ V[:, hq // G].abs()
            d = 2 * u * (2 * D * A + 6 * A + 4)
            t = (h + 2 * d + 2 * L * u)[:, None] * wv + 2 ** 8 * tiny * V[:, hq // G].abs().sum(0)
            out[a:b, hq] = torch.where(some[:, None], o, 0.0)
            tol[a:b, hq] = torch.where(some[:, None], t + h * (o.abs() + t) + tiny, 0.0)
            lse[a:b, hq] = torch.where(some, l, -math.inf)
            tol_l[a:b, hq] = torch.where(some, d + L * u + 8 * u * (1 + l.abs()), 0.0)
    return out, lse, tol, tol_l


def turned(x, weight, eps, freqs, positions, interleaved, scale):
    """Norm and rotation of [tokens, heads, dim] in 64 bits -> (y, tol).

    Bounds, u = 2^-24: the norm's sum, reciprocal root and two products are
    off by (D/2 + 8) u at most; a pair's angle (reduced in 64 bits) by half a
    step of a number below 2 pi, its sine and cosine by 4 u, so the turned
    value by 16 u (|a| + |b|) on top of the norm's share; then one rounding."""
    h, tiny, u = HALF_STEP[x.dtype], TINY[x.dtype], 2.0 ** -24
    D = x.shape[-1]
    y = x.double()
    rel = 0.0
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * weight.double()
        rel = (D / 2 + 8) * u
    mag = y.abs()
    if freqs is not None:
        R = 2 * freqs.numel()
        t = torch.arange(R // 2)
        first, second = (2 * t, 2 * t + 1) if interleaved else (t, t + R // 2)
        angle = positions.double()[:, None, None] * freqs.double()
        c, s = angle.cos(), angle.sin()
        a, b = y[..., first], y[..., second]
        y, mag = y.clone(), mag.clone()
        y[..., first], y[..., second] = (a * c - b * s) * scale, (b * c + a * s) * scale
        mag[..., first] = mag[..., second] = (a.abs() + b.abs()) * abs(scale)
        rel += 16 * u
    off = rel * mag
    if weight is None and freqs is None:
        return y, torch.zeros_like(y)
    return y, off + h * (y.abs() + off) + tiny
