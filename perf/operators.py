"""Measured cases of the paged-cache operators: appending new keys and values
to a paged KV cache (head norms, position rotation and exponent counts on the
way) and attention of new tokens over that cache.

``own`` selects the framework's calls; otherwise ``run`` computes the same
results from elementary torch operations in 32 bits (angles in 64).

A cache layer is two tensors of pages, [pages, kv heads, page tokens, head
dim], and a table of page numbers per request.  Request r owns rows
q_begin[r] .. q_begin[r + 1] of the new tokens, and its cache holds kv_len[r]
tokens once they are in: new token i sits at position kv_len - new + i.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # ---- attention over the paged cache
        # one user of a chat, one new token over a short history: latency alone
        _attn("attn_token", 1, 1, 1, 333, 333, 32, 8),
        # a decode step of a serving batch: 64 requests of the paged workload's lengths
        _attn("attn_batch", 64, 1, 1, 128, 16384, 32, 8),
        # one request with a very long history: the split over the keys
        _attn("attn_long", 1, 1, 1, 131071, 131071, 64, 8),
        # several proposed tokens per request checked in one call, with the sums kept for a later join
        _attn("attn_verify", 16, 5, 5, 700, 8190, 64, 8, dtype="fp16", lse=True),
        # the last 4,096-token prefill chunk of the 32K-token cache
        _attn("attn_chunk", 1, 4096, 4096, 32768, 32768, 32, 8),
        # whole prompts of ragged lengths from an empty cache, a model of small heads
        _attn("attn_prompts", 6, 301, 2777, 0, 0, 16, 16, dim=64, dtype="fp16", page=64),
        # a 2,048-token chunk of a layer that looks back 4,096 tokens only
        _attn("attn_window", 1, 2048, 2048, 16001, 16001, 64, 8, window=4096),
        # ---- appending to the paged cache
        # a decode step: one token for each of 64 requests, queries rotated in the same pass
        _append("append_step", 64, 1, 1, 100, 600, 32, 8),
        # a 4,096-token prefill chunk with normalised heads
        _append("append_chunk", 1, 4096, 4096, 5000, 5000, 32, 8, norm=True),
        # ragged chunks, half of each head rotated, adjacent pairs
        _append("append_ragged", 7, 33, 1999, 2000, 4001, 16, 16, dtype="fp16", rotated=64, interleaved=True),
        # a layer without positions whose exponents are counted for the codec while it is written
        _append("append_counted", 3, 1000, 4096, 4096, 4500, 0, 8, rotated=0, counted=True),
        # positions far out in a long context, many heads
        _append("append_far", 2, 2048, 2048, 2500, 3001, 64, 8, first=900000),
    ]


def draw(rng):
    heads, kv_heads = rng.choice([(32, 8), (64, 8), (16, 16), (28, 4), (8, 1), (12, 4)])
    common = dict(dim=rng.choice([64, 128, 128]), dtype=rng.choice(["bf16", "fp16"]), page=rng.choice([16, 16, 32, 64]))
    mix = rng.randrange(1 << 20)
    if rng.random() < 0.6:
        kind = rng.choice(["token", "verify", "chunk", "prompts"])
        if kind == "chunk":
            n = _spread(rng, 1, 4)
            lo_q = _spread(rng, 16, 4096)
            lo_kv = _spread(rng, lo_q, 32768)
        elif kind == "prompts":
            n = _spread(rng, 1, 8)
            lo_q, lo_kv = _spread(rng, 16, 4096), 0
        else:
            n = _spread(rng, 1, 64)
            lo_q = 1 if kind == "token" else rng.randrange(2, 9)
            lo_kv = _spread(rng, max(lo_q, 16), 131072)
        hi_q = lo_q if kind in ("token", "verify") else max(lo_q, int(lo_q * rng.uniform(1, 2)))
        hi_kv = int(lo_kv * rng.uniform(1, 4))
        while True:
            case = _attn("drawn", n, lo_q, hi_q, lo_kv, hi_kv, heads, kv_heads, window=0, lse=mix % 3 == 0, mix=mix, **common)
            q, kv = lengths(case)
            scores, keys = n * max(q) * heads * max(kv), n * max(kv) * kv_heads * case["dim"]
            cost = work(case)
            if scores <= 4096 * 32 * 32768 and keys <= 64 * 16384 * 8 * 128 and cost["flops"] <= 2e12 and cost["bytes"] <= 7e8:
                break
            if n > 1:
                n -= 1
            else:
                lo_q, hi_q, lo_kv, hi_kv = (x if x <= 8 else x * 7 // 8 for x in (lo_q, hi_q, lo_kv, hi_kv))
        if kind in ("token", "chunk") and rng.random() < 0.3:
            case["window"] = _spread(rng, 100, 8192)
    else:
        n = _spread(rng, 1, 64)
        lo_q = _spread(rng, 1, max(1, 4096 // n))
        hi_q = max(lo_q, int(lo_q * rng.uniform(1, 2)))
        rotated = rng.choice([0, common["dim"] // 2, common["dim"], common["dim"]])
        case = _append("drawn", n, lo_q, hi_q, hi_q, 2 * hi_q + 64, heads if rng.random() < 0.8 else 0, kv_heads, rotated=rotated,
                       interleaved=rng.random() < 0.4, norm=rotated > 0 and rng.random() < 0.5, counted=rotated == 0,
                       first=rng.choice([0, 0, _spread(rng, 1000, 1000000)]), mix=mix, **common)
    del case["name"]
    return case


def _spread(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _attn(name, requests, lo_q, hi_q, lo_kv, hi_kv, heads, kv_heads, dim=128, dtype="bf16", page=16, window=0, lse=False, mix=1):
    return {"name": name, "op": "attention", "requests": requests, "lo_q": lo_q, "hi_q": hi_q, "lo_kv": lo_kv, "hi_kv": hi_kv, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "page": page, "window": window, "lse": lse, "mix": mix}


def _append(name, requests, lo_q, hi_q, lo_kv, hi_kv, heads, kv_heads, dim=128, dtype="bf16", page=16, rotated=128, interleaved=False,
            norm=False, counted=False, first=0, mix=1):
    return {"name": name, "op": "append", "requests": requests, "lo_q": lo_q, "hi_q": hi_q, "lo_kv": lo_kv, "hi_kv": hi_kv, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "page": page, "rotated": rotated, "interleaved": interleaved, "norm": norm,
            "counted": counted, "first": first, "mix": mix}


def lengths(case):
    """New tokens and cached tokens (the new ones included) of each request.  lo_kv = 0: nothing but the new tokens."""
    rng = random.Random(case["mix"])
    q, kv = [], []
    for _ in range(case["requests"]):
        a = _spread(rng, case["lo_q"], case["hi_q"])
        q.append(a)
        kv.append(a if case["lo_kv"] == 0 else max(a, _spread(rng, case["lo_kv"], max(case["lo_kv"], case["hi_kv"]))))
    return q, kv


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev, dtype = "cuda", TYPES[case["dtype"]]
    q_len, kv_len = lengths(case)
    n, page, dim, kv_heads = case["requests"], case["page"], case["dim"], case["kv_heads"]
    need = [-(-v // page) for v in kv_len]
    pages = sum(need) + 3  # a few pages of the pool belong to nobody

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    # requests hold scattered pages; entries behind a request's last page are -1
    order = torch.randperm(pages, generator=gen, device=dev)[: sum(need)].tolist()
    table = torch.full((n, max(need)), -1, dtype=torch.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = torch.tensor(order[at: at + m], dtype=torch.int32)
        at += m
    starts = [0]
    for v in q_len:
        starts.append(starts[-1] + v)
    tokens = starts[-1]
    state = {
        "case": dict(case), "tokens": tokens, "max_q": max(q_len), "max_kv": max(kv_len),
        "page_table": table.to(dev), "q_begin": torch.tensor(starts, dtype=torch.int32, device=dev),
        "kv_len": torch.tensor(kv_len, dtype=torch.int32, device=dev),
        # pages as the codec's paged workload holds them: channels and heads of different sizes
        "k_pages": normal(pages, kv_heads, page, dim), "v_pages": normal(pages, kv_heads, page, dim),
    }
    sizes = torch.exp2(torch.rand((kv_heads, 1, dim), generator=gen, device=dev) * 2 - 1).to(dtype)
    state["k_pages"].mul_(sizes)
    if case["op"] == "attention":
        state["q"] = normal(tokens, case["heads"], dim, scale=2.0)
        state["scale"] = 1.0 / math.sqrt(dim)
        return state
    # the projections' output: one row of q, k and v heads per token, read in place
    heads = case["heads"]
    row = normal(tokens, heads + 2 * kv_heads, dim)
    state["q"] = row[:, :heads] if heads else None
    state["k"], state["v"] = row[:, heads: heads + kv_heads], row[:, heads + kv_heads:]
    state["k"].mul_(sizes.reshape(kv_heads, dim))
    state["positions"] = state["freqs"] = state["q_norm"] = state["k_norm"] = None
    if case["first"]:
        place = [kv_len[r] - q_len[r] + i + case["first"] for r in range(n) for i in range(q_len[r])]
        state["positions"] = torch.tensor(place, dtype=torch.int64, device=dev)
    if case["rotated"]:
        rd = case["rotated"]
        state["freqs"] = 500000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=dev) / rd)
    if case["norm"]:
        state["k_norm"] = (1 + 0.2 * torch.randn(dim, generator=gen, device=dev)).to(dtype)
        if heads:
            state["q_norm"] = (1 + 0.2 * torch.randn(dim, generator=gen, device=dev)).to(dtype)
    return state


def run(state):
    c = state["case"]
    if own:
        import lossless_bf16_kv_splitzip_b200 as sz
        if c["op"] == "attention":
            out, lse, _ = sz.paged_attention(state["q"], state["k_pages"], state["v_pages"], state["page_table"], state["q_begin"],
                                             state["kv_len"], scale=state["scale"], window=c["window"], return_lse=c["lse"])
            return {"out": out, "lse": lse}
        hists = torch.zeros((2 * c["requests"], 256), dtype=torch.int32, device="cuda") if c["counted"] else None
        q, _ = sz.append_kv(state["k"], state["v"], state["k_pages"], state["v_pages"], state["page_table"], state["q_begin"],
                            state["kv_len"], q=state["q"], rope_freqs=state["freqs"], rope_interleaved=c["interleaved"],
                            positions=state["positions"], q_norm=state["q_norm"], k_norm=state["k_norm"], eps=1e-6, hists=hists)
        return {"q": q, "k_pages": state["k_pages"], "v_pages": state["v_pages"], "hists": hists}
    if c["op"] == "attention":
        return _attention_plain(state, c)
    return _append_plain(state, c)


def _places(state):
    """Request, index within the request and cache position of every new token."""
    begin, length = state["q_begin"].long(), state["kv_len"].long()
    token = torch.arange(state["tokens"], device=begin.device)
    req = torch.searchsorted(begin, token, right=True) - 1
    index = token - begin[req]
    return req, index, length[req] - (begin[req + 1] - begin[req]) + index


def _attention_plain(state, c):
    heads, kv_heads, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    group, n, Q, T = heads // kv_heads, c["requests"], state["max_q"], state["max_kv"]
    begin, length = state["q_begin"].long(), state["kv_len"].long()
    new = begin[1:] - begin[:-1]
    dev = begin.device
    # every request padded to the longest: [requests, kv heads, group, new, keys]
    i = torch.arange(Q, device=dev)
    rows = (begin[:-1, None] + i).clamp(max=state["tokens"] - 1)
    q = state["q"][rows].float().mul_(state["scale"])
    q = q.view(n, Q, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(n, kv_heads, group * Q, dim)
    slots = state["page_table"].long().clamp(min=0)
    k = state["k_pages"][slots].permute(0, 2, 1, 3, 4).reshape(n, kv_heads, -1, dim)[:, :, :T].float()
    s = torch.matmul(q, k.transpose(2, 3)).view(n, kv_heads, group, Q, T)
    del k
    place = (length - new)[:, None] + i
    j = torch.arange(T, device=dev)
    seen = (j <= place[:, :, None]) & (j < length[:, None, None])
    if c["window"]:
        seen &= j > place[:, :, None] - c["window"]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = state["v_pages"][slots].permute(0, 2, 1, 3, 4).reshape(n, kv_heads, -1, dim)[:, :, :T].float()
    o = torch.matmul(p.view(n, kv_heads, group * Q, T), v).view(n, kv_heads, group, Q, dim)
    o = torch.where(total > 0, o / total, 0.0)
    req, index, _ = _places(state)
    out = o.permute(0, 3, 1, 2, 4).reshape(n, Q, heads, dim)[req, index].to(state["q"].dtype)
    lse = None
    if c["lse"]:
        lse = (m + total.log()).view(n, heads, Q).permute(0, 2, 1)[req, index]
    return {"out": out, "lse": lse}


def _norm_rotate(x, weight, cos, sin, c):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    if cos is not None:
        rd = c["rotated"]
        a, b = (y[..., 0:rd:2], y[..., 1:rd:2]) if c["interleaved"] else (y[..., : rd // 2], y[..., rd // 2: rd])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        y = torch.cat((turned, y[..., rd:]), -1)
    return y.to(x.dtype)


def _append_plain(state, c):
    req, _, place = _places(state)
    cos = sin = None
    if c["rotated"]:
        turn = state["positions"] if state["positions"] is not None else place
        angle = (turn.double()[:, None] * state["freqs"])[:, None]
        cos, sin = angle.cos().float(), angle.sin().float()
    k, v = _norm_rotate(state["k"], state["k_norm"], cos, sin, c), state["v"]
    slot = state["page_table"][req, place // c["page"]].long()
    state["k_pages"][slot, :, place % c["page"]] = k
    state["v_pages"][slot, :, place % c["page"]] = v
    q = _norm_rotate(state["q"], state["q_norm"], cos, sin, c) if state["q"] is not None else None
    hists = None
    if c["counted"]:
        hists = torch.zeros(2 * c["requests"] * 256, dtype=torch.int32, device="cuda")
        both = torch.stack((k, v)).view(torch.int16).int()
        row = torch.stack((req, req + c["requests"]))[:, :, None, None]
        at = (row * 256 + ((both >> 7) & 255)).reshape(-1)
        hists = hists.index_add_(0, at, torch.ones_like(at, dtype=torch.int32)).view(-1, 256)
    return {"q": q, "k_pages": state["k_pages"], "v_pages": state["v_pages"], "hists": hists}


def work(case):
    q_len, kv_len = lengths(case)
    heads, kv_heads, dim, window = case["heads"], case["kv_heads"], case["dim"], case.get("window", 0)
    tokens = sum(q_len)
    if case["op"] == "append":
        rows = 2 * tokens * (heads + 2 * kv_heads) * dim * 2  # q, k and v in, q and the cache rows out
        counts = 2 * case["requests"] * 256 * 4 if case["counted"] else 0
        turned = tokens * (heads + kv_heads)
        flops = turned * (3 * case["rotated"] + (4 * dim if case["norm"] else 0))
        return {"bytes": rows + counts + (8 * tokens if case["first"] else 0), "flops": flops}
    pairs = keys = 0
    for q, kv in zip(q_len, kv_len):
        first = kv - q  # position of the first new token
        full = q * (q + 1) // 2 + q * first
        cut = 0
        if window:  # keys that lie behind the window, summed over the queries
            a, b = max(0, first + 1 - window), max(0, kv - window)
            cut = (b * (b + 1) - max(0, a - 1) * a) // 2 if b else 0
            keys += kv - max(0, first + 1 - window)
        else:
            keys += kv
        pairs += full - cut
    bytes_ = 2 * keys * kv_heads * dim * 2 + 2 * tokens * heads * dim * 2 + (4 * tokens * heads if case["lse"] else 0)
    return {"bytes": bytes_, "flops": 4 * pairs * heads * dim}


def exact(case, seed):
    s = prepare(case, seed)
    q_len, kv_len = lengths(case)
    page, heads, kv_heads, dim = case["page"], case["heads"], case["kv_heads"], case["dim"]
    table = s["page_table"].long()
    if case["op"] == "attention":
        group = heads // kv_heads
        out = torch.zeros((s["tokens"], heads, dim), dtype=torch.float64, device="cuda")
        lse = torch.full((s["tokens"], heads), -math.inf, dtype=torch.float64, device="cuda")
        at = 0
        for r, (nq, nk) in enumerate(zip(q_len, kv_len)):
            slots = table[r, : -(-nk // page)]
            where = torch.arange(nk, device="cuda")[None] - torch.arange(nk - nq, nk, device="cuda")[:, None]  # key minus query
            hidden = where > 0
            if case["window"]:
                hidden |= where <= -case["window"]
            for h in range(heads):
                key = s["k_pages"][slots, h // group].reshape(-1, dim)[:nk].double()
                val = s["v_pages"][slots, h // group].reshape(-1, dim)[:nk].double()
                score = s["q"][at: at + nq, h].double() @ key.T / math.sqrt(dim)
                score[hidden] = -math.inf
                total = torch.logsumexp(score, 1)
                out[at: at + nq, h] = torch.exp(score - total[:, None]) @ val
                lse[at: at + nq, h] = total
            at += nq
        return {"out": out, "lse": lse if case["lse"] else None}

    def turned(x, weight, angle):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / dim + 1e-6) * weight.double()
        rd = case["rotated"]
        if rd:
            first = torch.arange(0, rd, 2, device="cuda") if case["interleaved"] else torch.arange(rd // 2, device="cuda")
            second = first + (1 if case["interleaved"] else rd // 2)
            z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None]
            x = x.clone()
            x[..., first], x[..., second] = z.real, z.imag
        return x

    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    q_out = torch.zeros((s["tokens"], heads, dim), dtype=torch.float64, device="cuda") if heads else None
    hists = torch.zeros((2 * case["requests"], 256), dtype=torch.int64) if case["counted"] else None
    at = 0
    for r, (nq, nk) in enumerate(zip(q_len, kv_len)):
        here = torch.arange(nk - nq, nk, device="cuda")
        angle = None
        if case["rotated"]:
            angle = (here + case["first"]).double()[:, None] * s["freqs"]
        k, v = turned(s["k"][at: at + nq], s["k_norm"], angle), s["v"][at: at + nq].double()
        slots = table[r, here // page]
        kp[slots, :, here % page], vp[slots, :, here % page] = k, v
        if heads:
            q_out[at: at + nq] = turned(s["q"][at: at + nq], s["q_norm"], angle)
        if case["counted"]:
            for row, x in ((r, s["k"]), (case["requests"] + r, s["v"])):
                bits = x[at: at + nq].contiguous().view(torch.int16).to(torch.int64) & 0x7FFF
                hists[row] = torch.bincount((bits >> 7).reshape(-1), minlength=256).cpu()
        at += nq
    return {"q": q_out, "k_pages": kp, "v_pages": vp, "hists": hists.int() if hists is not None else None}
