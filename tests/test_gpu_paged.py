"""The paged-cache operators on the GPU against their 64-bit definitions
(tests/paged_reference.py gives the values and the error bounds)."""
import math
import random

import numpy as np
import pytest

import paged_reference as ref

torch = pytest.importorskip("torch")
import lossless_bf16_kv_splitzip_b200 as sz  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda:0"
BF16, FP16 = torch.bfloat16, torch.float16


class Batch:
    """Random requests over scattered pages of a host copy of the cache; what
    lies behind a request's end, in pages nobody owns and behind the last row
    is NaN."""

    def __init__(self, new, kv, heads, kv_heads, dim, page, dtype, seed=0, extra_rows=0, extra_pages=2, width=None):
        g = torch.Generator().manual_seed(1000 + seed)
        self.new, self.kv, self.heads, self.page, self.dtype = list(new), list(kv), heads, page, dtype
        need = [-(-max(n, 0) // page) for n in kv]
        total = sum(need) + extra_pages
        self.k = torch.full((total, kv_heads, page, dim), math.nan, dtype=dtype)
        self.v = self.k.clone()
        order = list(range(total))
        random.Random(seed).shuffle(order)
        width = max(need + [1]) if width is None else width
        self.table = torch.full((len(kv), width), -1, dtype=torch.int32)
        for r, m in enumerate(need):
            for i in range(m):
                p = order.pop()
                self.table[r, i] = p
                t = min(page, kv[r] - i * page)
                self.k[p, :, :t] = torch.randn((kv_heads, t, dim), generator=g).to(dtype)
                self.v[p, :, :t] = torch.randn((kv_heads, t, dim), generator=g).to(dtype)
        self.q_begin = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.kv_len = torch.tensor(list(kv), dtype=torch.int32)
        self.rows = int(self.q_begin[-1]) + extra_rows
        self.q = (1.5 * torch.randn((self.rows, heads, dim), generator=g)).to(dtype)
        self.g = g

    def cache(self):
        return [t.to(DEV) for t in (self.k, self.v, self.table, self.q_begin, self.kv_len)]


def check(got, want, tol, what=""):
    got = got.cpu().double()
    use = ~torch.isnan(tol)
    assert bool(torch.isfinite(got[use]).all() | ~torch.isfinite(want[use]).all()), what + ": not finite"
    same = got == want  # infinities
    over = ((got - want).abs() - tol)[use & ~same]
    assert over.numel() == 0 or float(over.max()) <= 0, "%s: %g over its bound, %d of %d values" % (
        what, float(over.max()), int((over > 0).sum()), over.numel())


def attend_and_check(b, causal=True, window=0, scale=None, **kw):
    k, v, table, q_begin, kv_len = b.cache()
    q = b.q.to(DEV)
    out, lse, status = sz.paged_attention(q, k, v, table, q_begin, kv_len, scale=scale, causal=causal, window=window, return_lse=True, **kw)
    torch.cuda.synchronize()
    assert status.cpu().tolist() == [0] * len(b.kv)
    want = ref.attention(b.q, b.k, b.v, b.table, b.q_begin, b.kv_len, scale or 1 / math.sqrt(b.q.shape[2]), causal, window)
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")
    return out, lse


SHAPES = [  # new tokens, cached tokens, query heads, KV heads, dim, page, type
    ([1], [1], 4, 4, 64, 16, BF16),
    ([1], [17], 32, 8, 128, 16, BF16),
    ([1, 1, 1], [5, 300, 128], 8, 1, 128, 16, FP16),
    ([1, 0, 3, 1], [40, 33, 3, 0], 8, 2, 64, 32, BF16),  # no new token; only new tokens; nothing cached
    ([5, 5], [130, 515], 64, 8, 128, 16, FP16),
    ([7], [7], 7, 1, 64, 8, BF16),  # a group of seven
    ([129], [129], 2, 2, 128, 16, BF16),
    ([257, 1, 64], [400, 257, 64], 4, 2, 128, 64, FP16),
    ([300], [555], 12, 4, 64, 128, BF16),
    ([33, 31], [129, 128], 28, 4, 128, 256, BF16),
    ([40], [1000], 16, 1, 128, 24, FP16),  # pages that do not divide a tile
    ([3, 9], [77, 9], 6, 2, 80, 16, BF16),
    ([2, 30], [50, 31], 4, 1, 256, 16, FP16),
    ([4], [21], 2, 1, 8, 5, BF16),
    ([6, 1], [13, 29], 4, 2, 128, 1, FP16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:6])).replace(" ", ""))
@pytest.mark.parametrize("mode", ["causal", "full", "window"])
def test_attention(shape, mode):
    new, kv, hq, hk, dim, page, dtype = shape
    attend_and_check(Batch(new, kv, hq, hk, dim, page, dtype), causal=mode != "full", window=37 if mode == "window" else 0)


@pytest.mark.parametrize("window", [1, 16, 127, 128, 129, 1000])
def test_attention_windows(window):
    attend_and_check(Batch([200, 1, 3], [333, 401, 500], 8, 2, 64, 16, BF16, seed=window), window=window)


@pytest.mark.parametrize("hq,hk,dim,dtype", [(4, 1, 128, BF16), (16, 4, 64, FP16), (2, 2, 128, FP16)])
def test_attention_of_long_rows(hq, hk, dim, dtype):
    # few rows over many keys: the keys are split over the whole GPU
    attend_and_check(Batch([1, 2], [9001, 2300], hq, hk, dim, 16, dtype, seed=3))


def test_attention_of_a_long_chunk():
    attend_and_check(Batch([700, 90], [1500, 1203], 4, 1, 128, 16, BF16, seed=4))


@pytest.mark.parametrize("new,kv", [([1, 1, 2], [40, 9001, 700]), ([300, 9], [555, 1400]), ([2, 0, 1] * 50, [90, 3, 1] * 50)], ids=str)
@pytest.mark.parametrize("dim", [64, 128])
def test_page_tables_of_millions_of_columns(new, kv, dim):
    # whose sizes no longer say that the shares can be counted in 32 bits
    b = Batch(new, kv, 8, 8 if dim == 64 else 2, dim, 512, BF16, seed=21)
    out = []
    k, v, table, q_begin, kv_len = b.cache()
    far = torch.full((len(kv), (1 << 21) // (1 if len(kv) < 4 else 32)), -1, dtype=torch.int32, device=DEV)
    far[:, : table.shape[1]] = table
    for t in (table, far):
        out.append(sz.paged_attention(b.q.to(DEV), k, v, t, q_begin, kv_len, return_lse=True))
        assert not out[-1][2].any()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    want = ref.attention(b.q, b.k, b.v, b.table, b.q_begin, b.kv_len, 1 / math.sqrt(dim))
    check(out[1][0], want[0], want[2])


@pytest.mark.parametrize("dim,page", [(128, 16), (64, 64), (80, 16)])
def test_more_new_tokens_than_cached(dim, page):
    # the first rows stand before the cache's beginning and see nothing
    out, lse = attend_and_check(Batch([9, 150, 4], [4, 20, 0], 4, 2, dim, page, BF16))
    assert not out[:5].any() and bool((lse[:5] == -math.inf).all())


@pytest.mark.parametrize("dim", [64, 128, 72])
def test_extreme_scores(dim):
    # scores of hundreds, equal scores, and the type's lowest value as a key
    b = Batch([3, 130], [200, 131], 4, 2, dim, 16, BF16)
    b.q *= 30
    b.k[int(b.table[0, 1]), 0] = 0.0
    b.k[int(b.table[0, 2]), 1, 3] = 100.0
    attend_and_check(b, scale=0.5)
    # keys hidden from a row may score anything: the last ones are visible to the last rows only
    b = Batch([2], [130], 4, 2, dim, 16, BF16, seed=1)
    b.q = b.q.abs()
    page, at = int(b.table[0, 129 // 16]), 129 % 16
    b.k[page, :, at] = torch.finfo(BF16).min
    b.v[page, :, at] = 1.0
    k, v, table, q_begin, kv_len = b.cache()
    out, lse, status = sz.paged_attention(b.q.to(DEV), k, v, table, q_begin, kv_len, return_lse=True)
    want = ref.attention(b.q, b.k, b.v, b.table, b.q_begin, b.kv_len, 1 / math.sqrt(dim))
    assert bool(torch.isfinite(out).all())
    check(out[:1], want[0][:1], want[2][:1])
    # the last row scores -inf or the lowest number there: weight 0 either way
    hidden = ref.attention(b.q[1:], b.k, b.v, b.table, torch.tensor([0, 1]), torch.tensor([129]), 1 / math.sqrt(dim))
    check(out[1:], hidden[0], hidden[2])


@pytest.mark.parametrize("dim", [64, 128, 72])
@pytest.mark.parametrize("scale,size", [(3e-38, 5e17), (2e-30, 6e13), (-0.1, 1.0), (3e30, 2e-16)])
def test_scales_of_any_size(dim, scale, size):
    # queries and keys whose scores the scale brings back to ordinary numbers
    b = Batch([3, 130], [200, 131], 4, 2, dim, 16, BF16)
    b.q = (b.q.float() * size).to(BF16)
    b.k = (b.k.float() * size).to(BF16)
    attend_and_check(b, scale=scale)


@pytest.mark.parametrize("dim", [128, 72])
def test_infinite_and_nan_scores(dim):
    b = Batch([1, 1, 1, 1], [20, 200, 20, 20], 2, 1, dim, 16, BF16)
    b.q[:] = b.q.abs() + 0.1
    b.k[int(b.table[0, 0]), :, 3] = -math.inf  # one key at -inf: weight 0
    b.k[b.table[1].long()[: 200 // 16 + 1]] = -math.inf  # all at -inf: 0 / 0
    b.k[int(b.table[2, 0]), :, 3] = math.nan
    b.v[int(b.table[3, 1]), :, 2, 1] = math.inf
    k, v, table, q_begin, kv_len = b.cache()
    out, lse, _ = sz.paged_attention(b.q.to(DEV), k, v, table, q_begin, kv_len, return_lse=True)
    out, lse = out.float().cpu(), lse.cpu()
    b.k[int(b.table[0, 0]), :, 3] = 0.0
    keep = [j for j in range(20) if j != 3]
    x = b.q[0].double()
    K, V = ref.gather(b.k, b.table[0], 20)[keep, 0], ref.gather(b.v, b.table[0], 20)[keep, 0]
    want = torch.softmax(x @ K.T / math.sqrt(dim), 1) @ V
    assert float((out[0].double() - want).abs().max()) <= 2.0 ** -6 * float(V.abs().max())  # four half steps of the largest value
    assert bool(out[1:3].isnan().all()) and bool((lse[1] == -math.inf).all()) and bool(lse[2].isnan().all())
    assert bool(torch.isinf(out[3, :, 1]).all()) and bool(torch.isfinite(out[3, :, 2:]).all())


@pytest.mark.parametrize("shape", [([5], [40], 4, 2, 128), ([200], [200], 4, 1, 128), ([150], [290], 2, 2, 64), ([2, 1], [9000, 60], 4, 1, 64),
                                   ([9], [30], 2, 1, 72)], ids=str)
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_values_hidden_from_a_row_do_not_reach_it(shape, value):
    # the last token's value is not finite: the rows before it do not see it;
    # with a window, nor do rows past the first key's
    new, kv, hq, hk, dim = shape
    for window in (0, 33):
        b = Batch(new, kv, hq, hk, dim, 16, BF16)
        k, v, table, q_begin, kv_len = b.cache()
        last, early = kv[0] - 1, max(0, kv[0] - new[0] - 20)
        want = ref.attention(b.q, b.k, b.v, b.table, b.q_begin, b.kv_len, 1 / math.sqrt(dim), True, window)
        v[int(b.table[0, last // 16]), :, last % 16, 3::5] = value
        if window:
            v[int(b.table[0, early // 16]), :, early % 16, 1] = value
        out, lse, status = sz.paged_attention(b.q.to(DEV), k, v, table, q_begin, kv_len, window=window, return_lse=True)
        assert not status.any()
        out = out.cpu()
        # rows of request 0 that see neither key; all of the others
        p = torch.arange(kv[0] - new[0], kv[0])
        clean = p < last
        if window:
            clean &= (p < early) | (p - window >= early)
        clean = torch.cat((clean, torch.ones(b.rows - new[0], dtype=torch.bool)))
        check(out[clean], want[0][clean], want[2][clean])
        check(lse, want[1], want[3])
        assert not torch.isfinite(out[new[0] - 1, :, 3::5].float()).any()
        same = torch.ones(dim, dtype=torch.bool)
        same[3::5] = False
        check(out[new[0] - 1, :, same], want[0][new[0] - 1, :, same], want[2][new[0] - 1, :, same]) if not window else None


def spoil(b, values, hidden=None):
    """Values of request 0, (key, channel, value), put into b.v; what a row
    that sees them comes to: a list of (key, channel, value) for expect()."""
    for key, channel, value in values + ([hidden] if hidden else []):
        b.v[int(b.table[0, key // b.page]), :, key % b.page, channel] = value


def expect(want, tol, p, values, window=0):
    """The definition's result where values (key, channel, value) of request 0
    are not finite: rows at positions p that see them hold +-inf, or NaN where
    both signs or a NaN meet."""
    want, tol = want.clone(), tol.clone()
    for channel in {c for _, c, _ in values}:
        met = torch.zeros(len(p), dtype=torch.float64)
        for key, c, value in values:
            if c == channel:
                met[(p >= key) & ((p - window < key) if window else True)] += value
        rows = met != 0  # inf, -inf or NaN
        want[: len(p), :, channel][rows] = met[rows, None]
        tol[: len(p), :, channel][rows] = 0.0
    return want, tol


def check_with_nan(got, want, tol, what=""):
    got = got.cpu().double()
    assert torch.equal(got.isnan(), want.isnan()), what + ": NaN in other places"
    check(torch.nan_to_num(got, nan=0.0, posinf=math.inf, neginf=-math.inf), torch.nan_to_num(want, nan=0.0, posinf=math.inf, neginf=-math.inf), tol, what)


INF = math.inf
SPOILED = {  # values that rows see, (key, channel, value), and one that the last row alone sees
    "early": ([(5, 3, INF)], None),
    "early_nan": ([(5, 3, math.nan)], None),
    "both_signs": ([(5, 3, INF), (70, 3, -INF), (70, 60, -INF)], None),
    "early_and_last": ([(5, 3, -INF)], (None, 40, INF)),
    "last": ([], (None, 9, math.nan)),
    "a_channel": ([(key, 17, INF) for key in range(2000)], None),
}


@pytest.mark.parametrize("case", SPOILED)
@pytest.mark.parametrize("new,kv,hq,hk,dim,dtype", [([300, 5], [20000, 40], 2, 1, 128, BF16), ([300], [20000], 2, 2, 64, FP16), ([6, 1], [20000, 300], 8, 1, 128, FP16),
                                                    ([7], [9000], 4, 2, 64, BF16)], ids=["chunk128", "chunk64", "few128", "few64"])
def test_values_that_are_not_finite_in_long_caches(case, new, kv, hq, hk, dim, dtype):
    # a row that sees one has it in its result, whatever the weight; a row that
    # does not is computed from what it sees; neither costs the call its status,
    # though computing rows again may take longer than a wait is allowed to
    b = Batch(new, kv, hq, hk, dim, 16, dtype, seed=41)
    values, hidden = SPOILED[case]
    hidden = hidden and (kv[0] - 1, hidden[1], hidden[2])
    want, wl, tol, tl = ref.attention(b.q, b.k, b.v, b.table, b.q_begin, b.kv_len, 1 / math.sqrt(dim))
    spoil(b, values, hidden)
    p = torch.arange(kv[0] - new[0], kv[0])
    want, tol = expect(want, tol, p, values + ([hidden] if hidden else []))
    k, v, table, q_begin, kv_len = b.cache()
    try:
        sz.sz_set_wait_limit_ns(20_000_000)
        out, lse, status = sz.paged_attention(b.q.to(DEV), k, v, table, q_begin, kv_len, return_lse=True)
        torch.cuda.synchronize()
    finally:
        sz.sz_set_wait_limit_ns(1_000_000_000)
    assert not status.any()
    check_with_nan(out, want, tol, "out")
    check(lse, wl, tl, "lse")


@pytest.mark.parametrize("new,kv,dim", [(1, 9000, 128), (3, 9000, 64), (200, 5000, 64), (1, 60, 64), (150, 150, 128), (1, 60, 72), (20, 300, 40)])
@pytest.mark.parametrize("first", [0, 2])
def test_values_of_keys_that_score_minus_infinity(new, kv, dim, first):
    # weight 0 exactly: 0 times a value that is not finite is NaN, wherever the
    # key lies among those that are summed together, and where whole tiles score
    # -inf; other channels are those of the other keys.  Rows that do not see it
    # are clean (below, behind the window).
    b = Batch([new], [kv], 2, 1, dim, 16, BF16, seed=43)
    b.q = b.q.abs() + 0.1
    bad = [first, first + 1, *range(kv // 2, kv // 2 + (300 if kv > 4000 else 1))]
    for j in bad:
        b.k[int(b.table[0, j // 16]), :, j % 16] = -math.inf
    b.v[int(b.table[0, 0]), :, first + 1, 5] = math.inf
    b.v[int(b.table[0, (kv // 2) // 16]), :, (kv // 2) % 16, 7] = math.nan
    k, v, table, q_begin, kv_len = b.cache()
    x = b.q.double().transpose(0, 1)
    K, V = (ref.gather(t, b.table[0], kv)[:, 0].double() for t in (b.k, b.v))
    K[bad], V[bad] = 0.0, 0.0
    p, j = torch.arange(kv - new, kv)[:, None], torch.arange(kv)[None]
    for window in (0, kv // 2 - 20):
        out, lse, status = sz.paged_attention(b.q.to(DEV), k, v, table, q_begin, kv_len, window=window, return_lse=True)
        assert not status.any()
        out = out.double().cpu().transpose(0, 1)
        inside = (j <= p) & ((j > p - window) if window else True)
        seen = inside.clone()
        seen[:, bad] = False
        some = seen.any(1)
        s = (x @ K.T / math.sqrt(dim)).masked_fill(~seen, -math.inf)
        want = torch.softmax(s, -1) @ V
        for channel, key in ((5, first + 1), (7, kv // 2)):
            assert torch.equal(out[:, some, channel].isnan(), inside[some, key][None].expand(2, -1))
            want[:, inside[:, key], channel] = out[:, inside[:, key], channel] = 0.0
        assert float((out - want)[:, some].abs().max()) <= 2.0 ** -6 * float(V.abs().max())  # four half steps of the largest value
        assert bool(out[:, ~some & inside.any(1)].isnan().any(-1).all())


@pytest.mark.parametrize("new,hq", [(200, 1), (3, 4)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("over", [False, True])
def test_infinities_of_small_weights(new, hq, dtype, over):
    # keys whose weights are far below what 16 bits hold: an infinite value of
    # theirs is in the result all the same, and NaN where the score is -inf
    dim, kv = 128, 260
    b = Batch([new], [kv], hq, 1, dim, 16, dtype, seed=42)
    b.q = b.q.abs() + 0.5
    for key in (2, 7):  # scores about 10 below the others': exp(-30) or so
        b.k[int(b.table[0, 0]), 0, key] = -4.0
    want, _, tol, _ = ref.attention(b.q, b.k, b.v, b.table, b.q_begin, b.kv_len, 1 / math.sqrt(dim))
    spoil(b, [(2, 3, INF), (7, 50, -INF), (7, 3, INF)])
    want, tol = expect(want, tol, torch.arange(kv - new, kv), [(2, 3, INF), (7, 50, -INF)])
    k, v, table, q_begin, kv_len = b.cache()
    q = b.q.to(DEV)
    out, _, status = sz.paged_attention(q, k, v, table, q_begin, kv_len, out=q if over else None)
    assert not status.any()
    check_with_nan(out, want, tol)
    k[int(b.table[0, 0]), 0, 7] = -math.inf  # weight 0 exactly
    out, _, status = sz.paged_attention(b.q.to(DEV), k, v, table, q_begin, kv_len)
    assert not status.any() and bool(out[:, :, 50].isnan().all()) and bool(out[:, :, 3].isnan().all())


@pytest.mark.parametrize("dim,hidden", [(128, None), (128, math.inf), (64, None), (64, math.nan)], ids=str)
def test_short_blocks_behind_long_ones(dim, hidden):
    # a CTA's blocks of 64 and of 8 rows in turn: a warp that holds rows of the
    # first alone must not let the next block's products begin while the other
    # warp of its rows still reads.  A value that is not finite, in the upper
    # channels of a key that the rows before do not see, keeps that one longest.
    b = Batch([8, 1] * 20, [1500, 1400] * 20, 64, 8, dim, 16, BF16, seed=31)
    want = ref.attention(b.q, b.k, b.v, b.table, b.q_begin, b.kv_len, 1 / math.sqrt(dim))
    clean = torch.ones(b.rows, dtype=torch.bool)
    k, v, table, q_begin, kv_len = b.cache()
    if hidden is not None:
        for r in range(0, len(b.kv), 2):
            last = b.kv[r] - 1
            v[int(b.table[r, last // 16]), :, last % 16, dim // 2 + 5] = hidden
            clean[int(b.q_begin[r + 1]) - 1] = False  # the row that sees it
    for _ in range(5):
        out, lse, status = sz.paged_attention(b.q.to(DEV), k, v, table, q_begin, kv_len, return_lse=True)
        assert not status.any()
        out = out.cpu()
        check(out[clean], want[0][clean], want[2][clean])
        check(lse, want[1], want[3])
        seen = torch.arange(dim) != dim // 2 + 5
        check(out[~clean][..., seen], want[0][~clean][..., seen], want[2][~clean][..., seen])
        assert not torch.isfinite(out[~clean][..., dim // 2 + 5].float()).any()


def test_waits_that_run_out_are_reported():
    # the copy warps issue nothing, so every wait ends by its limit
    few, many = Batch([1, 2], [3000, 70], 8, 2, 128, 16, BF16), Batch([300], [900], 8, 2, 64, 16, FP16)
    ws = torch.empty(sz.sz_plan_attention(128), dtype=torch.uint8, device=DEV)
    for b in (few, many):
        args = [b.q.to(DEV)] + b.cache()
        good = sz.paged_attention(*args, workspace=ws)[0].clone()
        try:
            sz.sz_debug_set_flags(1)
            sz.sz_set_wait_limit_ns(2_000_000)
            _, _, status = sz.paged_attention(*args, workspace=ws)
            torch.cuda.synchronize()
        finally:
            sz.sz_debug_set_flags(0)
            sz.sz_set_wait_limit_ns(1_000_000_000)
        assert status.cpu().tolist() == [sz.SZ_ERR_DEVICE_TIMEOUT] * len(b.kv)
        again, _, status = sz.paged_attention(*args, workspace=ws)
        assert not status.any() and torch.equal(again, good)


@pytest.mark.parametrize("new,kv,dim", [([1, 2] * 30, [3000, 70] * 30, 128), ([5] * 12, [900] * 12, 64), ([300, 200], [900, 2000], 64),
                                        ([700, 90], [1500, 1203], 128)], ids=["few128", "few64", "many64", "many128"])
@pytest.mark.parametrize("limit", [0, 1, 1000, 5000])
def test_waits_that_run_out_with_copies_under_way(new, kv, dim, limit):
    # limits shorter than a copy takes (a wait that the hardware ends before it
    # looks at the clock is none that ran out): the call ends with one status for
    # all, after everything that it set going, and the next one is as good as ever
    b = Batch(new, kv, 8, 2, dim, 16, BF16)
    args = [b.q.to(DEV)] + b.cache()
    ws = torch.empty(sz.sz_plan_attention(dim), dtype=torch.uint8, device=DEV)
    good = sz.paged_attention(*args, workspace=ws)[0].clone()
    for _ in range(4):
        try:
            sz.sz_set_wait_limit_ns(limit)
            out, _, status = sz.paged_attention(*args, workspace=ws)
            torch.cuda.synchronize()
        finally:
            sz.sz_set_wait_limit_ns(1_000_000_000)
        got = set(status.cpu().tolist())
        assert got in ({0}, {sz.SZ_ERR_DEVICE_TIMEOUT})
        assert got != {0} or torch.equal(out, good)
        again, _, status = sz.paged_attention(*args, workspace=ws)
        assert not status.any() and torch.equal(again, good)


@pytest.mark.parametrize("new,kv,dim", [([5] * 12, [40] * 12, 128), ([7], [200], 64), ([200], [200], 128), ([4, 3], [5000, 70], 128)], ids=str)
def test_hidden_values_with_the_output_over_the_queries(new, kv, dim):
    # such rows are computed from their queries once more, which stay until
    # every warp that needs them has read them
    b = Batch(new, kv, 8, 2, dim, 16, BF16)
    k, v, table, q_begin, kv_len = b.cache()
    for r, n in enumerate(kv):
        v[int(b.table[r, (n - 1) // 16]), :, (n - 1) % 16] = math.inf
    q = b.q.to(DEV)
    apart, _, _ = sz.paged_attention(q, k, v, table, q_begin, kv_len)
    assert int(torch.isfinite(apart).all(-1).all(-1).sum()) == b.rows - len(kv)
    for _ in range(20):
        over = q.clone()
        sz.paged_attention(over, k, v, table, q_begin, kv_len, out=over)
        assert torch.equal(over.view(torch.int16), apart.view(torch.int16))


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("reqs,new", [(1, 4864), (40, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_small_weights_behind_one_large(dtype, reqs, new, dim):
    # one key with value 0, 131,071 with value 1 whose weights are 2^-25.5 of its:
    # together 2^-8.5.  A weight is off by half a step of 16 bits, or half of FP16's
    # smallest step, 2^-25 against a sum of at least 2^7: n 2^-32 in all.  The sums
    # of weights take 32 steps in a tile and n / 128 tiles, each off by 2^-24: 2^-13.9
    # together; those of weights times values n / 16 steps, cut off at 2^-23: 2^-10.
    # The exponential's argument of 25.5 adds 2^-18, and the result is rounded once.
    n, heads, page = 131072, 8, 1024
    k = torch.zeros((n // page, heads, page, dim), dtype=dtype, device=DEV)
    v = torch.ones_like(k)
    k[0, :, 0], v[0, :, 0] = 1.0, 0.0
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).repeat(reqs, 1)
    q_begin = torch.arange(reqs + 1, dtype=torch.int32, device=DEV) * new
    kv_len = torch.full((reqs,), n, dtype=torch.int32, device=DEV)
    q = torch.ones((reqs * new, heads, dim), dtype=dtype, device=DEV)
    out, lse, status = sz.paged_attention(q, k, v, table, q_begin, kv_len, scale=25.5 / dim * math.log(2), causal=False, return_lse=True)
    assert not status.any()
    mass = (n - 1) * 2.0 ** -25.5
    want = mass / (1 + mass)
    h = ref.HALF_STEP[dtype]
    sums = (32 + n / 128) * 2.0 ** -24
    tol = want * (2 * h + 2.0 ** -10 + sums + 2.0 ** -18) + (n * 2.0 ** -32 if dtype == FP16 else 0.0)
    assert float((out.double() - want).abs().max()) <= tol
    full = 25.5 * math.log(2) + math.log1p(mass)
    assert float((lse.double() - full).abs().max()) <= sums + 2.0 ** -18 * full


@pytest.mark.parametrize("layout", ["token_major", "one_pool", "rows_of_a_projection", "in_place"])
@pytest.mark.parametrize("dim", [128, 40])
def test_attention_layouts(layout, dim):
    b = Batch([5, 130, 1], [50, 131, 90], 8, 2, dim, 16, BF16, extra_rows=3)
    k, v, table, q_begin, kv_len = b.cache()
    q, out = b.q.to(DEV), None
    if layout == "token_major":
        k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    elif layout == "one_pool":
        pool = torch.stack((k, v), 1)
        k, v = pool[:, 0], pool[:, 1]
        table = torch.cat((table, table), 1)[:, : table.shape[1]]
    elif layout == "rows_of_a_projection":
        row = torch.cat((q, torch.full((q.shape[0], 4, dim), math.nan, dtype=BF16, device=DEV)), 1)
        q = row[:, :8]
        out = torch.full((8, b.rows, dim), 7.0, dtype=BF16, device=DEV).transpose(0, 1)
    else:
        out = q
    got, _, status = sz.paged_attention(q, k, v, table, q_begin, kv_len, out=out)
    assert status.cpu().tolist() == [0, 0, 0]
    want = ref.attention(b.q, b.k, b.v, b.table, b.q_begin, b.kv_len, 1 / math.sqrt(dim))
    check(got[: b.rows - 3], want[0][: b.rows - 3], want[2][: b.rows - 3])
    if layout == "rows_of_a_projection":
        assert bool((got[b.rows - 3:] == 7.0).all())  # rows of no request
    if layout == "in_place":
        assert torch.equal(got[b.rows - 3:].cpu(), b.q[b.rows - 3:])


@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("repeat", ["heads", "tokens", "both", "overlap"])
def test_rows_that_repeat(dim, repeat):
    # queries, keys and values that are views with a stride of 0, or of less than a row
    b = Batch([5, 60], [50, 131], 4, 2, dim, 16, BF16)
    k, v, table, q_begin, kv_len = b.cache()
    n = b.rows
    base = torch.randn(n * dim + 4096, generator=b.g).to(BF16).to(DEV)

    def rows(heads):
        strides = {"heads": (dim, 0, 1), "tokens": (0, dim, 1), "both": (0, 0, 1), "overlap": (8, 16, 1)}[repeat]
        return base.as_strided((n, heads, dim), strides)

    q = rows(4)
    out, _, status = sz.paged_attention(q, k, v, table, q_begin, kv_len)
    assert not status.any()
    want = ref.attention(q.cpu(), b.k, b.v, b.table, b.q_begin, b.kv_len, 1 / math.sqrt(dim))
    check(out, want[0], want[2])
    got = []
    for new, q1 in ((rows(2), q), (rows(2).contiguous(), q.contiguous())):
        k1, v1 = k.clone(), v.clone()
        q_out, status = sz.append_kv(new, new, k1, v1, table, q_begin, kv_len, q=q1, rope_freqs=sz.rope_frequencies(dim // 16 * 16, device=DEV))
        assert not status.any()
        got.append([t.view(torch.int16) for t in (k1, v1, q_out)])
    assert all(torch.equal(x, y) for x, y in zip(*got))
    with pytest.raises(sz.SzError):  # written rows must lie apart
        sz.paged_attention(q, k, v, table, q_begin, kv_len, out=rows(4))


@pytest.mark.parametrize("dim", [128, 24])
def test_pages_behind_the_window_may_be_gone(dim):
    b = Batch([1, 20], [300, 200], 4, 2, dim, 16, BF16)
    b.table[0, : (300 - 64) // 16] = -1
    b.table[1, : (200 - 20 + 1 - 64) // 16] = 1 << 20
    attend_and_check(b, window=64)


@pytest.mark.parametrize("dim", [128, 24])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1])
def test_windows_wider_than_any_cache(dim, window):
    # more new tokens than cached: the window begins before the cache, by more
    # than 31 bits hold, and a bad page in it is found
    b = Batch([9, 6], [4, 2], 4, 2, dim, 16, BF16)
    attend_and_check(b, window=window)
    b.table[1, 0] = 1 << 20
    _, _, status = sz.paged_attention(b.q.to(DEV), *b.cache(), window=window)
    assert status.tolist() == [0, sz.SZ_ERR_INVALID]


@pytest.mark.parametrize("dim", [128, 24])
def test_refused_requests(dim):
    b = Batch([2, 1, 1, 1, 1], [40, 40, 20, 33, 9], 4, 2, dim, 16, BF16)
    b.table[1, 1] = 1 << 30  # outside the pool
    b.table[2, 0] = -5
    b.kv_len[3] = 49  # the table holds 48
    k, v, table, q_begin, kv_len = b.cache()
    out, _, status = sz.paged_attention(b.q.to(DEV), k, v, table, q_begin, kv_len)
    assert status.cpu().tolist() == [0, sz.SZ_ERR_INVALID, sz.SZ_ERR_INVALID, sz.SZ_ERR_CAPACITY, 0]
    want = ref.attention(b.q[:2], b.k, b.v, b.table, torch.tensor([0, 2]), torch.tensor([40]), 1 / math.sqrt(dim))
    check(out[:2], want[0], want[2])
    new = torch.randn(6, 2, dim, dtype=torch.float32).to(BF16).to(DEV)
    before = k.clone()
    _, status = sz.append_kv(new, new, k, v, table, q_begin, torch.tensor([40, 17, 1, 49, 0], dtype=torch.int32, device=DEV))
    # request 1's token would go to its bad page, request 4 has more tokens than its length
    assert status.cpu().tolist() == [0, sz.SZ_ERR_INVALID, sz.SZ_ERR_INVALID, sz.SZ_ERR_CAPACITY, sz.SZ_ERR_INVALID]
    changed = (k.view(torch.int16) != before.view(torch.int16)).any(-1).any(1).nonzero().cpu().tolist()
    page = int(b.table[0, 2])
    assert changed == [[page, 6], [page, 7]]
    # rows out of order, or more than there are
    bad = torch.tensor([0, 2, 1, 3, 9, 9], dtype=torch.int32, device=DEV)
    table[:] = torch.arange(5, dtype=torch.int32, device=DEV)[:, None]
    for call in (lambda: sz.paged_attention(b.q.to(DEV), k, v, table, bad, kv_len.clamp(max=16))[2],
                 lambda: sz.append_kv(new, new, k, v, table, bad, kv_len.clamp(max=16))[1]):
        assert call().cpu().tolist() == [0, sz.SZ_ERR_INVALID, 0, sz.SZ_ERR_INVALID, sz.SZ_ERR_INVALID]


@pytest.mark.parametrize("reqs,rows,heads,kv_heads", [(32, 65536, 32, 8), (512, 4096, 32, 8), (512, 32768, 8, 8)])
def test_requests_that_overlap_are_not_computed(reqs, rows, heads, kv_heads):
    # q_begin goes back and forth, so that every second request claims all rows:
    # far more work than n_tokens rows are, and more than 32-bit shares count
    dim, page, kv = 64, 128, 32768
    k = torch.zeros((4, kv_heads, page, dim), dtype=BF16, device=DEV)
    table = torch.zeros((reqs, kv // page), dtype=torch.int32, device=DEV)
    q = torch.zeros((rows, heads, dim), dtype=BF16, device=DEV)
    out = torch.full_like(q, 7.0)
    back = torch.tensor([0, rows] * (reqs // 2) + [0], dtype=torch.int32, device=DEV)
    kv_len = torch.full((reqs,), kv, dtype=torch.int32, device=DEV)
    need = sz.sz_plan_attention(dim)
    buffer = torch.full((need + (1 << 20),), 77, dtype=torch.uint8, device=DEV)
    _, _, status = sz.paged_attention(q, k, k, table, back, kv_len, out=out, workspace=buffer[:need])
    torch.cuda.synchronize()
    assert status.cpu().tolist() == [0, sz.SZ_ERR_INVALID] * (reqs // 2)
    assert bool((out == 7.0).all()) and bool((buffer[need:] == 77).all())


def test_attention_repeats_bit_for_bit_and_on_two_streams():
    b = Batch([1, 3, 200], [5000, 700, 900], 8, 2, 128, 16, BF16)
    args = [b.q.to(DEV)] + b.cache()
    first, _, _ = sz.paged_attention(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [sz.paged_attention(*args, stream=streams[i % 2])[0] for i in range(8)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)


def test_two_host_threads_call_at_once():
    from concurrent.futures import ThreadPoolExecutor
    batches = [Batch([3, 40], [300, 700], 8, 2, 128, 16, BF16, seed=11), Batch([1, 1, 1], [2000, 5, 90], 16, 4, 64, 32, FP16, seed=12)]
    given = [(b.q.to(DEV), *b.cache()) for b in batches]
    alone = [sz.paged_attention(*x)[0].clone() for x in given]
    torch.cuda.synchronize()

    def work(x, want):
        s = torch.cuda.Stream()
        for _ in range(50):
            out, _, status = sz.paged_attention(*x, stream=s)
            rows = x[0][:, : x[1].shape[1]].contiguous()
            pages = [t.clone() for t in x[1:3]]
            s.wait_stream(torch.cuda.current_stream())
            _, put = sz.append_kv(rows, rows, *pages, *x[3:], stream=s)
            s.synchronize()
            assert torch.equal(out, want) and not status.any() and not put.any()

    with ThreadPoolExecutor(2) as pool:
        for f in [pool.submit(work, x, want) for x, want in zip(given, alone)]:
            f.result()


def test_captured_calls_follow_their_lengths():
    b = Batch([1, 1, 2], [600, 40, 90], 8, 2, 128, 16, FP16, width=64)
    k, v, table, q_begin, kv_len = b.cache()
    q, out = b.q.to(DEV), torch.zeros_like(b.q, device=DEV)
    new = torch.randn(4, 2, 128).to(FP16).to(DEV)
    freqs = sz.rope_frequencies(128, device=DEV)
    ws = torch.empty(sz.sz_plan_attention(128), dtype=torch.uint8, device=DEV)
    q_rot = torch.empty_like(q)

    def step():
        sz.append_kv(new, new, k, v, table, q_begin, kv_len, q=q, q_out=q_rot, rope_freqs=freqs)
        return sz.paged_attention(q_rot, k, v, table, q_begin, kv_len, out=out, workspace=ws)[2]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        status = step()
    for kv in ([600, 40, 90], [3, 40, 2], [601, 33, 64]):
        kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert status.cpu().tolist() == [0, 0, 0]
        replayed = out.clone()
        out.zero_()
        step()
        assert torch.equal(replayed, out)
        want = ref.attention(q_rot.cpu(), k.cpu(), v.cpu(), b.table, b.q_begin, kv_len.cpu(), 1 / math.sqrt(128))
        check(replayed, want[0], want[2])


def test_the_output_is_encoded_behind_the_call():
    # the one-pass encode reads its input before the kernel ahead of it has
    # ended, unless that kernel holds it back
    b = Batch([1] * 20, [300] * 20, 32, 8, 128, 16, BF16, seed=9)
    k, v, table, q_begin, kv_len = b.cache()
    q = b.q.to(DEV)
    out = torch.zeros_like(q)
    book = torch.arange(112, 128, dtype=torch.uint8, device=DEV)
    want, _, _ = sz.paged_attention(q, k, v, table, q_begin, kv_len)
    for _ in range(20):
        out.zero_()
        sz.paged_attention(q, k, v, table, q_begin, kv_len, out=out)
        blob, _, status = sz.encode_one_pass(out, book)
        back, st = sz.decode(blob, out.numel())
        assert int(status) == 0 and int(st) == 0
        assert torch.equal(back.view(-1), want.view(torch.int16).view(-1))


@pytest.mark.parametrize("new,kv,split", [([1, 2], [300, 70], False), ([1, 2], [3000, 70], True)])
def test_a_timeout_does_not_stick_to_a_captured_call(new, kv, split):
    # A call that ran into its limit leaves its tag and the time in the workspace
    # (the only words of it that a call without split rows writes); the tag counts
    # calls.  Given a captured call's tag there, its next replay reports it, and
    # after the join, or if it is long ago, no later one does.
    b = Batch(new, kv, 8, 2, 128, 16, BF16)
    args = [b.q.to(DEV)] + b.cache()
    ws = torch.zeros(sz.sz_plan_attention(128) // 8, dtype=torch.int64, device=DEV)
    short = Batch([1], [20], 8, 2, 128, 16, BF16)
    try:
        sz.sz_debug_set_flags(1)
        sz.sz_set_wait_limit_ns(2_000_000)
        _, _, status = sz.paged_attention(short.q.to(DEV), *short.cache(), workspace=ws)
        torch.cuda.synchronize()
    finally:
        sz.sz_debug_set_flags(0)
        sz.sz_set_wait_limit_ns(1_000_000_000)
    assert status.tolist() == [sz.SZ_ERR_DEVICE_TIMEOUT]
    at = ws.nonzero().flatten().tolist()
    assert len(at) == 2 and at[1] == at[0] + 1
    mark = ws[at[0]:at[1] + 1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, status = sz.paged_attention(*args, workspace=ws)

    def replay(mark):
        ws[at[0]:at[1] + 1] = mark
        got = []
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            got.append(set(status.tolist()))
        return got

    now, ago = mark + torch.tensor([1, 0], device=DEV), mark + torch.tensor([1, -12_000_000_000], device=DEV)
    late = {sz.SZ_ERR_DEVICE_TIMEOUT}
    assert replay(mark) == [{0}, {0}]  # another call's
    assert replay(now) == [late, {0} if split else late]
    assert replay(ago) == [{0}, {0}]
    assert torch.equal(out, sz.paged_attention(*args)[0])


def test_two_captured_calls_share_a_workspace():
    b = Batch([1, 2], [3000, 700], 8, 2, 128, 16, BF16)
    c = Batch([200], [900], 8, 2, 128, 16, BF16, seed=9)
    ws = torch.empty(sz.sz_plan_attention(128), dtype=torch.uint8, device=DEV)
    calls, graphs = [], []
    for x in (b, c):
        args = [x.q.to(DEV)] + x.cache()
        eager = sz.paged_attention(*args)[0].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = sz.paged_attention(*args, workspace=ws)[0]
        calls.append((out, eager, args))
        graphs.append(g)
    for _ in range(3):
        for g, (out, eager, _) in zip(graphs, calls):
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for out, eager, _ in calls:
            assert torch.equal(out, eager)


def test_cache_beyond_32_bits():
    # pools of more than 2^32 values; the request's pages lie at the end
    P, H, D = 16, 8, 128
    pages = (1 << 32) // (P * H * D) + 300
    k = torch.empty((pages, H, P, D), dtype=BF16, device=DEV)
    v = torch.empty_like(k)
    b = Batch([3, 1], [40, 200], 16, 8, D, P, BF16)
    k[-b.k.shape[0]:], v[-b.k.shape[0]:] = b.k.to(DEV), b.v.to(DEV)
    _, _, table, q_begin, kv_len = b.cache()
    far = torch.where(table >= 0, table + (pages - b.k.shape[0]), table).int()
    out, _, status = sz.paged_attention(b.q.to(DEV), k, v, far, q_begin, kv_len)
    assert status.cpu().tolist() == [0, 0]
    want = ref.attention(b.q, b.k, b.v, b.table, b.q_begin, b.kv_len, 1 / math.sqrt(D))
    check(out, want[0], want[2])
    new = torch.randn(4, H, D).to(BF16).to(DEV)
    _, status = sz.append_kv(new, new, k, v, far, q_begin, kv_len)
    assert status.cpu().tolist() == [0, 0]
    for t, (r, at) in enumerate([(0, 37), (0, 38), (0, 39), (1, 199)]):
        assert torch.equal(k[int(far[r, at // P]), :, at % P], new[t])
        assert torch.equal(v[int(far[r, at // P]), :, at % P], new[t])


# ------------------------------------------------------------------ append
def append_and_check(b, rot=0, interleaved=False, norm=False, with_q=True, positions=None, scale=1.0, rows=None):
    hk, dim = b.k.shape[1], b.k.shape[3]
    tokens = b.rows
    new_k, new_v = torch.randn((tokens, hk, dim), generator=b.g).to(b.dtype), torch.randn((tokens, hk, dim), generator=b.g).to(b.dtype)
    freqs = sz.rope_frequencies(rot, 1e6) if rot else None
    qw = (1 + 0.3 * torch.randn(dim, generator=b.g)).to(b.dtype) if norm and with_q else None
    kw = (1 + 0.3 * torch.randn(dim, generator=b.g)).to(b.dtype) if norm else None
    k, v, table, q_begin, kv_len = b.cache()
    n = len(b.kv)
    hists = torch.full((3 * n, 256), 5, dtype=torch.int32, device=DEV)

    def dev(t):
        return None if t is None else t.to(DEV)

    q_out, status = sz.append_kv(new_k.to(DEV), new_v.to(DEV), k, v, table, q_begin, kv_len, q=b.q.to(DEV) if with_q else None,
                                 rope_freqs=dev(freqs), rope_interleaved=interleaved, rope_scale=scale, positions=dev(positions),
                                 q_norm=dev(qw), k_norm=dev(kw), eps=1e-5, hists=hists, hist_rows=dev(rows))
    torch.cuda.synchronize()
    assert status.cpu().tolist() == [0] * n
    place = torch.zeros(tokens, dtype=torch.int64)
    owner = [-1] * tokens
    for r in range(n):
        for i in range(b.new[r]):
            t = int(b.q_begin[r]) + i
            place[t], owner[t] = b.kv[r] - b.new[r] + i, r
    pos = positions if positions is not None else place
    want_k, tol_k = ref.turned(new_k, kw, 1e-5, freqs, pos, interleaved, scale)
    got_k, got_v = k.cpu(), v.cpu()
    counts = torch.full((3 * n, 256), 5, dtype=torch.int64)
    at = rows.tolist() if rows is not None else list(range(2 * n))
    touched = torch.zeros(b.k.shape[:3], dtype=torch.bool)
    for t in range(tokens):
        r = owner[t]
        if r < 0:
            continue
        p, s = int(b.table[r, int(place[t]) // b.page]), int(place[t]) % b.page
        touched[p, :, s] = True
        check(got_k[p, :, s], want_k[t], tol_k[t], "k")
        assert torch.equal(got_v[p, :, s], new_v[t])
        for row, x in ((at[r], got_k[p, :, s]), (at[n + r], new_v[t])):
            e = (x.contiguous().view(torch.int16).long() >> 7) & 255
            counts[row] += torch.bincount(e.reshape(-1), minlength=256)
    for got, was in ((got_k, b.k), (got_v, b.v)):  # nothing else changed, NaN patterns included
        assert torch.equal(got.view(torch.int16)[~touched], was.view(torch.int16)[~touched])
    assert torch.equal(hists.cpu().long(), counts)
    if with_q:
        want_q, tol_q = ref.turned(b.q, qw, 1e-5, freqs, pos, interleaved, scale)
        mine = torch.tensor([o >= 0 for o in owner])
        check(q_out.cpu()[mine], want_q[mine], tol_q[mine], "q")


APPENDS = [  # new, cached, query heads, KV heads, dim, page, type
    ([1], [1], 32, 8, 128, 16, BF16),
    ([1, 1, 0, 1], [16, 17, 5, 300], 8, 2, 64, 16, FP16),
    ([40, 3, 17], [40, 500, 33], 6, 3, 128, 32, BF16),
    ([5, 64], [5, 80], 4, 1, 256, 8, FP16),
    ([9], [20], 3, 1, 80, 5, BF16),
    ([3], [3], 1, 1, 16, 1, BF16),
    ([200], [1000], 28, 4, 128, 16, BF16),
]


@pytest.mark.parametrize("shape", APPENDS, ids=lambda s: "-".join(map(str, s[:6])).replace(" ", ""))
@pytest.mark.parametrize("mode", ["plain", "half", "adjacent", "norm", "norm_half_part", "norm_adjacent_part", "no_q"])
def test_append(shape, mode):
    new, kv, hq, hk, dim, page, dtype = shape
    b = Batch(new, kv, hq, hk, dim, page, dtype, extra_rows=2)
    part = max(16, dim // 32 * 16)
    append_and_check(b, rot={"plain": 0, "norm": 0, "norm_half_part": part, "norm_adjacent_part": part}.get(mode, dim), norm="norm" in mode,
                     interleaved="adjacent" in mode, with_q=mode != "no_q", scale=1.25 if "part" in mode else 1.0)


def test_append_at_far_positions():
    b = Batch([30, 2], [40, 5], 4, 2, 128, 16, BF16)
    far = torch.tensor([(1 << 20) * (i + 1) + i for i in range(30)] + [-7, 0], dtype=torch.int64)
    append_and_check(b, rot=128, positions=far)


def test_append_into_chosen_histogram_rows():
    b = Batch([30, 2, 5], [40, 5, 5], 4, 2, 128, 16, BF16)
    append_and_check(b, rot=64, rows=torch.tensor([4, 4, 0, 8, 7, 4], dtype=torch.int32))  # several requests in one row
    k, v, table, q_begin, kv_len = b.cache()
    new = torch.zeros((b.rows, 2, 128), dtype=BF16, device=DEV)
    hists = torch.zeros((4, 256), dtype=torch.int32, device=DEV)
    rows = torch.tensor([0, 1, 4, 0, -1, 3], dtype=torch.int32, device=DEV)
    _, status = sz.append_kv(new, new, k, v, table, q_begin, kv_len, hists=hists, hist_rows=rows)
    assert status.cpu().tolist() == [0, sz.SZ_ERR_INVALID, sz.SZ_ERR_INVALID]
    assert int(hists.sum()) == 2 * 30 * 2 * 128 and int(hists[0].sum()) == int(hists.sum())


@pytest.mark.parametrize("shape", APPENDS, ids=lambda s: "-".join(map(str, s[:6])).replace(" ", ""))
@pytest.mark.parametrize("interleaved", [False, True])
def test_counting_changes_nothing_else(shape, interleaved):
    new, kv, hq, hk, dim, page, dtype = shape
    b = Batch(new, kv, hq, hk, dim, page, dtype, extra_rows=2)
    rows = [torch.randn((b.rows, h, dim), generator=b.g).to(dtype).to(DEV) for h in (hq, hk, hk)]
    w = (1 + 0.3 * torch.randn(dim, generator=b.g)).to(dtype).to(DEV)
    freqs = sz.rope_frequencies(dim // 16 * 16, device=DEV)
    got = []
    for counted in (False, True):
        k, v, table, q_begin, kv_len = b.cache()
        hists = torch.zeros((2 * len(kv), 256), dtype=torch.int32, device=DEV) if counted else None
        q_out = torch.full_like(rows[0], 3.0)
        _, status = sz.append_kv(rows[1], rows[2], k, v, table, q_begin, kv_len, q=rows[0], q_out=q_out, rope_freqs=freqs,
                                 rope_interleaved=interleaved, q_norm=w, k_norm=w, hists=hists)
        assert not status.any()
        got.append([x.view(torch.int16) for x in (k, v, q_out)])
    for a, c in zip(*got):
        assert torch.equal(a, c)


@pytest.mark.parametrize("counted", [False, True])
@pytest.mark.parametrize("ahead", [3, 400])
def test_rows_that_no_request_has(counted, ahead):
    # rows before the first request, and padding rows as requests that nothing
    # is cached for: neither is written, and every other row is
    n, dim = [5, 6, 40, 2], 64
    k = torch.zeros((30, 2, 16, dim), dtype=BF16, device=DEV)
    v = torch.zeros_like(k)
    table = torch.randperm(30)[:20].view(4, 5).to(torch.int32).to(DEV)
    q_begin = torch.tensor([ahead] + [ahead + sum(n[: i + 1]) for i in range(4)], dtype=torch.int32, device=DEV)
    kv_len = torch.tensor([20, 0, 40, 9], dtype=torch.int32, device=DEV)
    tokens = ahead + sum(n) + 7
    new = torch.randn((tokens, 2, dim), device=DEV).to(BF16)
    hists = torch.zeros((8, 256), dtype=torch.int32, device=DEV) if counted else None
    q_out = torch.full((tokens, 4, dim), 3.0, dtype=BF16, device=DEV)
    q = torch.randn((tokens, 4, dim), device=DEV).to(BF16)
    _, status = sz.append_kv(new, new, k, v, table, q_begin, kv_len, q=q, q_out=q_out, hists=hists)
    assert status.cpu().tolist() == [0, sz.SZ_ERR_INVALID, 0, 0]
    mine = torch.zeros(tokens, dtype=torch.bool, device=DEV)
    for r in (0, 2, 3):
        for i in range(n[r]):
            t, at = int(q_begin[r]) + i, int(kv_len[r]) - n[r] + i
            mine[t] = True
            assert torch.equal(k[int(table[r, at // 16]), :, at % 16], new[t]) and torch.equal(v[int(table[r, at // 16]), :, at % 16], new[t])
    assert torch.equal(q_out[mine], q[mine]) and bool((q_out[~mine] == 3.0).all())
    assert int((k != 0).any(-1).any(1).sum()) == int(mine.sum())
    if counted:
        assert hists.sum(1).cpu().tolist() == [2 * dim * m for m in (5, 0, 40, 2)] * 2
    out = torch.full_like(q, 3.0)
    _, _, status = sz.paged_attention(q, k, v, table, q_begin, kv_len, out=out)
    assert status.cpu().tolist() == [0, 0, 0, 0]
    pad = torch.arange(int(q_begin[1]), int(q_begin[2]))
    assert not out[pad].any() and bool((out[:ahead] == 3.0).all()) and bool((out[int(q_begin[4]):] == 3.0).all())
    lone, _, _ = sz.paged_attention(q[int(q_begin[2]): int(q_begin[3])], k, v, table[2:3], torch.tensor([0, 40], dtype=torch.int32, device=DEV),
                                    kv_len[2:3])
    got = out[int(q_begin[2]): int(q_begin[3])]
    assert float((got.double() - lone.double()).abs().max()) <= 2.0 ** -6 * float(v.abs().max())  # each within 2^-7 of the largest value


@pytest.mark.parametrize("layout", ["token_major", "rows_of_a_projection"])
def test_append_layouts_and_in_place(layout):
    b = Batch([5, 20], [50, 31], 4, 2, 128, 16, BF16)
    k, v, table, q_begin, kv_len = b.cache()
    row = torch.randn(25, 8, 128).to(BF16).to(DEV)
    freqs = sz.rope_frequencies(128, device=DEV)
    plain = [row[:, :4].clone(), row[:, 4:6].clone(), row[:, 6:].clone()]
    q0, _ = sz.append_kv(plain[1], plain[2], k, v, table, q_begin, kv_len, q=plain[0], rope_freqs=freqs)
    k2, v2 = (t.to(DEV) for t in (b.k, b.v))
    if layout == "token_major":
        k2, v2 = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k2, v2))
    q = row[:, :4]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sz.append_kv(row[:, 4:6], row[:, 6:], k2, v2, table, q_begin, kv_len, q=q, q_out=q, rope_freqs=freqs, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(q, q0)
    assert torch.equal(k2.contiguous().view(torch.int16), k.view(torch.int16)) and torch.equal(v2.contiguous().view(torch.int16), v.view(torch.int16))


def test_tensors_that_are_written_tell_so():
    b = Batch([3, 1], [40, 20], 4, 2, 64, 16, BF16)
    k, v, table, q_begin, kv_len = b.cache()
    q, new = b.q.to(DEV), torch.randn(4, 2, 64, device=DEV).to(BF16)
    q_out, out, hists = torch.empty_like(q), torch.empty_like(q), torch.zeros((4, 256), dtype=torch.int32, device=DEV)
    read, put, got = (q, new, table, q_begin, kv_len), (k, v, q_out, hists), (out,)
    was = [[t._version for t in g] for g in (read, put, got)]
    sz.append_kv(new, new, k, v, table, q_begin, kv_len, q=q, q_out=q_out, hists=hists)
    assert [t._version for t in put] == [n + 1 for n in was[1]]
    sz.paged_attention(q_out, k, v, table, q_begin, kv_len, out=out)
    assert [t._version for t in got] == [n + 1 for n in was[2]] and [t._version for t in put] == [n + 1 for n in was[1]]
    assert [t._version for t in read] == was[0]
    w = torch.ones(64, dtype=BF16, device=DEV, requires_grad=True)
    y = (out * w).sum()  # `out` is saved
    sz.paged_attention(q_out, k, v, table, q_begin, kv_len, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        k2, v2 = k.clone(), v.clone()
        sz.append_kv(new, new, k2, v2, table, q_begin, kv_len)
    _, status = sz.append_kv(new, new, k2, v2, table, q_begin, kv_len)  # and outside of it
    assert not status.any() and torch.equal(k2.view(torch.int16), k.view(torch.int16))


# --------------------------------------------------------------- together
def test_prefill_transfer_and_continue():
    """A prefill in chunks writes the cache and counts it, the codec ships the
    pages to another pool, and decoding continues there: the containers are
    the two-pass call's, and attention over the rebuilt pages is bit for bit
    attention over the originals."""
    R, HQ, HK, D, P = 3, 8, 2, 128, 16
    total = [160, 64, 336]
    g = torch.Generator(device=DEV).manual_seed(5)
    pages = sum(total) // P + R + 5
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    width = max(total) // P + 1
    table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r in range(R):
        table[r, : total[r] // P + 1] = perm[at: at + total[r] // P + 1]
        at += total[r] // P + 1
    k, v = (torch.zeros((pages, HK, P, D), dtype=BF16, device=DEV) for _ in range(2))
    hists = torch.zeros((2 * R, 256), dtype=torch.int32, device=DEV)
    freqs = sz.rope_frequencies(D, 500000.0, device=DEV)
    norm = torch.ones(D, dtype=BF16, device=DEV)
    done = [0] * R
    outs = []
    for share in (0.4, 1.0):
        new = [int(total[r] * share) - done[r] for r in range(R)]
        done = [d + n for d, n in zip(done, new)]
        q_begin = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
        kv_len = torch.tensor(done, dtype=torch.int32, device=DEV)
        row = torch.randn((sum(new), HQ + 2 * HK, D), generator=g, device=DEV).to(BF16)
        q, st = sz.append_kv(row[:, HQ:HQ + HK], row[:, HQ + HK:], k, v, table, q_begin, kv_len, q=row[:, :HQ], rope_freqs=freqs,
                             q_norm=norm, k_norm=norm, hists=hists)
        out, _, st2 = sz.paged_attention(q, k, v, table, q_begin, kv_len)
        assert not st.any() and not st2.any()
        want = ref.attention(q.cpu(), k.cpu(), v.cpu(), table.cpu(), q_begin.cpu(), kv_len.cpu(), 1 / math.sqrt(D))
        check(out, want[0], want[2])
        outs.append(out)
    # the codec: keys of every request, then values, each request's pages one stream
    elems = HK * P * D
    lens = [n * HK * D for n in total] * 2
    src = torch.cat([(t.data_ptr() + 2 * elems * table[r, : total[r] // P].long()) for t in (k, v) for r in range(R)])
    plan = sz.BatchPlan(lens, elems, device=DEV)
    cbs, _ = sz.select_codebooks(hists)
    plan.encode_one_pass(src, cbs)
    twice = sz.BatchPlan(lens, elems, device=DEV)
    twice.encode(src)
    torch.cuda.synchronize()
    assert not plan.enc_status.any() and not twice.enc_status.any()
    assert torch.equal(plan.sizes, twice.sizes)
    for i in range(2 * R):
        n = int(plan.sizes[i])
        assert np.array_equal(plan.container_bytes(i, n), twice.container_bytes(i, n))
    # the other side: its own pool and pages
    k2, v2 = (torch.full_like(k, math.nan) for _ in range(2))
    table2 = torch.where(table >= 0, pages - 1 - table, table)
    dst = torch.cat([(t.data_ptr() + 2 * elems * table2[r, : total[r] // P].long()) for t in (k2, v2) for r in range(R)])
    plan.decode(dst)
    assert not plan.dec_status.any()
    q_begin = torch.arange(R + 1, dtype=torch.int32, device=DEV)
    kv_len = torch.tensor([n + 1 for n in total], dtype=torch.int32, device=DEV)
    row = torch.randn((R, HQ + 2 * HK, D), generator=g, device=DEV).to(BF16)
    got = []
    for kk, vv, tt in ((k, v, table), (k2, v2, table2)):
        q, st = sz.append_kv(row[:, HQ:HQ + HK], row[:, HQ + HK:], kk, vv, tt, q_begin, kv_len, q=row[:, :HQ], rope_freqs=freqs,
                             q_norm=norm, k_norm=norm)
        out, _, st2 = sz.paged_attention(q, kk, vv, tt, q_begin, kv_len)
        assert not st.any() and not st2.any()
        got.append(out)
    assert torch.equal(got[0], got[1])
