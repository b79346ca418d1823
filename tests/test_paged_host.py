"""Host side of the paged-cache operators: argument errors come back before
anything reaches a device, and the frequency tables follow their formulas."""
import ctypes
import math

import pytest

import lossless_bf16_kv_splitzip_b200 as sz

torch = pytest.importorskip("torch")

A = 1 << 40  # a 16-byte aligned fake device address, never dereferenced


def cache(**kw):
    d = dict(d_k=A, d_v=A, k_stride=(16384, 2048, 128), v_stride=(16384, 2048, 128), n_pages=10, heads=8, head_dim=128, page_tokens=16,
             dtype=1, d_page_table=A, table_stride=4, d_q_begin=A, d_kv_len=A, n_reqs=2, max_pages=4, n_tokens=5)
    d.update(kw)
    for k in ("k_stride", "v_stride"):
        d[k] = (ctypes.c_uint64 * 3)(*d[k])
    return sz.sz_paged_kv(**d)


def append(**kw):
    d = dict(d_k=A, d_v=A, k_stride=(1024, 128), v_stride=(1024, 128), d_q_or_null=A, d_q_out=A, q_stride=(4096, 128),
             q_out_stride=(4096, 128), d_freqs_or_null=A, q_heads=32, rot_dim=128, rot_scale=1.0, eps=1e-6)
    d.update(kw)
    for k in ("k_stride", "v_stride", "q_stride", "q_out_stride"):
        d[k] = (ctypes.c_uint64 * 2)(*d[k])
    return sz.sz_append_args(**d)


def attn(**kw):
    d = dict(d_q=A, d_out=A, q_stride=(4096, 128), out_stride=(4096, 128), q_heads=32, causal=1, window=0, scale=0.1)
    d.update(kw)
    for k in ("q_stride", "out_stride"):
        d[k] = (ctypes.c_uint64 * 2)(*d[k])
    return sz.sz_attention_args(**d)


def status(f, *args):
    with pytest.raises(sz.SzError) as e:
        f(*args)
    return e.value.status


CACHE_ERRORS = [
    (dict(d_k=None), sz.SZ_ERR_NULL), (dict(d_q_begin=None), sz.SZ_ERR_NULL), (dict(d_kv_len=None), sz.SZ_ERR_NULL),
    (dict(d_page_table=None), sz.SZ_ERR_NULL), (dict(d_v=A + 8), sz.SZ_ERR_ALIGN), (dict(d_kv_len=A + 2), sz.SZ_ERR_ALIGN),
    (dict(dtype=0), sz.SZ_ERR_INVALID), (dict(dtype=3), sz.SZ_ERR_INVALID), (dict(heads=0), sz.SZ_ERR_INVALID),
    (dict(head_dim=0), sz.SZ_ERR_INVALID), (dict(head_dim=100), sz.SZ_ERR_INVALID), (dict(head_dim=264), sz.SZ_ERR_INVALID),
    (dict(page_tokens=0), sz.SZ_ERR_INVALID), (dict(table_stride=3), sz.SZ_ERR_INVALID),
    (dict(max_pages=1 << 28, table_stride=1 << 28), sz.SZ_ERR_TOO_LARGE), (dict(n_tokens=1 << 31), sz.SZ_ERR_TOO_LARGE),
    (dict(n_pages=1 << 31), sz.SZ_ERR_TOO_LARGE),
    (dict(k_stride=(16384, 2048, 130)), sz.SZ_ERR_ALIGN),
    (dict(k_stride=(16384, 2048, 64)), sz.SZ_ERR_INVALID),  # tokens overlap
    (dict(v_stride=(8192, 2048, 128)), sz.SZ_ERR_INVALID),  # pages overlap
    (dict(v_stride=(0, 2048, 128)), sz.SZ_ERR_INVALID),
    (dict(k_stride=(1 << 40, 2048, 128)), sz.SZ_ERR_TOO_LARGE),
]


@pytest.mark.parametrize("change,want", CACHE_ERRORS)
def test_cache_errors(change, want):
    assert status(sz.sz_append_kv, cache(**change), append(), A, 0) == want
    assert status(sz.sz_paged_attention, cache(**change), attn(), A, A, 1 << 40, 0) == want


@pytest.mark.parametrize("change,want", [
    (dict(d_k=None), sz.SZ_ERR_NULL), (dict(d_v=None), sz.SZ_ERR_NULL), (dict(d_q_or_null=None), sz.SZ_ERR_NULL),
    (dict(d_q_out=None), sz.SZ_ERR_NULL), (dict(d_freqs_or_null=None), sz.SZ_ERR_NULL), (dict(d_k=A + 4), sz.SZ_ERR_ALIGN),
    (dict(v_stride=(1024, 100)), sz.SZ_ERR_ALIGN), (dict(q_stride=(4100, 128)), sz.SZ_ERR_ALIGN),
    (dict(q_out_stride=(4096, 64)), sz.SZ_ERR_INVALID), (dict(rot_dim=120), sz.SZ_ERR_INVALID),
    (dict(rot_dim=144), sz.SZ_ERR_INVALID), (dict(d_k_norm_or_null=A + 2), sz.SZ_ERR_ALIGN),
    (dict(d_positions_or_null=A + 4), sz.SZ_ERR_ALIGN), (dict(n_hists=4), sz.SZ_ERR_NULL),
])
def test_append_errors(change, want):
    assert status(sz.sz_append_kv, cache(), append(**change), A, 0) == want


@pytest.mark.parametrize("change,want", [
    (dict(d_q=None), sz.SZ_ERR_NULL), (dict(d_out=None), sz.SZ_ERR_NULL), (dict(d_out=A + 2), sz.SZ_ERR_ALIGN),
    (dict(q_heads=0), sz.SZ_ERR_INVALID), (dict(q_heads=12), sz.SZ_ERR_INVALID), (dict(window=5, causal=0), sz.SZ_ERR_INVALID),
    (dict(out_stride=(128, 128)), sz.SZ_ERR_INVALID), (dict(q_stride=(4096, 4)), sz.SZ_ERR_ALIGN),
    (dict(d_lse_or_null=A + 1), sz.SZ_ERR_ALIGN),
])
def test_attention_errors(change, want):
    assert status(sz.sz_paged_attention, cache(), attn(**change), A, A, 1 << 40, 0) == want


def test_workspace_and_status_are_required():
    need = sz.sz_plan_attention(128)
    assert need > 0
    assert status(sz.sz_paged_attention, cache(), attn(), A, A, need - 1, 0) == sz.SZ_ERR_WORKSPACE
    assert status(sz.sz_paged_attention, cache(), attn(), A, A + 8, need, 0) == sz.SZ_ERR_ALIGN
    assert status(sz.sz_paged_attention, cache(), attn(), None, A, need, 0) == sz.SZ_ERR_NULL
    assert status(sz.sz_paged_attention, cache(), attn(), A, None, need, 0) == sz.SZ_ERR_NULL
    assert status(sz.sz_append_kv, cache(), append(), None, 0) == sz.SZ_ERR_NULL
    for dim in (0, 12, 264):
        assert status(sz.sz_plan_attention, dim) == sz.SZ_ERR_INVALID


def test_nothing_to_do():
    sz.sz_append_kv(cache(n_reqs=0), append(), None, 0)
    sz.sz_paged_attention(cache(n_reqs=0), attn(), None, None, 0, 0)


# ---- the helpers' own checks, on host tensors
def tensors(dtype=torch.bfloat16, heads=8, kv_heads=2, dim=64, tokens=3):
    z = lambda *s, t=dtype: torch.zeros(s, dtype=t)  # noqa: E731
    return dict(q=z(tokens, heads, dim), k=z(tokens, kv_heads, dim), v=z(tokens, kv_heads, dim), k_pages=z(4, kv_heads, 16, dim),
                v_pages=z(4, kv_heads, 16, dim), page_table=z(1, 2, t=torch.int32), q_begin=z(2, t=torch.int32), kv_len=z(1, t=torch.int32))


def attend(t, **kw):
    return sz.paged_attention(t["q"], t["k_pages"], t["v_pages"], t["page_table"], t["q_begin"], t["kv_len"], **kw)


def put(t, **kw):
    return sz.append_kv(t["k"], t["v"], t["k_pages"], t["v_pages"], t["page_table"], t["q_begin"], t["kv_len"], **kw)


@pytest.mark.parametrize("change,match", [
    (dict(k_pages=torch.zeros(4, 2, 16, 64)), "bfloat16 or float16"),
    (dict(v_pages=torch.zeros(4, 2, 16, 64, dtype=torch.float16)), "the same"),
    (dict(v_pages=torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16)), "one shape"),
    (dict(k_pages=torch.zeros(4, 2, 64, 16, dtype=torch.bfloat16).transpose(2, 3)), "side by side"),
    (dict(page_table=torch.zeros(1, 2, dtype=torch.int64)), "page_table"),
    (dict(page_table=torch.zeros(1, 4, dtype=torch.int32)[:, ::2]), "page_table"),
    (dict(q_begin=torch.zeros(3, dtype=torch.int32)), "requests"),
    (dict(kv_len=torch.zeros(1, dtype=torch.float32)), "kv_len"),
])
def test_helpers_refuse_bad_caches(change, match):
    t = tensors()
    t.update(change)
    for call in (lambda: attend(t), lambda: put(t)):
        with pytest.raises((ValueError, TypeError), match=match):
            call()


def test_helpers_refuse_bad_rows():
    t = tensors()
    with pytest.raises(ValueError, match="CUDA device"):
        attend(t)
    with pytest.raises(ValueError, match="CUDA device"):
        put(t)
    for bad in (dict(q=t["q"].half()), dict(q=t["q"][..., :32]), dict(q=t["q"].repeat(1, 1, 2)[..., ::2])):
        with pytest.raises(ValueError, match="q "):
            attend({**t, **bad})
    with pytest.raises(ValueError, match="gradient"):
        attend({**t, "q": t["q"].clone().requires_grad_()})
    with pytest.raises(ValueError, match="gradient"):
        put({**t, "k": t["k"].clone().requires_grad_()})
    with pytest.raises(ValueError, match="out of shape"):
        attend(t, out=t["q"][:2])
    with pytest.raises(ValueError, match="window"):
        attend(t, window=-1)
    with pytest.raises(ValueError, match="heads"):
        put({**t, "k": t["q"], "v": t["q"]})
    with pytest.raises(ValueError, match="need q"):
        put(t, q_norm=torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="k_norm"):
        put(t, k_norm=torch.ones(64))
    with pytest.raises(ValueError, match="rope_freqs"):
        put(t, rope_freqs=torch.ones(32))
    with pytest.raises(ValueError, match="positions"):
        put(t, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="hists"):
        put(t, hists=torch.zeros(2, 128, dtype=torch.int32))
    with pytest.raises(ValueError, match="hist_rows"):
        put(t, hist_rows=torch.zeros(2, dtype=torch.int32))


# ---- frequency tables
def test_frequencies():
    f = sz.rope_frequencies(64, 10000.0)
    assert f.dtype == torch.float64 and f.shape == (32,)
    for t in (0, 1, 17, 31):
        assert math.isclose(float(f[t]), 10000.0 ** (-2 * t / 64), rel_tol=1e-14)
    assert torch.allclose(sz.rope_frequencies(64, 10000.0, scaling="linear", factor=4.0), f / 4, rtol=1e-15, atol=0)
    g = sz.rope_frequencies(64, 10000.0, scaling="base", factor=8.0)
    assert float(g[0]) == 1.0 and math.isclose(float(g[31]), float(f[31]) / 8, rel_tol=1e-12)
    assert bool((g[1:] < f[1:]).all()) and bool((g >= f / 8 * (1 - 1e-12)).all())


def test_frequencies_in_bands():
    f = sz.rope_frequencies(128, 500000.0)
    g = sz.rope_frequencies(128, 500000.0, scaling="bands", factor=8.0, trained_len=8192)
    for t in range(64):
        turns = float(f[t]) * 8192 / (2 * math.pi)
        want = float(f[t]) if turns >= 4 else float(f[t]) / 8 if turns <= 1 else \
            float(f[t]) * ((turns - 1) / 3 + (1 - (turns - 1) / 3) / 8)
        assert math.isclose(float(g[t]), want, rel_tol=1e-12)
    with pytest.raises(ValueError, match="trained_len"):
        sz.rope_frequencies(128, scaling="bands", factor=8.0)
    with pytest.raises(ValueError, match="scaling"):
        sz.rope_frequencies(128, scaling="other")
    for bad in (0, 7):
        with pytest.raises(ValueError, match="rot_dim"):
            sz.rope_frequencies(bad)


def test_gradients_are_refused_only_where_they_are_recorded():
    t = tensors()
    w = torch.nn.Parameter(torch.ones(t["q"].shape[2], dtype=t["q"].dtype))
    with pytest.raises(ValueError, match="k_norm requires a gradient"):
        put(t, k_norm=w)
    with pytest.raises(ValueError, match="k_pages requires a gradient"):
        attend({**t, "k_pages": t["k_pages"].clone().requires_grad_()})
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):  # the next check
        put({**t, "k": t["k"].clone().requires_grad_()}, k_norm=w)


def test_learned_frequencies_and_tangents_are_refused():
    import torch.autograd.forward_ad as fwd
    t = tensors()
    with pytest.raises(ValueError, match="rope_freqs requires a gradient"):
        put(t, rope_freqs=sz.rope_frequencies(64).requires_grad_())
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):  # the next check
        put(t, rope_freqs=sz.rope_frequencies(64).requires_grad_())
    with fwd.dual_level():
        for name, call in (("q", attend), ("k_pages", attend), ("v_pages", put), ("k", put), ("v", put)):
            dual = fwd.make_dual(t[name], torch.ones_like(t[name]))
            with pytest.raises(ValueError, match=name + " carries a tangent"):
                call({**t, name: dual})
        w = torch.ones(t["q"].shape[2], dtype=t["q"].dtype)
        with pytest.raises(ValueError, match="k_norm carries a tangent"):
            put(t, k_norm=fwd.make_dual(w, w))


def test_a_binding_of_another_torch_is_built_anew(monkeypatch):
    from lossless_bf16_kv_splitzip_b200 import _build
    sz.paged.binding()
    assert not _build.binding_is_stale()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "1")
    assert _build.binding_is_stale()
    monkeypatch.undo()
    assert not _build.binding_is_stale()
    monkeypatch.setattr("sysconfig.get_config_var", lambda name: "cpython-39")
    assert _build.binding_is_stale()
