// sz_binding.cpp -- the Python side of sz_append_kv and sz_paged_attention:
// checks of the tensors, new tensors for the results, the call.
//
// A decode step makes these calls once per layer.  With the checks and the
// packing of the arguments in Python a call took the host 16.5 us (a single
// token's append and its attention take the GPU 4.6 and 12 us); here it takes
// 6.6 us for an append, 7.4 us for an attention of one launch and 11 us for one
// of two, most of which are the launches and the allocation of the results.  The C entry
// points are those of the library that the package has loaded (init), and
// the errors that they return go back as their codes.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <optional>

#include "splitzip.h"

namespace {

using Append = sz_status (*)(const sz_paged_kv *, const sz_append_args *, int32_t *, void *);
using Attention = sz_status (*)(const sz_paged_kv *, const sz_attention_args *, int32_t *, void *, uint64_t, void *);
Append g_append = nullptr;
Attention g_attention = nullptr;

// A Python exception on its way: its type and text are set already.
struct Raised {};
[[noreturn]] void fail(PyObject *type, const char *format, ...) {
    va_list a;
    va_start(a, format);
    char text[512];
    vsnprintf(text, sizeof text, format, a);
    va_end(a);
    PyErr_SetString(type, text);
    throw Raised();
}

std::string shape_of(const at::Tensor &t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}
const char *type_of(const at::Tensor &t) { return toString(t.scalar_type()); }

// An argument that is a tensor, or None where that is allowed.
const at::Tensor *tensor(PyObject *o, const char *name, bool optional) {
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}

void *at(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

void ints(const at::Tensor &t, const char *name, int64_t dims) {
    if (t.scalar_type() != at::kInt || t.dim() != dims || (t.size(dims - 1) > 1 && t.stride(dims - 1) != 1))
        fail(PyExc_ValueError, "%s must be an int32 tensor of %d dimension(s) with entries side by side", name, (int)dims);
}

// Neither direction of differentiation goes through these operators.
void no_gradient(const at::Tensor &t, const char *name) {
    if (!t.unsafeGetTensorImpl()->autograd_meta()) return;
    if (t.requires_grad() && c10::GradMode::is_enabled()) fail(PyExc_ValueError, "%s requires a gradient, and this operator has none", name);
    if (t._fw_grad(0).defined()) fail(PyExc_ValueError, "%s carries a tangent, and this operator has none", name);
}

// A tensor of the caller's that the call writes: whoever saved it for a
// gradient finds out.  (Tensors of inference mode have no version.)
void written(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Rows [tokens, heads, dim]; returns the heads.
uint32_t rows(const at::Tensor &t, const char *name, at::ScalarType type, int64_t tokens, int64_t dim, uint64_t (&stride)[2]) {
    if (t.scalar_type() != type || t.dim() != 3 || t.size(0) != tokens || t.size(2) != dim)
        fail(PyExc_ValueError, "%s must be %s [%lld tokens, heads, %lld], got %s %s", name, toString(type), (long long)tokens, (long long)dim,
             type_of(t), shape_of(t).c_str());
    if (t.size(1) > UINT32_MAX) fail(PyExc_ValueError, "%s has 2^32 heads or more", name);
    if (t.stride(2) != 1) fail(PyExc_ValueError, "%s needs its channels side by side", name);
    no_gradient(t, name);
    stride[0] = (uint64_t)t.stride(0);
    stride[1] = (uint64_t)t.stride(1);
    return (uint32_t)t.size(1);
}

sz_paged_kv cache(const at::Tensor &k, const at::Tensor &v, const at::Tensor &table, const at::Tensor &q_begin, const at::Tensor &kv_len,
                  int64_t tokens) {
    if ((k.scalar_type() != at::kBFloat16 && k.scalar_type() != at::kHalf) || v.scalar_type() != k.scalar_type())
        fail(PyExc_TypeError, "pages are bfloat16 or float16, the same for keys and values; got %s and %s", type_of(k), type_of(v));
    if (k.dim() != 4 || v.sizes() != k.sizes())
        fail(PyExc_ValueError, "pages are two tensors [pages, heads, page tokens, channels] of one shape");
    if (k.stride(3) != 1 || v.stride(3) != 1) fail(PyExc_ValueError, "pages need their channels side by side");
    no_gradient(k, "k_pages");
    no_gradient(v, "v_pages");
    ints(table, "page_table", 2);
    ints(q_begin, "q_begin", 1);
    ints(kv_len, "kv_len", 1);
    const int64_t reqs = table.size(0);
    if (q_begin.size(0) != reqs + 1 || kv_len.size(0) != reqs)
        fail(PyExc_ValueError, "%lld requests in page_table, %lld in q_begin, %lld in kv_len", (long long)reqs, (long long)q_begin.size(0) - 1,
             (long long)kv_len.size(0));
    if (reqs > UINT32_MAX || k.size(1) > UINT32_MAX || k.size(2) > UINT32_MAX || k.size(3) > UINT32_MAX || table.size(1) > UINT32_MAX)
        fail(PyExc_ValueError, "a dimension is 2^32 or larger");
    sz_paged_kv p{};
    p.d_k = k.data_ptr();
    p.d_v = v.data_ptr();
    for (int i = 0; i < 3; ++i) {
        const int from[3] = {0, 1, 2};  // pages, heads, tokens
        p.k_stride[i] = (uint64_t)k.stride(from[i]);
        p.v_stride[i] = (uint64_t)v.stride(from[i]);
    }
    p.n_pages = (uint64_t)k.size(0);
    p.heads = (uint32_t)k.size(1);
    p.page_tokens = (uint32_t)k.size(2);
    p.head_dim = (uint32_t)k.size(3);
    p.dtype = k.scalar_type() == at::kBFloat16 ? SZ_BF16 : SZ_FP16;
    p.d_page_table = static_cast<const int32_t *>(table.data_ptr());
    p.max_pages = (uint32_t)table.size(1);
    p.table_stride = reqs > 1 ? (uint64_t)table.stride(0) : p.max_pages;
    p.d_q_begin = static_cast<const int32_t *>(q_begin.data_ptr());
    p.d_kv_len = static_cast<const int32_t *>(kv_len.data_ptr());
    p.n_reqs = (uint32_t)reqs;
    p.n_tokens = (uint64_t)tokens;
    return p;
}

// The tensors' one CUDA device, made current, and the stream of the call:
// the given one (also for what is allocated meanwhile), or the current one.
class On {
  public:
    On(std::initializer_list<const at::Tensor *> tensors, PyObject *stream) {
        const at::Tensor *first = *tensors.begin();
        for (const at::Tensor *t : tensors)
            if (t && t->device() != first->device())
                fail(PyExc_ValueError, "tensors on %s and %s", first->device().str().c_str(), t->device().str().c_str());
        if (!first->is_cuda()) fail(PyExc_ValueError, "the tensors must be on a CUDA device, not on %s", first->device().str().c_str());
        const c10::DeviceIndex device = first->device().index();
        if (stream == Py_None) {
            if (c10::cuda::current_device() != device) device_.emplace(device);
            stream_ = c10::cuda::getCurrentCUDAStream(device).stream();
        } else {
            stream_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
            if (PyErr_Occurred()) throw Raised();
            device_.emplace(device);
            on_stream_.emplace(c10::cuda::getStreamFromExternal(stream_, device));
        }
    }
    void *stream() const { return stream_; }

  private:
    std::optional<c10::cuda::CUDAGuard> device_;
    std::optional<c10::cuda::CUDAStreamGuard> on_stream_;
    cudaStream_t stream_ = nullptr;
};

double number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised();
    return x;
}
bool truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Raised();
    return x != 0;
}
PyObject *wrap(const at::Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
PyObject *object(PyObject *given, const at::Tensor &made) {
    if (given != Py_None) {
        Py_INCREF(given);
        return given;
    }
    return wrap(made);
}

// (code, results ...): the caller raises a code other than 0.
PyObject *append_kv(PyObject *const *a, Py_ssize_t n) {
    if (n != 19) fail(PyExc_TypeError, "append_kv takes 19 arguments");
    const at::Tensor &k = *tensor(a[0], "k", false), &v = *tensor(a[1], "v", false), &kp = *tensor(a[2], "k_pages", false),
                     &vp = *tensor(a[3], "v_pages", false), &table = *tensor(a[4], "page_table", false), &q_begin = *tensor(a[5], "q_begin", false),
                     &kv_len = *tensor(a[6], "kv_len", false);
    const at::Tensor *q = tensor(a[7], "q", true), *q_out = tensor(a[8], "q_out", true), *freqs = tensor(a[9], "rope_freqs", true),
                     *positions = tensor(a[12], "positions", true), *q_norm = tensor(a[13], "q_norm", true), *k_norm = tensor(a[14], "k_norm", true),
                     *hists = tensor(a[16], "hists", true), *hist_rows = tensor(a[17], "hist_rows", true);
    if (k.dim() != 3) fail(PyExc_ValueError, "k must be [tokens, heads, channels], got %s", shape_of(k).c_str());
    const int64_t tokens = k.size(0);
    const sz_paged_kv kv = cache(kp, vp, table, q_begin, kv_len, tokens);
    const at::ScalarType type = kp.scalar_type();
    const int64_t dim = kp.size(3);
    sz_append_args x{};
    const uint32_t hk = rows(k, "k", type, tokens, dim, x.k_stride), hv = rows(v, "v", type, tokens, dim, x.v_stride);
    if (hk != kv.heads || hv != kv.heads) fail(PyExc_ValueError, "pages of %u heads, k of %u, v of %u", kv.heads, hk, hv);
    if (q) {
        x.q_heads = rows(*q, "q", type, tokens, dim, x.q_stride);
        if (q_out && q_out->sizes() != q->sizes())
            fail(PyExc_ValueError, "q_out of shape %s for q of %s", shape_of(*q_out).c_str(), shape_of(*q).c_str());
    } else if (q_out || q_norm) {
        fail(PyExc_ValueError, "q_out and q_norm need q");
    }
    if (freqs) {
        if (freqs->scalar_type() != at::kDouble || freqs->dim() != 1 || !freqs->is_contiguous())
            fail(PyExc_ValueError, "rope_freqs must be a contiguous float64 vector");
        no_gradient(*freqs, "rope_freqs");
        if (freqs->size(0) > 1 << 20) fail(PyExc_ValueError, "rope_freqs of %lld pairs", (long long)freqs->size(0));
        x.rot_dim = (uint32_t)(2 * freqs->size(0));
    }
    if (positions && (positions->scalar_type() != at::kLong || positions->dim() != 1 || positions->size(0) != tokens || !positions->is_contiguous()))
        fail(PyExc_ValueError, "positions must be a contiguous int64 tensor [%lld]", (long long)tokens);
    for (const at::Tensor *w : {q_norm, k_norm}) {
        if (!w) continue;
        const char *const name = w == q_norm ? "q_norm" : "k_norm";
        if (w->scalar_type() != type || w->dim() != 1 || w->size(0) != dim || !w->is_contiguous())
            fail(PyExc_ValueError, "%s must be a contiguous %s tensor [%lld]", name, toString(type), (long long)dim);
        no_gradient(*w, name);
    }
    if (hists) {
        if ((hists->scalar_type() != at::kInt && hists->scalar_type() != at::kUInt32) || hists->dim() < 1 || hists->size(-1) != 256 ||
            !hists->is_contiguous() || hists->numel() / 256 > UINT32_MAX)
            fail(PyExc_ValueError, "hists must be a contiguous 32-bit tensor of rows of 256 counts");
        x.n_hists = (uint32_t)(hists->numel() / 256);
    }
    if (hist_rows) {
        if (!hists) fail(PyExc_ValueError, "hist_rows needs hists");
        if ((hist_rows->scalar_type() != at::kInt && hist_rows->scalar_type() != at::kUInt32) || hist_rows->numel() != 2 * (int64_t)kv.n_reqs ||
            !hist_rows->is_contiguous())
            fail(PyExc_ValueError, "hist_rows must be a contiguous 32-bit tensor of %lld rows", 2ll * kv.n_reqs);
    }
    const bool interleaved = truth(a[10]);
    const double rot_scale = number(a[11]), eps = number(a[15]);
    const On on({&kp, &vp, &k, &v, &table, &q_begin, &kv_len, q, q_out, freqs, positions, q_norm, k_norm, hists, hist_rows}, a[18]);
    const at::Tensor status = at::empty({(int64_t)kv.n_reqs}, kv_len.options());
    at::Tensor made;
    if (q) {
        if (!q_out) made = at::empty(q->sizes(), q->options());
        rows(q_out ? *q_out : made, "q_out", type, tokens, dim, x.q_out_stride);
        x.d_q_or_null = q->data_ptr();
        x.d_q_out = q_out ? q_out->data_ptr() : made.data_ptr();
    }
    x.d_k = k.data_ptr();
    x.d_v = v.data_ptr();
    x.d_q_norm_or_null = at(q_norm);
    x.d_k_norm_or_null = at(k_norm);
    x.d_freqs_or_null = static_cast<const double *>(at(freqs));
    x.d_positions_or_null = static_cast<const int64_t *>(at(positions));
    x.d_hists_or_null = static_cast<uint32_t *>(at(hists));
    x.d_hist_rows_or_null = static_cast<const uint32_t *>(at(hist_rows));
    written(kp);
    written(vp);
    if (q_out) written(*q_out);
    if (hists) written(*hists);
    x.interleaved = interleaved ? 1 : 0;
    x.rot_scale = (float)rot_scale;
    x.eps = (float)eps;
    sz_status st;
    int32_t *const d_status = static_cast<int32_t *>(status.data_ptr());
    Py_BEGIN_ALLOW_THREADS
    st = g_append(&kv, &x, d_status, on.stream());
    Py_END_ALLOW_THREADS
    return Py_BuildValue("iNN", (int)st, q ? object(a[8], made) : object(Py_None, at::Tensor()), wrap(status));
}

PyObject *paged_attention(PyObject *const *a, Py_ssize_t n) {
    if (n != 14) fail(PyExc_TypeError, "paged_attention takes 14 arguments");
    const at::Tensor &q = *tensor(a[0], "q", false), &kp = *tensor(a[1], "k_pages", false), &vp = *tensor(a[2], "v_pages", false),
                     &table = *tensor(a[3], "page_table", false), &q_begin = *tensor(a[4], "q_begin", false), &kv_len = *tensor(a[5], "kv_len", false);
    const at::Tensor *out = tensor(a[9], "out", true), *workspace = tensor(a[11], "workspace", true);
    if (q.dim() != 3) fail(PyExc_ValueError, "q must be [tokens, heads, channels], got %s", shape_of(q).c_str());
    const int64_t tokens = q.size(0);
    const sz_paged_kv kv = cache(kp, vp, table, q_begin, kv_len, tokens);
    const at::ScalarType type = kp.scalar_type();
    const int64_t dim = kp.size(3);
    sz_attention_args x{};
    x.q_heads = rows(q, "q", type, tokens, dim, x.q_stride);
    if (out && out->sizes() != q.sizes()) fail(PyExc_ValueError, "out of shape %s for q of %s", shape_of(*out).c_str(), shape_of(q).c_str());
    x.scale = a[6] == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : (float)number(a[6]);
    x.causal = truth(a[7]) ? 1 : 0;
    const long long window = PyLong_AsLongLong(a[8]);
    if (window == -1 && PyErr_Occurred()) throw Raised();
    if (window < 0 || window > UINT32_MAX) fail(PyExc_ValueError, "window must be 0 (none) or a number of keys below 2^32");
    x.window = (uint32_t)window;
    const bool with_lse = truth(a[10]);
    const long long need = PyLong_AsLongLong(a[12]);
    if (need == -1 && PyErr_Occurred()) throw Raised();
    const On on({&kp, &vp, &q, &table, &q_begin, &kv_len, out, workspace}, a[13]);
    if (workspace && (!workspace->is_contiguous() || (long long)workspace->nbytes() < need))
        fail(PyExc_ValueError, "workspace must be contiguous and holds %lld bytes, the call needs %lld", (long long)workspace->nbytes(), need);
    at::Tensor ws, made, lse;
    if (!workspace) ws = at::empty({need}, q.options().dtype(at::kByte));
    if (!out) made = at::empty(q.sizes(), q.options());
    if (with_lse) lse = at::empty({tokens, (int64_t)x.q_heads}, q.options().dtype(at::kFloat));
    const at::Tensor status = at::empty({(int64_t)kv.n_reqs}, kv_len.options());
    rows(out ? *out : made, "out", type, tokens, dim, x.out_stride);
    if (out) written(*out);
    x.d_q = q.data_ptr();
    x.d_out = out ? out->data_ptr() : made.data_ptr();
    x.d_lse_or_null = with_lse ? static_cast<float *>(lse.data_ptr()) : nullptr;
    const at::Tensor &w = workspace ? *workspace : ws;
    sz_status st;
    int32_t *const d_status = static_cast<int32_t *>(status.data_ptr());
    void *const d_ws = w.data_ptr();
    const uint64_t ws_bytes = (uint64_t)w.nbytes();
    Py_BEGIN_ALLOW_THREADS
    st = g_attention(&kv, &x, d_status, d_ws, ws_bytes, on.stream());
    Py_END_ALLOW_THREADS
    return Py_BuildValue("iNNN", (int)st, object(a[9], made), wrap(lse), wrap(status));
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS  // C++ exceptions of the tensor library become Python's
    try {
        return F(args, n);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *init(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "init takes the addresses of sz_append_kv and sz_paged_attention");
        return nullptr;
    }
    g_append = reinterpret_cast<Append>(PyLong_AsVoidPtr(args[0]));
    g_attention = reinterpret_cast<Attention>(PyLong_AsVoidPtr(args[1]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", (PyCFunction)(void *)init, METH_FASTCALL, nullptr},
    {"append_kv", (PyCFunction)(void *)entry<append_kv>, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void *)entry<paged_attention>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
// The module's docstring: what this file was compiled against, which the build
// looks for in it.
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", SZ_MADE_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
