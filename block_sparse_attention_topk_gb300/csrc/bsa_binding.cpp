// bsa_binding.cpp -- argument checks and marshalling of the cache operators
// (bsa_rope, bsa_append_kv_*, bsa_sparse_decode_attention_q8) for Python.
//
// A decode step calls these on a few rows, where a call's kernels take 4 to 10
// us.  Checking a dozen tensors attribute by attribute in Python and passing 20
// arguments through ctypes took 8 to 10 us more; here it takes under one.  Every
// argument is checked before anything is launched, and a mismatch raises
// ValueError; the C call's own refusals raise BsaError, as in the rest of the
// package.  PyTorch supplies tensors, memory and streams only.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <initializer_list>
#include <string>

#include "../../include/bsa_topk.h"
#include "bsa_overlap.h"

namespace {

PyObject* g_error = nullptr;        // BsaError(fn, status, message)
PyObject* g_raw_stream = nullptr;   // device index -> cudaStream_t of the current stream
PyObject* g_workspace = nullptr;    // (device, bytes) -> the device's and stream's workspace

using at::Tensor;

bool fail(const char* format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(PyExc_ValueError, format, args);
    va_end(args);
    return false;
}

// The tensor of an argument; null for None and (with an error set) for others.
bool tensor(PyObject* o, const char* name, const Tensor** t) {
    *t = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) return fail("%s must be a tensor", name);
    *t = &THPVariable_Unpack(o);
    return true;
}
bool needed(PyObject* o, const char* name, const Tensor** t) {
    if (!tensor(o, name, t)) return false;
    return *t != nullptr || fail("%s is needed", name);
}

// A contiguous tensor of this type, place and shape (-1: any size).
bool whole(const Tensor& t, const char* name, at::ScalarType type, const at::Device& device,
           std::initializer_list<int64_t> shape) {
    bool ok = t.scalar_type() == type && t.device() == device && t.dim() == (int64_t)shape.size() && t.is_contiguous();
    int64_t i = 0;
    for (int64_t n : shape) {
        if (ok && n >= 0 && t.size(i) != n) ok = false;
        ++i;
    }
    if (ok) return true;
    std::string want;
    for (int64_t n : shape) want += (want.empty() ? "" : ", ") + (n < 0 ? std::string("*") : std::to_string(n));
    return fail("%s must be a contiguous %s tensor [%s] on %s", name, at::toString(type), want.c_str(),
                device.str().c_str());
}

struct Heads {
    int64_t T, H, D, ts, hs;
};

// [T, heads, D] with contiguous head rows, any token and head strides.
bool heads(const Tensor& t, const char* name, at::ScalarType type, const at::Device& device, int64_t T, int64_t H,
           int64_t D, Heads* out) {
    if (t.dim() != 3 || t.scalar_type() != type || t.device() != device)
        return fail("%s must be a %s tensor [T, heads, D] on %s", name, at::toString(type), device.str().c_str());
    *out = Heads{t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
    if ((T >= 0 && out->T != T) || (H >= 0 && out->H != H) || (D >= 0 && out->D != D))
        return fail("%s has shape [%lld, %lld, %lld], expected [%lld, %lld, %lld] (-1: any)", name, (long long)out->T,
                    (long long)out->H, (long long)out->D, (long long)T, (long long)H, (long long)D);
    if (out->D > 1 && t.stride(2) != 1) return fail("%s must be contiguous along its last dimension", name);
    return true;
}

// The memory of a tensor with these heads, and of a contiguous one.
bsa::Rows rows_of(const Tensor* t, const Heads& h) {
    if (t == nullptr) return bsa::whole_rows(nullptr, 0);
    const int64_t size = (int64_t)t->element_size();
    return bsa::Rows{t->const_data_ptr(), h.T, h.H, h.D * size, h.ts * size, h.hs * size};
}
bsa::Rows rows_of(const Tensor* t) {
    return t == nullptr ? bsa::whole_rows(nullptr, 0) : bsa::whole_rows(t->const_data_ptr(), (int64_t)t->nbytes());
}

struct Rope {
    const int32_t* positions = nullptr;
    const float* inv_freq = nullptr;
    const int32_t* freq_axis = nullptr;
    int32_t axes = 1, rot_dim = 0;
};

bool rope_args(PyObject* positions, PyObject* inv_freq, PyObject* freq_axis, int64_t T, const at::Device& device,
               Rope* r) {
    const Tensor *p, *f, *a;
    if (!tensor(positions, "positions", &p) || !tensor(inv_freq, "inv_freq", &f) || !tensor(freq_axis, "freq_axis", &a))
        return false;
    if (f != nullptr) {
        if (!whole(*f, "inv_freq", at::kFloat, device, {-1})) return false;
        if (f->size(0) > INT32_MAX / 2) return fail("inv_freq is too long");
        r->rot_dim = (int32_t)(2 * f->size(0));
    }
    if (p != nullptr) {
        if (p->dim() == 2) {
            if (!whole(*p, "positions", at::kInt, device, {-1, T})) return false;
            if (p->size(0) > INT32_MAX) return fail("positions has too many axes");
            r->axes = (int32_t)p->size(0);
        } else if (!whole(*p, "positions", at::kInt, device, {T})) {
            return false;
        }
    }
    if (a != nullptr) {
        if (!whole(*a, "freq_axis", at::kInt, device, {r->rot_dim / 2})) return false;
    } else if (r->axes > 1 && r->rot_dim > 0) {
        return fail("freq_axis is needed with several position axes");
    }
    if (f != nullptr) r->inv_freq = f->const_data_ptr<float>();
    if (p != nullptr) r->positions = p->const_data_ptr<int32_t>();
    if (a != nullptr) r->freq_axis = a->const_data_ptr<int32_t>();
    return true;
}

// The caches and their scales: dtype code and page count.
bool caches(PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso, const at::Device& device, int64_t H, int64_t D,
            int32_t* code, int64_t* pages, const Tensor* (&t)[4]) {
    if (!needed(ko, "k_cache", &t[0]) || !needed(vo, "v_cache", &t[1]) || !tensor(kso, "k_scale", &t[2]) ||
        !tensor(vso, "v_scale", &t[3]))
        return false;
    const at::ScalarType type = t[0]->scalar_type();
    if (type == at::kBFloat16) *code = BSA_DTYPE_BF16;
    else if (type == at::kFloat8_e4m3fn) *code = BSA_DTYPE_E4M3;
    else if (type == at::kFloat8_e5m2) *code = BSA_DTYPE_E5M2;
    else return fail("k_cache must be bfloat16, float8_e4m3fn or float8_e5m2");
    if (!whole(*t[0], "k_cache", type, device, {-1, BSA_SUB_PAGE_SIZE, H, D})) return false;
    *pages = t[0]->size(0);
    if (!whole(*t[1], "v_cache", type, device, {*pages, BSA_SUB_PAGE_SIZE, H, D})) return false;
    if (*code == BSA_DTYPE_BF16) {
        if (t[2] != nullptr || t[3] != nullptr) return fail("k_scale and v_scale must be None with a bfloat16 cache");
        return true;
    }
    if (t[2] == nullptr || t[3] == nullptr) return fail("k_scale and v_scale are needed with an 8-bit cache");
    return whole(*t[2], "k_scale", at::kFloat, device, {*pages, H}) &&
           whole(*t[3], "v_scale", at::kFloat, device, {*pages, H});
}

const void* data(const Tensor* t) { return t == nullptr ? nullptr : t->const_data_ptr(); }
void* data_rw(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

// A call has written to the tensor: autograd's version counter moves.
void changed(const Tensor* t) {
    if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

bool on_gpu(const at::Device& device, const char* name) {
    return device.is_cuda() || fail("%s must be on a CUDA device, not %s", name, device.str().c_str());
}

// The current stream of the device as a cudaStream_t.
bool stream_of(const at::Device& device, void** stream) {
    PyObject* index = PyLong_FromLong(device.index());
    if (index == nullptr) return false;
    PyObject* s = PyObject_CallOneArg(g_raw_stream, index);
    Py_DECREF(index);
    if (s == nullptr) return false;
    *stream = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return PyErr_Occurred() == nullptr;
}

bool done(const char* fn, int status) {
    if (status == BSA_OK) return true;
    PyObject* e = PyObject_CallFunction(g_error, "sis", fn, status, bsa_status_string(status));
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return false;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// rope(x, positions, inv_freq, freq_axis, interleaved, inverse, out) -> out
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Tensor *x, *out;
    if (!count(n, 7) || !needed(a[0], "x", &x) || !tensor(a[6], "out", &out)) return nullptr;
    const at::ScalarType type = x->scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return fail("x must be bfloat16 or float32"), nullptr;
    const at::Device device = x->device();
    Heads xh, oh;
    if (!heads(*x, "x", type, device, -1, -1, -1, &xh)) return nullptr;
    if (a[1] == Py_None || a[2] == Py_None) return fail("positions and inv_freq are needed"), nullptr;
    Rope r;
    if (!rope_args(a[1], a[2], a[3], xh.T, device, &r)) return nullptr;
    const int interleaved = PyObject_IsTrue(a[4]), inverse = PyObject_IsTrue(a[5]);
    if (interleaved < 0 || inverse < 0) return nullptr;
    Tensor made;
    if (out != nullptr) {
        if (!heads(*out, "out", type, device, xh.T, xh.H, xh.D, &oh)) return nullptr;
        const bool same = x->const_data_ptr() == out->const_data_ptr() && (xh.T == 1 || xh.ts == oh.ts) && (xh.H == 1 || xh.hs == oh.hs);
        if (!same && bsa::rows_overlap(rows_of(x, xh), rows_of(out, oh)))
            return fail("out must not overlap x, unless it is x"), nullptr;
    }
    if (!on_gpu(device, "x")) return nullptr;
    if (out == nullptr) {
        made = at::empty({xh.T, xh.H, xh.D}, x->options().requires_grad(false));
        out = &made;
        oh = Heads{xh.T, xh.H, xh.D, xh.H * xh.D, xh.D};
    }
    void* stream;
    if (!stream_of(device, &stream)) return nullptr;
    const c10::DeviceGuard guard(device);
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = bsa_rope(data(x), type == at::kBFloat16 ? BSA_DTYPE_BF16 : BSA_DTYPE_FP32, xh.T, xh.H, xh.D, xh.ts, xh.hs,
                      r.positions, r.axes, r.inv_freq, r.freq_axis, r.rot_dim,
                      (interleaved ? BSA_ROPE_INTERLEAVED : 0) | (inverse ? BSA_ROPE_INVERSE : 0), data_rw(out), oh.ts,
                      oh.hs, stream);
    Py_END_ALLOW_THREADS
    if (!done("bsa_rope", status)) return nullptr;
    changed(out);
    return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[6]);
    END_HANDLE_TH_ERRORS
}

// append(k, v, k_cache, v_cache, block_table, rows, more, q, inv_freq, positions, freq_axis,
//        interleaved, k_scale, v_scale, q_out) -> q_out.  Decode: rows is seq_lens, more the query
// length (an integer).  Varlen: rows is prefix_lens, more cu_seqlens_q.
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Tensor *k, *v, *q, *q_out, *table, *rows, *cu = nullptr, *c[4];
    if (!count(n, 15) || !needed(a[0], "k", &k) || !needed(a[1], "v", &v) || !needed(a[4], "block_table", &table))
        return nullptr;
    const bool varlen = THPVariable_Check(a[6]);
    if (!needed(a[5], varlen ? "prefix_lens" : "seq_lens", &rows) || !tensor(a[7], "q", &q) || !tensor(a[14], "q_out", &q_out))
        return nullptr;
    const at::Device device = k->device();
    bsa_append_args_t p{};
    Heads kh, vh, qh{0, 0, 0, 0, 0};
    if (!heads(*k, "k", at::kBFloat16, device, -1, -1, -1, &kh) ||
        !heads(*v, "v", at::kBFloat16, device, kh.T, kh.H, kh.D, &vh))
        return nullptr;
    if (q != nullptr) {
        if (!heads(*q, "q", at::kBFloat16, device, kh.T, -1, kh.D, &qh)) return nullptr;
        if (q_out != nullptr && !whole(*q_out, "q_out", at::kBFloat16, device, {qh.T, qh.H, qh.D})) return nullptr;
    } else if (q_out != nullptr) {
        return fail("q_out without q"), nullptr;
    }
    if (!caches(a[2], a[3], a[12], a[13], device, kh.H, kh.D, &p.cache_dtype, &p.num_pages, c)) return nullptr;
    if (!whole(*rows, varlen ? "prefix_lens" : "seq_lens", at::kInt, device, {-1})) return nullptr;
    p.num_reqs = rows->size(0);
    if (!whole(*table, "block_table", at::kInt, device, {p.num_reqs, -1})) return nullptr;
    p.max_blocks = table->size(1);
    long long dql = 0;
    if (varlen) {
        if (!needed(a[6], "cu_seqlens_q", &cu) || !whole(*cu, "cu_seqlens_q", at::kInt, device, {p.num_reqs + 1}))
            return nullptr;
    } else {
        dql = PyLong_AsLongLong(a[6]);
        if (dql == -1 && PyErr_Occurred()) return nullptr;
        if (dql < INT32_MIN || dql > INT32_MAX) return fail("decode_query_len is out of range"), nullptr;
    }
    Rope r;
    if (!rope_args(a[9], a[8], a[10], kh.T, device, &r)) return nullptr;
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) return nullptr;
    {
        const char* name[8] = {"q_out", "k_cache", "v_cache", "k_scale", "v_scale", "q", "k", "v"};
        const bsa::Rows r[8] = {rows_of(q_out), rows_of(c[0]), rows_of(c[1]), rows_of(c[2]), rows_of(c[3]),
                                rows_of(q, qh), rows_of(k, kh), rows_of(v, vh)};
        for (int i = 0; i < 5; ++i)
            for (int j = i + 1; j < 8; ++j)
                if (bsa::rows_overlap(r[i], r[j])) return fail("%s must not overlap %s", name[i], name[j]), nullptr;
    }
    if (!on_gpu(device, "k")) return nullptr;
    Tensor made;
    if (q != nullptr && q_out == nullptr) {
        made = at::empty({qh.T, qh.H, qh.D}, q->options().requires_grad(false));
        q_out = &made;
    }
    p.k = data(k);
    p.v = data(v);
    p.q = data(q);
    p.T = kh.T;
    p.H = kh.H;
    p.Hq = qh.H;
    p.D = kh.D;
    p.k_token_stride = kh.ts;
    p.k_head_stride = kh.hs;
    p.v_token_stride = vh.ts;
    p.v_head_stride = vh.hs;
    p.q_token_stride = qh.ts;
    p.q_head_stride = qh.hs;
    p.q_out = data_rw(q_out);
    p.positions = r.positions;
    p.inv_freq = r.inv_freq;
    p.freq_axis = r.freq_axis;
    p.axes = r.axes;
    p.rot_dim = r.rot_dim;
    p.flags = interleaved ? BSA_ROPE_INTERLEAVED : 0;
    p.k_cache = data_rw(c[0]);
    p.v_cache = data_rw(c[1]);
    p.k_scale = static_cast<float*>(data_rw(c[2]));
    p.v_scale = static_cast<float*>(data_rw(c[3]));
    p.block_table = static_cast<const int32_t*>(data(table));
    void* stream;
    if (!stream_of(device, &stream)) return nullptr;
    const c10::DeviceGuard guard(device);
    const int32_t* row_ptr = static_cast<const int32_t*>(data(rows));
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = varlen ? bsa_append_kv_varlen(&p, static_cast<const int32_t*>(data(cu)), row_ptr, stream)
                    : bsa_append_kv_decode(&p, row_ptr, (int32_t)dql, stream);
    Py_END_ALLOW_THREADS
    if (!done(varlen ? "bsa_append_kv_varlen" : "bsa_append_kv_decode", status)) return nullptr;
    for (const Tensor* t : c) changed(t);
    changed(q_out);
    return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[14]);
    END_HANDLE_TH_ERRORS
}

// attention_q8(q, k_cache, v_cache, k_scale, v_scale, sparse_bt, sparse_ctx, scale, out, workspace) -> out
PyObject* py_attention_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Tensor *q, *bt, *ctx, *out, *ws, *c[4];
    if (!count(n, 10) || !needed(a[0], "q", &q) || !needed(a[5], "sparse_bt", &bt) || !needed(a[6], "sparse_ctx", &ctx) ||
        !tensor(a[8], "out", &out) || !tensor(a[9], "workspace", &ws))
        return nullptr;
    const at::Device device = q->device();
    if (!whole(*q, "q", at::kBFloat16, device, {-1, -1, -1, -1})) return nullptr;
    const int64_t T = q->size(0), H = q->size(1), G = q->size(2), D = q->size(3);
    int32_t code;
    int64_t pages;
    if (!caches(a[1], a[2], a[3], a[4], device, H, D, &code, &pages, c)) return nullptr;
    if (code == BSA_DTYPE_BF16) return fail("the caches must be float8_e4m3fn or float8_e5m2"), nullptr;
    if (!whole(*bt, "sparse_bt", at::kInt, device, {T, H, -1}) || !whole(*ctx, "sparse_ctx", at::kInt, device, {T, H}))
        return nullptr;
    if (bt->size(2) % BSA_PAGES_PER_SPARSE_BLOCK != 0 || bt->size(2) / BSA_PAGES_PER_SPARSE_BLOCK > INT32_MAX)
        return fail("sparse_bt must be [T, H, K*8]"), nullptr;
    const int32_t K = (int32_t)(bt->size(2) / BSA_PAGES_PER_SPARSE_BLOCK);
    double scale = 0.0;
    if (a[7] != Py_None) {
        scale = PyFloat_AsDouble(a[7]);
        if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    } else {
        scale = 1.0 / std::sqrt((double)D);
    }
    if (out != nullptr) {
        if (!whole(*out, "out", at::kBFloat16, device, {T, H, G, D})) return nullptr;
        const char* name[4] = {"k_cache", "v_cache", "k_scale", "v_scale"};
        for (int i = 0; i < 4; ++i)
            if (bsa::rows_overlap(rows_of(out), rows_of(c[i]))) return fail("out must not overlap %s", name[i]), nullptr;
        if (out->const_data_ptr() != q->const_data_ptr() && bsa::rows_overlap(rows_of(out), rows_of(q)))
            return fail("out must not overlap q, unless it is q"), nullptr;
    }
    if (ws != nullptr && (ws->device() != device || !ws->is_contiguous()))
        return fail("workspace must be a contiguous tensor on %s", device.str().c_str()), nullptr;
    if (!on_gpu(device, "q")) return nullptr;
    const c10::DeviceGuard guard(device);
    Tensor made;
    if (out == nullptr) {
        made = at::empty({T, H, G, D}, q->options().requires_grad(false));
        out = &made;
    }
    PyObject* held = nullptr;      // keeps the package's workspace for the call
    if (ws == nullptr) {
        const size_t need = bsa_attention_q8_workspace_bytes(T, H, G, D, K);
        if (need > 0) {
            PyObject* dev = PyObject_GetAttrString(a[0], "device");
            if (dev == nullptr) return nullptr;
            held = PyObject_CallFunction(g_workspace, "On", dev, (Py_ssize_t)need);
            Py_DECREF(dev);
            if (held == nullptr) return nullptr;
            ws = &THPVariable_Unpack(held);
        }
    }
    void* stream;
    if (!stream_of(device, &stream)) {
        Py_XDECREF(held);
        return nullptr;
    }
    void* ws_ptr = data_rw(ws);
    const size_t ws_bytes = ws == nullptr ? 0 : (size_t)ws->nbytes();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = bsa_sparse_decode_attention_q8(data(q), data(c[0]), data(c[1]), code, static_cast<const float*>(data(c[2])),
                                            static_cast<const float*>(data(c[3])), pages,
                                            static_cast<const int32_t*>(data(bt)), static_cast<const int32_t*>(data(ctx)),
                                            T, H, G, D, K, (float)scale, data_rw(out), ws_ptr, ws_bytes, stream);
    Py_END_ALLOW_THREADS
    Py_XDECREF(held);
    if (!done("bsa_sparse_decode_attention_q8", status)) return nullptr;
    changed(out);
    return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[8]);
    END_HANDLE_TH_ERRORS
}

// setup(BsaError, raw_stream, workspace)
PyObject* py_setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 3)) return nullptr;
    Py_XSETREF(g_error, Py_NewRef(a[0]));
    Py_XSETREF(g_raw_stream, Py_NewRef(a[1]));
    Py_XSETREF(g_workspace, Py_NewRef(a[2]));
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {
    {"rope", FAST(py_rope), nullptr},
    {"append", FAST(py_append), nullptr},
    {"attention_q8", FAST(py_attention_q8), nullptr},
    {"setup", FAST(py_setup), nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "bsa_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_bsa_binding() { return PyModule_Create(&g_module); }
