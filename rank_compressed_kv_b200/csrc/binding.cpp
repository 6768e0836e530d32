// binding.cpp -- argument marshalling of the position and paged-cache calls: torch tensors become
// device pointers and strides, the current torch stream the cudaStream_t.
//
// These calls belong to the step of a few tokens, which takes two to ten microseconds on the GPU.
// The same checks and marshalling written over ctypes cost more than that (rope of 4 rows: 11.2 us
// a call from Python, 2.5 us of them on the GPU), so this part of the binding is native.  Nothing
// is computed or kept here; every check comes before the library's call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <stdexcept>
#include <string>

#include "kvpack.h"

namespace {

struct Refused : std::runtime_error { using std::runtime_error::runtime_error; };   // ValueError
struct BadCall : std::runtime_error { using std::runtime_error::runtime_error; };   // TypeError
struct PyFailed {};                                                                 // the error is set already

// ------------------------------------------------------------------------------- arguments

template <int N>
struct Signature {
    const char *function;
    const char *name[N];
    int required;
    PyObject *key[N];           // interned at import

    void intern() {
        for (int i = 0; i < N; ++i) key[i] = PyUnicode_InternFromString(name[i]);
    }
    void parse(PyObject *const *args, Py_ssize_t nargs, PyObject *kwnames, PyObject *(&out)[N]) const {
        if (nargs > N) throw BadCall(std::string(function) + "() takes at most " + std::to_string(N) + " arguments");
        for (int i = 0; i < N; ++i) out[i] = i < nargs ? args[i] : nullptr;
        const Py_ssize_t nk = kwnames != nullptr ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t k = 0; k < nk; ++k) {
            PyObject *w = PyTuple_GET_ITEM(kwnames, k);
            int at = -1;
            for (int i = 0; i < N && at < 0; ++i)
                if (w == key[i]) at = i;
            for (int i = 0; i < N && at < 0; ++i)
                if (PyUnicode_Compare(w, key[i]) == 0) at = i;
            if (at < 0) throw BadCall(std::string(function) + "() got an unexpected keyword argument");
            if (out[at] != nullptr) throw BadCall(std::string(function) + "() got " + name[at] + " twice");
            out[at] = args[nargs + k];
        }
        for (int i = 0; i < required; ++i)
            if (out[i] == nullptr) throw BadCall(std::string(function) + "() needs " + name[i]);
    }
};

inline bool none(PyObject *o) { return o == nullptr || o == Py_None; }

int64_t integer(PyObject *o, const char *what) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyFailed();
    if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(what) + " is out of range");
    return v;
}

// The C structure of a Rope or PagedDims object, which its attribute _c holds as a ctypes structure of the type that
// structures() was given: copied out, so that nothing here follows an address that an object carries.
PyObject *g_c = nullptr, *g_cuda_stream = nullptr;
PyObject *g_spec_type = nullptr, *g_dims_type = nullptr;

template <typename T>
T structure(PyObject *o, PyObject *type, const char *what) {
    T v;
    PyObject *c = PyObject_GetAttr(o, g_c);
    Py_buffer b;
    bool ok = c != nullptr && type != nullptr && PyObject_TypeCheck(c, reinterpret_cast<PyTypeObject *>(type)) &&
              PyObject_GetBuffer(c, &b, PyBUF_SIMPLE) == 0;
    if (ok) {
        ok = b.len == (Py_ssize_t)sizeof(T);
        if (ok) std::memcpy(&v, b.buf, sizeof(T));
        PyBuffer_Release(&b);
    }
    Py_XDECREF(c);
    if (!ok) {
        PyErr_Clear();
        throw BadCall(what);
    }
    return v;
}

kvpack_rope_spec rope_spec(PyObject *o) { return structure<kvpack_rope_spec>(o, g_spec_type, "spec is not a Rope"); }
kvpack_paged_dims paged_dims(PyObject *o) { return structure<kvpack_paged_dims>(o, g_dims_type, "dims is not a PagedDims"); }

PyObject *set_structures(PyObject *, PyObject *args) {
    PyObject *spec, *dims;
    if (!PyArg_ParseTuple(args, "O!O!", &PyType_Type, &spec, &PyType_Type, &dims)) return nullptr;
    Py_INCREF(spec);
    Py_INCREF(dims);
    Py_XSETREF(g_spec_type, spec);
    Py_XSETREF(g_dims_type, dims);
    Py_RETURN_NONE;
}

// --------------------------------------------------------------------------------- tensors

struct Call {
    static constexpr int kNone = -2;
    int device = kNone;             // of the first tensor; -1 is the CPU
    const char *first = "", *other = nullptr;   // its name, and that of one on another device

    const at::Tensor &tensor(PyObject *o, const char *what) {
        if (o == nullptr || !THPVariable_Check(o)) throw BadCall(std::string(what) + " is not a tensor");
        return THPVariable_Unpack(o);
    }
    // Devices are compared last, in ready(): tensors on the CPU get every other refusal too.
    void seen(const at::Tensor &t, const char *what) {
        const int d = t.is_cuda() ? (int)t.get_device() : -1;
        if (device == kNone) {
            device = d;
            first = what;
        } else if (d != device && other == nullptr) {
            other = what;
        }
    }
    void ready() const {
        const char *bad = device < 0 || device != c10::cuda::current_device() ? first : other;
        if (bad != nullptr) throw Refused(std::string(bad) + " is not on the current CUDA device");
    }
    static std::string shape_of(c10::IntArrayRef s) {
        std::string r = "(";
        for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
        return r + ")";
    }
    static void type(const at::Tensor &t, const char *what, at::ScalarType want) {
        const at::ScalarType have = t.scalar_type();
        if (have != want && !(want == at::kBFloat16 && have == at::kShort))
            throw Refused(std::string(what) + " is " + c10::toString(have) + ", not " + c10::toString(want));
    }
    // The address of a contiguous tensor of this type (bf16: or its bits) and shape, or of this many elements.
    void *dense(PyObject *o, const char *what, at::ScalarType want, c10::IntArrayRef shape, int64_t numel = -1) {
        const at::Tensor &t = tensor(o, what);
        type(t, what, want);
        if (numel >= 0 ? t.numel() != numel : t.sizes() != shape)
            throw Refused(std::string(what) + " has shape " + shape_of(t.sizes()) + ", not " +
                          (numel >= 0 ? std::to_string(numel) + " elements" : shape_of(shape)));
        if (!t.is_contiguous()) throw Refused(std::string(what) + ": kvpack takes contiguous tensors");
        seen(t, what);
        return t.data_ptr();
    }
    // kvpack_heads of a tensor [rows][heads][128], [outer][rows][heads][128] or, in the compression's
    // input layout, [outer][heads / 4][rows][4][128], with any strides that the structure can hold.
    kvpack_heads heads(PyObject *o, const char *what, int64_t outer, int64_t rows, int64_t n) {
        const at::Tensor &t = tensor(o, what);
        type(t, what, at::kBFloat16);
        const auto s = t.sizes(), st = t.strides();
        kvpack_heads h{nullptr, 0, 0, 512};
        int64_t sh = 0, s1 = 0;
        const size_t nd = s.size();
        if (nd == 4 && s[0] == outer && s[1] == rows && s[2] == n && s[3] == 128) {
            h.outer_stride = st[0]; h.row_stride = st[1]; sh = st[2]; s1 = st[3];
        } else if (nd == 3 && outer == 1 && s[0] == rows && s[1] == n && s[2] == 128) {
            h.row_stride = st[0]; sh = st[1]; s1 = st[2];
        } else if (nd == 5 && n % 4 == 0 && s[0] == outer && s[1] == n / 4 && s[2] == rows && s[3] == 4 && s[4] == 128) {
            h.outer_stride = st[0]; h.group_stride = st[1]; h.row_stride = st[2]; sh = st[3]; s1 = st[4];
        } else {
            throw Refused(std::string(what) + " has shape " + shape_of(s) + ": " + std::to_string(outer) + " x " +
                          std::to_string(rows) + " rows of " + std::to_string(n) + " heads of 128 are wanted");
        }
        if (s1 != 1 || (sh != 128 && n > 1))
            throw Refused(std::string(what) + ": a head's entries and the heads of a row (of four) lie side by side");
        // strides of dimensions of one are as good as any
        if (outer == 1) h.outer_stride = 0;
        if (rows == 1) h.row_stride = 0;
        if (n <= 4) h.group_stride = 512;
        seen(t, what);
        h.data = static_cast<uint16_t *>(t.data_ptr());
        return h;
    }
    static int64_t count_heads(const at::Tensor &t, const char *what) {
        if (t.dim() == 5) return t.size(1) * t.size(3);
        if (t.dim() == 3 || t.dim() == 4) return t.size(-2);
        throw Refused(std::string(what) + " has shape " + shape_of(t.sizes()) + ": rows of heads of 128 are wanted");
    }
    void *stream(PyObject *o) {
        if (none(o)) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        if (PyLong_Check(o)) {
            void *p = PyLong_AsVoidPtr(o);
            if (p == nullptr && PyErr_Occurred()) throw PyFailed();
            return p;
        }
        PyObject *a = PyObject_GetAttr(o, g_cuda_stream);
        if (a == nullptr) throw PyFailed();
        void *p = PyLong_AsVoidPtr(a);
        Py_DECREF(a);
        if (p == nullptr && PyErr_Occurred()) throw PyFailed();
        return p;
    }
};

// KvpackError of a status, as the rest of the binding raises it
PyObject *finish(int status, const char *what) {
    if (status == KVPACK_OK) Py_RETURN_NONE;
    PyObject *m = PyImport_ImportModule("rank_compressed_kv_b200._lib");
    if (m == nullptr) return nullptr;
    PyObject *r = PyObject_CallMethod(m, "_check", "is", status, what);
    Py_DECREF(m);
    return r;
}

template <typename F>
PyObject *guarded(F &&f) {
    try {
        return f();
    } catch (const PyFailed &) {
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const BadCall &e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// ----------------------------------------------------------------------------------- calls

Signature<9> rope_sig{"rope", {"spec", "freq", "pos", "q", "q_out", "k", "k_out", "inverse", "stream"}, 5, {}};

const char *rope_doc =
    "rope(spec, freq, pos, q, q_out, k=None, k_out=None, inverse=False, stream=None)\n--\n\n"
    "Rotate q into q_out and k into k_out (either pair may be None; an output may be its input).\n\n"
    "Rows are [batch][T][heads][128], [T][heads][128], or [batch][heads / 4][T][4][128] (what compress\n"
    "takes); pos is int32 [n_axes][batch][T] ([n_axes][T] for one batch row); freq float64 [rotary_dim / 2]\n"
    "(spec.frequencies).  inverse turns back: the gradient with respect to the input is\n"
    "rope(..., grad, grad_in, inverse=True).";

PyObject *call_rope(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        PyObject *a[9];
        rope_sig.parse(args, nargs, kw, a);
        const kvpack_rope_spec spec = rope_spec(a[0]);
        const bool has_q = !none(a[3]), has_k = !none(a[5]);
        if (has_q != !none(a[4]) || has_k != !none(a[6]) || (!has_q && !has_k))
            throw Refused("an input and its output, of q, of k or of both");
        Call c;
        const at::Tensor &pos = c.tensor(a[2], "pos");
        const auto ps = pos.sizes();
        if ((ps.size() != 2 && ps.size() != 3) || ps[0] != spec.n_axes)
            throw Refused("pos has shape " + Call::shape_of(ps) + ": [" + std::to_string(spec.n_axes) +
                          "][batch][T] is wanted");
        const int64_t outer = ps.size() == 3 ? ps[1] : 1, rows = ps.back();
        const void *pp = c.dense(a[2], "pos", at::kInt, ps);
        const void *fp = c.dense(a[1], "freq", at::kDouble, {spec.rotary_dim / 2});
        kvpack_heads q{}, qo{}, k{}, ko{};
        int64_t n_q = 0, n_k = 0;
        if (has_q) {
            n_q = Call::count_heads(c.tensor(a[3], "q"), "q");
            q = c.heads(a[3], "q", outer, rows, n_q);
            qo = c.heads(a[4], "q_out", outer, rows, n_q);
        }
        if (has_k) {
            n_k = Call::count_heads(c.tensor(a[5], "k"), "k");
            k = c.heads(a[5], "k", outer, rows, n_k);
            ko = c.heads(a[6], "k_out", outer, rows, n_k);
        }
        const int inverse = none(a[7]) ? 0 : PyObject_IsTrue(a[7]);
        if (inverse < 0) throw PyFailed();
        if (outer > INT32_MAX || rows > INT32_MAX) throw Refused("too many rows");
        c.ready();
        if (outer == 0 || rows == 0) Py_RETURN_NONE;
        void *st = c.stream(a[8]);
        int s;
        Py_BEGIN_ALLOW_THREADS
        s = kvpack_rope(&spec, static_cast<const double *>(fp), static_cast<const int32_t *>(pp), (int32_t)outer,
                        (int32_t)rows, (int32_t)n_q, &q, &qo, (int32_t)n_k, &k, &ko, inverse, st);
        Py_END_ALLOW_THREADS
        return finish(s, "kvpack_rope");
    });
}

struct Pool {
    uint16_t *K, *V;
    const int32_t *table, *lens;
};

Pool pool(Call &c, const kvpack_paged_dims *d, int64_t layers, PyObject *K, PyObject *V, PyObject *table, PyObject *lens) {
    int64_t n = layers;
    for (int64_t f : {d->n_pages, d->n_kv_heads, d->page_size, d->head_dim})
        if (__builtin_mul_overflow(n, f, &n)) n = INT64_MAX;             // more than any tensor has
    Pool p;
    p.K = static_cast<uint16_t *>(c.dense(K, "K_pages", at::kBFloat16, {}, n));
    p.V = static_cast<uint16_t *>(c.dense(V, "V_pages", at::kBFloat16, {}, n));
    p.table = static_cast<const int32_t *>(c.dense(table, "block_table", at::kInt, {d->batch, d->max_pages}));
    p.lens = static_cast<const int32_t *>(c.dense(lens, "seq_lens", at::kInt, {d->batch}));
    return p;
}

Signature<15> append_sig{"paged_append",
                         {"dims", "n_layers", "spec", "freq", "pos", "q", "k", "v", "row_offsets", "seq_lens",
                          "block_table", "q_out", "K_pages", "V_pages", "stream"}, 14, {}};

const char *append_doc =
    "paged_append(dims, n_layers, spec, freq, pos, q, k, v, row_offsets, seq_lens, block_table, q_out, K_pages,\n"
    "             V_pages, stream=None)\n--\n\n"
    "New tokens into their pages: k rotated, v as it is; q rotated into q_out (both may be None).\n\n"
    "q, k, v: [rows][heads][128] (n_layers 1) or [n_layers][rows][heads][128]; row_offsets int32 [batch + 1], or\n"
    "None for one row per sequence; seq_lens with the new tokens counted; spec None: no rotation.";

PyObject *call_append(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        PyObject *a[15];
        append_sig.parse(args, nargs, kw, a);
        const kvpack_paged_dims dims = paged_dims(a[0]), *d = &dims;
        const int64_t layers = integer(a[1], "n_layers");
        Call c;
        const at::Tensor &kt = c.tensor(a[6], "k");
        if (kt.dim() < 3) throw Refused("k has shape " + Call::shape_of(kt.sizes()) + ": rows of heads of 128 are wanted");
        const int64_t rows = kt.size(-3);
        if (none(a[8]) && rows != d->batch) throw Refused("without row_offsets there is one row per sequence");
        if (none(a[5]) != none(a[11])) throw Refused("q and q_out, or neither");
        const kvpack_heads k = c.heads(a[6], "k", layers, rows, d->n_kv_heads);
        const kvpack_heads v = c.heads(a[7], "v", layers, rows, d->n_kv_heads);
        kvpack_heads q{}, qo{};
        const bool has_q = !none(a[5]);
        if (has_q) {
            q = c.heads(a[5], "q", layers, rows, d->n_q_heads);
            qo = c.heads(a[11], "q_out", layers, rows, d->n_q_heads);
        }
        const Pool p = pool(c, d, layers, a[12], a[13], a[10], a[9]);
        const void *off = none(a[8]) ? nullptr : c.dense(a[8], "row_offsets", at::kInt, {d->batch + 1});
        kvpack_rope_spec rotation, *spec = nullptr;
        const void *fp = nullptr, *pp = nullptr;
        if (!none(a[2])) {
            rotation = rope_spec(a[2]);
            spec = &rotation;
            fp = c.dense(a[3], "freq", at::kDouble, {spec->rotary_dim / 2});
            pp = c.dense(a[4], "pos", at::kInt, {spec->n_axes, rows});
        }
        if (rows > INT32_MAX) throw Refused("too many rows");
        c.ready();
        if (rows == 0) Py_RETURN_NONE;
        void *st = c.stream(a[14]);
        int s;
        Py_BEGIN_ALLOW_THREADS
        s = kvpack_paged_append(d, (int32_t)layers, spec, static_cast<const double *>(fp),
                                static_cast<const int32_t *>(pp), (int32_t)rows, has_q ? &q : nullptr, &k, &v,
                                static_cast<const int32_t *>(off), p.lens, p.table, has_q ? &qo : nullptr, p.K, p.V, st);
        Py_END_ALLOW_THREADS
        return finish(s, "kvpack_paged_append");
    });
}

Signature<12> attend_sig{"paged_decode_attn",
                         {"dims", "n_layers", "q", "K_pages", "V_pages", "block_table", "seq_lens", "scale", "out",
                          "lse", "ws", "stream"}, 11, {}};

const char *attend_doc =
    "paged_decode_attn(dims, n_layers, q, K_pages, V_pages, block_table, seq_lens, scale, out, lse, ws, stream=None)\n"
    "--\n\n"
    "One query per sequence over its pages: out [n_layers * batch][n_q][128] bf16, lse [..][n_q] fp32 or None.";

PyObject *call_attend(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        PyObject *a[12];
        attend_sig.parse(args, nargs, kw, a);
        const kvpack_paged_dims dims = paged_dims(a[0]), *d = &dims;
        const int64_t layers = integer(a[1], "n_layers"), rows = layers * d->batch;
        const double scale = PyFloat_AsDouble(a[7]);
        if (scale == -1.0 && PyErr_Occurred()) throw PyFailed();
        Call c;
        const void *q = c.dense(a[2], "q", at::kBFloat16, {rows, d->n_q_heads, 128});
        void *out = c.dense(a[8], "out", at::kBFloat16, {rows, d->n_q_heads, 128});
        void *lse = none(a[9]) ? nullptr : c.dense(a[9], "lse", at::kFloat, {rows, d->n_q_heads});
        const Pool p = pool(c, d, layers, a[3], a[4], a[5], a[6]);
        const at::Tensor &wt = c.tensor(a[10], "ws");
        void *ws = c.dense(a[10], "ws", at::kByte, wt.sizes());
        const size_t ws_bytes = (size_t)wt.numel();
        c.ready();
        void *st = c.stream(a[11]);
        int s;
        Py_BEGIN_ALLOW_THREADS
        s = kvpack_paged_decode_attn(d, (int32_t)layers, static_cast<const uint16_t *>(q), p.K, p.V, p.table, p.lens,
                                     (float)scale, static_cast<uint16_t *>(out), static_cast<float *>(lse), ws, ws_bytes,
                                     st);
        Py_END_ALLOW_THREADS
        return finish(s, "kvpack_paged_decode_attn");
    });
}

PyMethodDef methods[] = {
    {"structures", set_structures, METH_VARARGS,
     "structures(spec_type, dims_type)\n--\n\nThe ctypes structures that Rope and PagedDims objects hold as _c."},
    {"rope", (PyCFunction)(void (*)(void))call_rope, METH_FASTCALL | METH_KEYWORDS, rope_doc},
    {"paged_append", (PyCFunction)(void (*)(void))call_append, METH_FASTCALL | METH_KEYWORDS, append_doc},
    {"paged_decode_attn", (PyCFunction)(void (*)(void))call_attend, METH_FASTCALL | METH_KEYWORDS, attend_doc},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", "Native argument marshalling of libkvpack's per-step calls.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

// The extension reads torch's and Python's own structures: one that was built for others is refused, not tried.
bool built_for_these() {
    const std::string python = std::to_string(PY_MAJOR_VERSION) + "." + std::to_string(PY_MINOR_VERSION) + ".";
    const std::string have = Py_GetVersion();
    if (have.compare(0, python.size(), python) != 0) {
        PyErr_Format(PyExc_ImportError, "_call.so was built for Python %sx, this is %s; run rank_compressed_kv_b200/build.py",
                     python.c_str(), have.c_str());
        return false;
    }
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *version = torch != nullptr ? PyObject_GetAttrString(torch, "__version__") : nullptr;
    Py_XDECREF(torch);
    const char *is = version != nullptr ? PyUnicode_AsUTF8(version) : nullptr;
    const bool same = is != nullptr && std::strcmp(is, KVPACK_TORCH) == 0;
    if (is != nullptr && !same)
        PyErr_Format(PyExc_ImportError, "_call.so was built for torch %s, this is %s; run rank_compressed_kv_b200/build.py",
                     KVPACK_TORCH, is);
    Py_XDECREF(version);
    return same;
}

}  // namespace

PyMODINIT_FUNC PyInit__call(void) {
    if (!built_for_these()) return nullptr;
    g_c = PyUnicode_InternFromString("_c");
    g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    rope_sig.intern();
    append_sig.intern();
    attend_sig.intern();
    return PyModule_Create(&module);
}
