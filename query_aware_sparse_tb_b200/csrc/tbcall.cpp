// _tbcall: argument marshalling of the calls that take several new tokens per
// sequence, for Python.
//
// These calls run once per layer of a step that may take a few microseconds
// altogether, and a call has up to eight tensors to check (type, shape, device,
// contiguity).  Done in Python with ctypes that took 7 to 10 us of host time a
// call; here the tensors are looked at through torch's C++ side.  The functions
// behind it are the C entry points of libtb.so: their addresses come from the
// library that the ctypes binding has loaded (bind), so both go to the same
// one.  A wrong argument raises the binding's TbError; a status other than
// TB_OK is returned for the binding to report.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "../../include/tb.h"

namespace {

decltype(&tb_norm_rope_append) g_rope = nullptr;
decltype(&tb_prompt_attn) g_prompt = nullptr;
decltype(&tb_tree_attn) g_tree = nullptr;
decltype(&tb_tree_accept) g_accept = nullptr;
PyObject *g_error = nullptr;  // TbError(status, message)

// Thrown on a wrong argument; `set` says that the Python error is set already.
struct Bad {
    bool set = false;
    std::string what;
};
[[noreturn]] void bad(const std::string &what) { throw Bad{false, what}; }

std::string text(c10::IntArrayRef shape) {
    std::ostringstream s;
    s << "(";
    for (size_t i = 0; i < shape.size(); ++i) s << (i ? ", " : "") << shape[i];
    s << ")";
    return s.str();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) bad(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}

// Address of a contiguous tensor of that type and shape on device `dev`.
void *address(PyObject *o, const char *name, c10::ScalarType type, c10::IntArrayRef shape, int dev) {
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda()) bad(std::string(name) + ": libtb takes device tensors");
    if (t.scalar_type() != type)
        bad(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(type));
    if (t.sizes() != shape) bad(std::string(name) + ": shape " + text(t.sizes()) + ", expected " + text(shape));
    if (t.get_device() != dev)
        bad(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", the workspace on cuda:" +
            std::to_string(dev));
    if (!t.is_contiguous()) bad(std::string(name) + ": libtb takes contiguous tensors");
    return t.data_ptr();
}

int64_t integer(PyObject *o, const char *name, int64_t lo = INT32_MIN, int64_t hi = INT32_MAX) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad{true, ""};
    if (v < lo || v > hi) bad(std::string(name) + " = " + std::to_string(v) + " is out of range");
    return v;
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad{true, ""};
    return (float)v;
}

// The dims, the workspace and its device; the device is current while this lives.
struct Call {
    tb_dims dims;
    void *ws;
    size_t ws_bytes;
    int dev;
    c10::cuda::OptionalCUDAGuard guard;
    Call(PyObject *d, PyObject *w) {
        Py_buffer b;
        if (PyObject_GetBuffer(d, &b, PyBUF_SIMPLE) != 0) throw Bad{true, ""};
        const bool fits = b.len == (Py_ssize_t)sizeof(tb_dims);
        if (fits) memcpy(&dims, b.buf, sizeof dims);
        PyBuffer_Release(&b);
        if (!fits) bad("d: expected TbDims");
        const at::Tensor &t = tensor(w, "ws");
        if (!t.is_cuda()) bad("ws: libtb takes device tensors");
        if (!t.is_contiguous()) bad("ws: libtb takes contiguous tensors");
        ws = t.data_ptr();
        ws_bytes = t.nbytes();
        dev = t.get_device();
        guard.set_index(dev);
    }
    void *stream(PyObject *s) const {
        if (s == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
        PyObject *v = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttrString(s, "cuda_stream");
        if (!v) throw Bad{true, ""};
        void *p = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (!p && PyErr_Occurred()) throw Bad{true, ""};
        return p;
    }
    const int32_t *lengths(PyObject *o, const char *name, int extra = 0) const {
        const int64_t shape[1] = {(int64_t)dims.batch + extra};
        return static_cast<int32_t *>(address(o, name, c10::kInt, shape, dev));
    }
    tb_bf16 *cache(PyObject *o, const char *name) const {
        const int64_t shape[4] = {dims.batch, dims.n_kv_heads, dims.ctx_cap, dims.head_dim};
        return static_cast<tb_bf16 *>(address(o, name, c10::kBFloat16, shape, dev));
    }
    tb_bf16 *rows(PyObject *o, const char *name, int64_t n) const {
        const int64_t shape[3] = {n, dims.n_q_heads, dims.head_dim};
        return static_cast<tb_bf16 *>(address(o, name, c10::kBFloat16, shape, dev));
    }
    tb_bf16 *weight(PyObject *o, const char *name) const {
        if (o == Py_None) return nullptr;
        const int64_t shape[1] = {dims.head_dim};
        return static_cast<tb_bf16 *>(address(o, name, c10::kBFloat16, shape, dev));
    }
};

int64_t tokens(PyObject *Q) {
    const at::Tensor &t = tensor(Q, "Q");
    if (t.dim() != 3) bad("Q: expected [n_tokens][Hq][d]");
    if (t.size(0) > INT32_MAX) bad("Q: too many tokens");
    return t.size(0);
}

// (d, qkv, q_begin, ctx_len, pos, q_weight, k_weight, eps, inv_freq, interleaved, Q, K, V, ws, stream)
int rope(PyObject *const *a) {
    Call c(a[0], a[13]);
    const int64_t n = tokens(a[10]), width = ((int64_t)c.dims.n_q_heads + 2 * (int64_t)c.dims.n_kv_heads) * c.dims.head_dim;
    const at::Tensor &qkv = tensor(a[1], "qkv");
    if (!qkv.is_cuda()) bad("qkv: libtb takes device tensors");
    if (qkv.get_device() != c.dev || qkv.scalar_type() != c10::kBFloat16 || qkv.dim() != 2 || qkv.size(0) != n ||
        qkv.size(1) != width || (width > 1 && qkv.stride(1) != 1))
        bad("qkv: expected bfloat16 (" + std::to_string(n) + ", " + std::to_string(width) + ") on cuda:" +
            std::to_string(c.dev) + " with contiguous rows");
    const int64_t one[1] = {n};
    const int32_t *pos = a[4] == Py_None ? nullptr : static_cast<int32_t *>(address(a[4], "pos", c10::kInt, one, c.dev));
    const double *inv = nullptr;
    int64_t freqs[1] = {0};
    if (a[8] != Py_None) {
        freqs[0] = tensor(a[8], "inv_freq").numel();
        inv = static_cast<double *>(address(a[8], "inv_freq", c10::kDouble, freqs, c.dev));
        if (freqs[0] > INT32_MAX / 2) bad("inv_freq: too long");
    }
    const int inter = PyObject_IsTrue(a[9]);
    if (inter < 0) throw Bad{true, ""};
    // (of one token the stride means nothing: it may be any number)
    return g_rope(&c.dims, static_cast<tb_bf16 *>(qkv.data_ptr()), n > 1 ? qkv.stride(0) : width,
                  c.lengths(a[2], "q_begin", 1), (int32_t)n, c.lengths(a[3], "ctx_len"), pos, c.weight(a[5], "q_weight"),
                  c.weight(a[6], "k_weight"), real(a[7]), inv, (int32_t)(2 * freqs[0]),
                  inter ? TB_ROPE_INTERLEAVED : TB_ROPE_HALF, c.rows(a[10], "Q", n), c.cache(a[11], "K"),
                  c.cache(a[12], "V"), c.ws, c.ws_bytes, c.stream(a[14]));
}

// (d, Q, K, V, q_begin, max_new, ctx_len, scale, out, ws, stream)
int prompt(PyObject *const *a) {
    Call c(a[0], a[9]);
    const int64_t n = tokens(a[1]);
    return g_prompt(&c.dims, c.rows(a[1], "Q", n), c.cache(a[2], "K"), c.cache(a[3], "V"), c.lengths(a[4], "q_begin", 1),
                    (int32_t)n, (int32_t)integer(a[5], "max_new"), c.lengths(a[6], "ctx_len"), real(a[7]),
                    c.rows(a[8], "out", n), c.ws, c.ws_bytes, c.stream(a[10]));
}

// (d, Q, K, V, q_begin, max_new, ctx_len, mask, scale, out, ws, stream)
int tree(PyObject *const *a) {
    Call c(a[0], a[10]);
    const int64_t n = tokens(a[1]), max_new = integer(a[5], "max_new");
    const int64_t words[2] = {n, (max_new + 31) / 32};
    const bool is_unsigned = tensor(a[7], "mask").scalar_type() == c10::kUInt32;
    const void *mask = address(a[7], "mask", is_unsigned ? c10::kUInt32 : c10::kInt, words, c.dev);
    return g_tree(&c.dims, c.rows(a[1], "Q", n), c.cache(a[2], "K"), c.cache(a[3], "V"), c.lengths(a[4], "q_begin", 1),
                  (int32_t)n, (int32_t)max_new, c.lengths(a[6], "ctx_len"), static_cast<const uint32_t *>(mask), real(a[8]),
                  c.rows(a[9], "out", n), c.ws, c.ws_bytes, c.stream(a[11]));
}

// (d, n_layers, caches, q_begin, ctx_len, path, path_len, new_len, ws, stream)
int accept(PyObject *const *a) {
    Call c(a[0], a[8]);
    const int64_t layers = integer(a[1], "n_layers"), addresses[1] = {2 * layers};
    const at::Tensor &path = tensor(a[5], "path");
    if (path.dim() != 2 || path.size(1) > INT32_MAX) bad("path: expected [batch][path_cap]");
    const int64_t shape[2] = {c.dims.batch, path.size(1)};
    return g_accept(&c.dims, (int32_t)layers,
                    static_cast<uint64_t *>(address(a[2], "caches", c10::kLong, addresses, c.dev)),
                    c.lengths(a[3], "q_begin", 1), c.lengths(a[4], "ctx_len"),
                    static_cast<int32_t *>(address(a[5], "path", c10::kInt, shape, c.dev)), (int32_t)path.size(1),
                    c.lengths(a[6], "path_len"), const_cast<int32_t *>(c.lengths(a[7], "new_len")), c.ws, c.ws_bytes,
                    c.stream(a[9]));
}

PyObject *raise(const Bad &b) {
    if (b.set) return nullptr;
    PyObject *e = PyObject_CallFunction(g_error, "is", (int)TB_ERR_INVALID_ARG, b.what.c_str());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

template <int (*F)(PyObject *const *), int N>
PyObject *wrap(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (!g_error) {
        PyErr_SetString(PyExc_RuntimeError, "_tbcall.bind has not been called");
        return nullptr;
    }
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const Bad &b) {
        return raise(b);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// bind(TbError, addresses of tb_norm_rope_append, tb_prompt_attn, tb_tree_attn, tb_tree_accept)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes the error class and four addresses");
        return nullptr;
    }
    void *f[4];
    for (int i = 0; i < 4; ++i) {
        f[i] = PyLong_AsVoidPtr(args[i + 1]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    g_rope = reinterpret_cast<decltype(g_rope)>(f[0]);
    g_prompt = reinterpret_cast<decltype(g_prompt)>(f[1]);
    g_tree = reinterpret_cast<decltype(g_tree)>(f[2]);
    g_accept = reinterpret_cast<decltype(g_accept)>(f[3]);
    Py_XDECREF(g_error);
    g_error = Py_NewRef(args[0]);
    Py_RETURN_NONE;
}

#define TB_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"bind", TB_FAST(bind), "bind(TbError, addresses)"},
    {"norm_rope_append", TB_FAST((wrap<rope, 15>)), nullptr},
    {"prompt_attn", TB_FAST((wrap<prompt, 11>)), nullptr},
    {"tree_attn", TB_FAST((wrap<tree, 12>)), nullptr},
    {"tree_accept", TB_FAST((wrap<accept, 10>)), nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tbcall", "marshalling of the multi-token calls", -1, methods};

}  // namespace

// built_for: the torch and the Python this was compiled against, which the
// binding compares with those it runs on.
PyMODINIT_FUNC PyInit__tbcall() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", TB_BUILT_FOR) != 0) {
        Py_DECREF(m);
        m = nullptr;
    }
    return m;
}
