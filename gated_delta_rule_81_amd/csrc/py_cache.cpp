// py_cache.cpp -- the Python front end's common case of the operators on a paged
// cache (include/kda_cache.h), as a CPython module: a decoding step of a few
// sessions is shorter than the checks of its tensors in Python.
//
// Each function takes the tensors of a call whose arguments are as the front
// end documents them, forms the output and the workspace, and calls the library.
// Whatever is not of that kind (another device, type, shape or order in memory, a
// given output) makes it return None before anything has been done: cache.py then
// goes through its own checks, which say in words what is wrong.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdint.h>

namespace {

constexpr int32_t kF32 = 0, kBf16 = 1;  // enum kda_dtype

// The library's entry points, found by cache.py.  (A stream is a pointer here.)
typedef int (*AppendFn)(const void *, const void *, const void *, const float *, const int32_t *,
                        const int32_t *, const int32_t *, const int32_t *, void *, void *, void *,
                        int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t,
                        int32_t, int32_t, int32_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                        int64_t, int64_t, int32_t, int32_t, void *);
typedef int (*AttnFn)(const void *, const void *, const void *, const int32_t *, const int32_t *,
                      const int32_t *, const int32_t *, const int32_t *, void *, float *, int32_t,
                      int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t,
                      int64_t, int64_t, int64_t, int64_t, int64_t, float, int32_t, void *, int64_t,
                      void *);
typedef int64_t (*WorkspaceFn)(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t,
                               int32_t, int32_t);
AppendFn append_fn;
AttnFn attn_fn;
WorkspaceFn workspace_fn;

struct Irregular {};  // not the common case

const at::Tensor *tensor(PyObject *o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Irregular{};
    return &THPVariable_Unpack(o);
}

void must(bool ok) {
    if (!ok) throw Irregular{};
}

int32_t size32(int64_t n) {
    must(n >= 0 && n <= INT32_MAX);
    return (int32_t)n;
}

// Other Python threads run while this lives: the allocations and the launches, and in debug mode the
// wait for the stream, touch no Python object.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// What every tensor of a call shares.
struct Kind {
    c10::Device device;
    at::ScalarType type;
    int32_t code;
    explicit Kind(const at::Tensor &t) : device(t.device()), type(t.scalar_type()), code(0) {
        must(device.is_cuda() && (type == at::kFloat || type == at::kBFloat16));
        code = type == at::kBFloat16 ? kBf16 : kF32;
    }
};

// [T, H, d] with the values of a token dense; returns the distance between tokens.
int64_t rows(const at::Tensor *t, const Kind &k, int64_t T, int64_t H, int64_t d) {
    must(t && t->device() == k.device && t->scalar_type() == k.type && t->dim() == 3);
    const auto n = t->sizes(), s = t->strides();
    must(n[0] == T && n[1] == H && n[2] == d && T > 0 && H > 0 && d > 1);
    must(s[2] == 1 && (H == 1 || s[1] == d) && (T == 1 || s[0] >= H * d));
    size32(t->numel());
    return T == 1 ? H * d : s[0];
}

// A dense tensor of 32-bit values.
void *dense(const at::Tensor *t, const Kind &k, at::ScalarType type, at::IntArrayRef shape) {
    if (!t) return nullptr;
    must(t->device() == k.device && t->scalar_type() == type && t->sizes() == shape &&
         t->is_contiguous());
    return t->data_ptr();
}

struct Cache {
    int32_t pages, size;
    int64_t page, token, head;
};
Cache cache(const at::Tensor *k, const at::Tensor *v, const Kind &kind, int64_t H, int64_t d) {
    must(k && k->device() == kind.device && k->scalar_type() == kind.type && k->dim() == 4);
    const auto n = k->sizes(), s = k->strides();
    must(n[0] > 0 && n[1] > 0 && n[2] == H && n[3] == d && s[3] == 1);
    if (v)
        must(v->device() == kind.device && v->scalar_type() == kind.type && v->sizes() == n &&
             v->strides() == s);
    return {size32(n[0]), size32(n[1]), n[0] > 1 ? s[0] : 0, n[1] > 1 ? s[1] : 0, H > 1 ? s[2] : 0};
}

struct Sessions {
    int32_t n, width;
    const int32_t *table, *lens, *cu;
};
Sessions sessions(const at::Tensor *table, const at::Tensor *lens, const at::Tensor *cu, const Kind &k,
                  int64_t T) {
    must(table && lens && table->dim() == 2);
    const int64_t n = table->size(0);
    must(n > 0 && (cu || T % n == 0));
    return {size32(n), size32(table->size(1)),
            static_cast<const int32_t *>(dense(table, k, at::kInt, table->sizes())),
            static_cast<const int32_t *>(dense(lens, k, at::kInt, {n})),
            static_cast<const int32_t *>(dense(cu, k, at::kInt, {n + 1}))};
}

void *pointer(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

PyObject *result(int status, const at::Tensor &a, const at::Tensor *b) {
    PyObject *x = a.defined() ? THPVariable_Wrap(a) : Py_NewRef(Py_None);
    PyObject *y = b && b->defined() ? THPVariable_Wrap(*b) : Py_NewRef(Py_None);
    if (!x || !y) {
        Py_XDECREF(x), Py_XDECREF(y);
        return nullptr;
    }
    return Py_BuildValue("(iNN)", status, x, y);
}

// append(stream, k, v, k_cache, v_cache, page_table, lens, cu_seqlens, q, table, positions,
//        rotary_offset, interleaved) -> (status, rotated q, None), or None
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        must(n == 13 && append_fn);
        const at::Tensor *k = tensor(a[1]), *v = tensor(a[2]), *kc = tensor(a[3]), *vc = tensor(a[4]);
        const at::Tensor *q = tensor(a[8]), *table = tensor(a[9]), *positions = tensor(a[10]);
        must(k && k->dim() == 3 && !v == !vc && !table == !positions);
        const Kind kind(*k);
        const int64_t T = k->size(0), H = k->size(1), d = k->size(2);
        const int64_t ks = rows(k, kind, T, H, d), vs = v ? rows(v, kind, T, H, d) : 0;
        const Cache c = cache(kc, vc, kind, H, d);
        const Sessions s = sessions(tensor(a[5]), tensor(a[6]), tensor(a[7]), kind, T);
        int64_t hq = 0, qs = 0, table_rows = 0, rot = 0;
        if (q) {
            must(q->dim() == 3);
            hq = q->size(1);
            qs = rows(q, kind, T, hq, d);
        }
        if (table) {
            must(table->dim() == 2);
            table_rows = table->size(0), rot = table->size(1);
            dense(table, kind, at::kFloat, table->sizes());
            dense(positions, kind, at::kInt, {T});
        }
        must(PyLong_Check(a[11]));
        const long at_channel = PyLong_AsLong(a[11]);
        must(at_channel >= 0 && at_channel <= INT32_MAX);
        const int interleaved = PyObject_IsTrue(a[12]);
        must(interleaved >= 0);
        void *stream = PyLong_AsVoidPtr(a[0]);
        must(!PyErr_Occurred());
        at::Tensor out;
        int status;
        {
            const Unlocked unlocked;
            if (q) out = at::empty({T, hq, d}, k->options());
            status = append_fn(
                pointer(q), pointer(k), pointer(v), static_cast<const float *>(pointer(table)),
                static_cast<const int32_t *>(pointer(positions)), s.table, s.lens, s.cu,
                q ? out.data_ptr() : nullptr, pointer(kc), pointer(vc), size32(T), s.n, size32(hq),
                size32(H), size32(d), size32(rot), (int32_t)at_channel, size32(table_rows), c.pages,
                c.size, s.width, qs, ks, vs, q ? hq * d : 0, c.page, c.token, c.head, interleaved,
                kind.code, stream);
        }
        return result(status, out, nullptr);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// attention(stream, q, k_cache, v_cache, page_table, lens, prefix_pages, prefix_len, cu_seqlens,
//           scale, v_dim, output_lse) -> (status, out, lse or None), or None
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        must(n == 12 && attn_fn && workspace_fn);
        const at::Tensor *q = tensor(a[1]), *kc = tensor(a[2]), *vc = tensor(a[3]);
        const at::Tensor *pages = tensor(a[6]), *length = tensor(a[7]);
        must(q && kc && q->dim() == 3 && kc->dim() == 4 && !pages == !length);
        const Kind kind(*q);
        const int64_t T = q->size(0), hq = q->size(1), d = q->size(2), H = kc->size(2);
        const int64_t qs = rows(q, kind, T, hq, d);
        must(H > 0 && hq % H == 0);
        const Cache c = cache(kc, vc, kind, H, d);
        const Sessions s = sessions(tensor(a[4]), tensor(a[5]), tensor(a[8]), kind, T);
        int64_t P = 0;
        if (pages) {
            must(pages->dim() == 1);
            P = pages->size(0);
            dense(pages, kind, at::kInt, {P});
            dense(length, kind, at::kInt, {1});
        }
        const double scale = PyFloat_AsDouble(a[9]);
        const long dv = PyLong_AsLong(a[10]);
        const int want = PyObject_IsTrue(a[11]);
        void *stream = PyLong_AsVoidPtr(a[0]);
        must(!PyErr_Occurred() && dv > 0 && dv <= INT32_MAX && want >= 0);
        at::Tensor out, lse, workspace;
        int status;
        {
            const Unlocked unlocked;
            const int64_t need =
                workspace_fn(size32(T), s.n, size32(hq), size32(H), size32(d), (int32_t)dv, c.size,
                             s.width, size32(P), kind.code);
            must(need >= 0);
            out = at::empty({T, hq, dv}, q->options());
            if (want) lse = at::empty({T, hq}, q->options().dtype(at::kFloat));
            if (need) workspace = at::empty({need}, q->options().dtype(at::kByte));
            status = attn_fn(
                pointer(q), pointer(kc), pointer(vc), s.table, s.lens,
                static_cast<const int32_t *>(pointer(pages)),
                static_cast<const int32_t *>(pointer(length)), s.cu, out.data_ptr(),
                want ? static_cast<float *>(lse.data_ptr()) : nullptr, size32(T), s.n, size32(hq),
                size32(H), size32(d), (int32_t)dv, c.pages, c.size, s.width, size32(P), qs, hq * dv,
                c.page, c.token, c.head, (float)scale, kind.code, need ? workspace.data_ptr() : nullptr,
                need, stream);
        }
        return result(status, out, &lse);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// bind(address of kda_cache_append, of kda_prefix_attn_fwd, of kda_prefix_attn_workspace_size)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "bind takes three addresses");
        return nullptr;
    }
    void *p[3];
    for (int i = 0; i < 3; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
    append_fn = reinterpret_cast<AppendFn>(p[0]);
    attn_fn = reinterpret_cast<AttnFn>(p[1]);
    workspace_fn = reinterpret_cast<WorkspaceFn>(p[2]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"append", (PyCFunction)(void *)append, METH_FASTCALL, "kda_cache_append, the common case"},
    {"attention", (PyCFunction)(void *)attention, METH_FASTCALL, "kda_prefix_attn_fwd, the common case"},
    {"bind", (PyCFunction)(void *)bind, METH_FASTCALL, "the library's entry points"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_calls(void) { return PyModule_Create(&module); }
