// binding.cpp -- argument marshalling of the decoder-layer calls (qmm_linear,
// qmm_kv_append, qmm_paged_attention) for Python: checks the tensors, fills the
// C ABI's argument blocks and calls the library.  In C++ because these calls
// are made many times for each token, where reading 30 tensor attributes from
// Python costs more than the kernels of a short step (one token: 4.5 to 5.8 us
// of 7 to 9 a call).  Nothing is computed here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "../../include/qmm.h"

namespace {

struct Library {
    decltype(&qmm_linear) linear;
    decltype(&qmm_linear_workspace) linear_workspace;
    decltype(&qmm_kv_append) kv_append;
    decltype(&qmm_paged_attention) attention;
    decltype(&qmm_paged_attention_workspace) attention_workspace;
} lib;
PyObject *raise_status, *raw_stream, *get_device, *set_device;   // Python callables, held for the process

struct Refused {
    PyObject *type;
    std::string text;
};
[[noreturn]] void bad_type(const std::string &text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void bad_value(const std::string &text) { throw Refused{PyExc_ValueError, text}; }
struct Raised {};   // a Python error is set

std::string show(at::IntArrayRef v)
{
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor *maybe(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }
const void *at(const at::Tensor *t) { return t ? t->const_data_ptr() : nullptr; }

void same_device(const at::Tensor &t, const char *name, int index)
{
    if (!t.is_cuda()) bad_value(std::string(name) + " must be a GPU tensor");
    if (t.get_device() != index) bad_value(std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(index));
}
void shaped(const at::Tensor &t, const char *name, at::IntArrayRef shape)
{
    if (t.sizes() != shape) bad_value(std::string(name) + " has shape " + show(t.sizes()) + ", expected " + show(shape));
}
void typed(const at::Tensor &t, const char *name, at::ScalarType type)
{
    if (t.scalar_type() != type) bad_type(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
}
void dense(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, int index)
{
    typed(t, name, type);
    same_device(t, name, index);
    shaped(t, name, shape);
    if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
}
// [tokens, heads, D] whose rows' elements stand side by side: strides of token and head
void rows(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, int index, int64_t (&stride)[2])
{
    typed(t, name, type);
    same_device(t, name, index);
    shaped(t, name, shape);
    if (t.stride(2) != 1 && shape[2] > 1) bad_value(std::string(name) + ": the elements of a row must stand side by side");
    stride[0] = t.stride(0);
    stride[1] = t.stride(1);
}
// two caches [pages, heads, page, D]; returns the type's code
int caches(const at::Tensor &k, const at::Tensor &v, at::ScalarType type, int code, int index, const at::Tensor *k_scale,
           const at::Tensor *v_scale, int64_t (&ks)[3], int64_t (&vs)[3])
{
    if (k.dim() != 4) bad_value("k_cache must be [pages, heads, page, D]");
    if (v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type()) bad_value("k_cache and v_cache must have one shape and one type");
    const bool e4m3 = k.scalar_type() == at::kFloat8_e4m3fn;
    if (!e4m3 && k.scalar_type() != type)
        bad_type(std::string("the caches must be ") + c10::toString(type) + " or Float8_e4m3fn, got " + c10::toString(k.scalar_type()));
    same_device(k, "k_cache", index);
    same_device(v, "v_cache", index);
    if ((k.stride(3) != 1 || v.stride(3) != 1) && k.size(3) > 1) bad_value("the elements of a cache's token must stand side by side");
    if (e4m3) {
        if (!k_scale || !v_scale) bad_value("e4m3 caches need k_scale and v_scale");
        dense(*k_scale, "k_scale", at::kFloat, {k.size(1)}, index);
        dense(*v_scale, "v_scale", at::kFloat, {k.size(1)}, index);
    } else if (k_scale || v_scale) {
        bad_value("k_scale and v_scale are for e4m3 caches");
    }
    for (int i = 0; i < 3; ++i) {
        ks[i] = k.stride(i);
        vs[i] = v.stride(i);
    }
    return e4m3 ? QMM_E4M3 : code;
}
// the tensor [tokens, heads, D] that leads a call: its device, and the code of its type
int leading(const at::Tensor &t, const char *name, int &index)
{
    const at::ScalarType type = t.scalar_type();
    if (type != at::kHalf && type != at::kBFloat16) bad_type(std::string(name) + " must be Half or BFloat16, got " + c10::toString(type));
    if (!t.is_cuda()) bad_value(std::string(name) + " must be a GPU tensor");
    if (t.dim() != 3) bad_value(std::string(name) + " must be [tokens, heads, D]");
    index = (int)t.get_device();
    return type == at::kHalf ? QMM_F16 : QMM_BF16;
}

int64_t integer(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        bad_type(std::string(name) + " must be an integer of 64 bits");
    }
    return v;
}
int64_t from(PyObject *callable, int argument, bool given)
{
    PyObject *r = given ? PyObject_CallFunction(callable, "i", argument) : PyObject_CallNoArgs(callable);
    if (!r) throw Raised{};
    const int64_t v = r == Py_None ? 0 : (int64_t)PyLong_AsUnsignedLongLong(r);
    Py_DECREF(r);
    return v;
}
// f(the device's current stream) with that device current
template <typename F>
void on_device(int index, F &&f)
{
    const void *stream = reinterpret_cast<const void *>(from(raw_stream, index, true));
    const int64_t now = from(get_device, 0, false);
    if (now != index) from(set_device, index, true);
    const int status = f(const_cast<void *>(stream));
    if (now != index) from(set_device, (int)now, true);
    if (status != QMM_OK) {
        PyObject *r = PyObject_CallFunction(raise_status, "i", status);
        Py_XDECREF(r);
        if (!r) throw Raised{};
    }
}
// scratch of this call: the allocator hands it out again only to work behind the call on its stream
at::Tensor scratch(int64_t bytes, const at::Tensor &like) { return at::empty({bytes}, like.options().dtype(at::kByte)); }

PyObject *give(PyObject *given, const at::Tensor &made)
{
    if (given != Py_None) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(made);
}

template <typename F>
PyObject *guarded(F &&f)
{
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.text.c_str());
        return nullptr;
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
void count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) bad_type("wrong number of arguments");
}

// (X, wq, s, z, bits, G, bias, act, mul, residual, out)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        count(n, 11);
        const at::Tensor &X = tensor(a[0], "X"), &wq = tensor(a[1], "wq"), &s = tensor(a[2], "s");
        const at::Tensor *z = maybe(a[3], "z"), *bias = maybe(a[6], "bias"), *mul = maybe(a[8], "mul"), *res = maybe(a[9], "residual"),
                         *out = maybe(a[10], "out");
        const int64_t bits = integer(a[4], "bits"), G = integer(a[5], "G"), act = integer(a[7], "act");
        if (X.dim() != 2 || s.dim() != 2) bad_value("X must be [M, K] and s [N, K / G]");
        if (G < 1 || bits < 1 || bits > 8) bad_value("G must be positive and bits 1 to 8");
        const int64_t M = X.size(0), K = X.size(1), N = s.size(0);
        typed(X, "X", at::kHalf);
        if (!X.is_cuda()) bad_value("X must be a GPU tensor");
        if (!X.is_contiguous()) bad_value("X must be contiguous");
        const int index = (int)X.get_device();
        dense(wq, "wq", at::kInt, {N, K * bits / 32}, index);
        dense(s, "s", at::kHalf, {N, K / G}, index);
        if (z) dense(*z, "z", at::kHalf, {N, K / G}, index);
        if (bias) dense(*bias, "bias", at::kHalf, {N}, index);
        if (mul) dense(*mul, "mul", at::kHalf, {M, N}, index);
        if (res) dense(*res, "residual", at::kHalf, {M, N}, index);
        if (out) dense(*out, "out", at::kHalf, {M, N}, index);
        const at::Tensor y = out ? *out : at::empty({M, N}, X.options());
        if (M > 0) {
            qmm_linear_args p{};
            p.X = (const qmm_half *)at(&X), p.wq = (const uint32_t *)at(&wq), p.s = (const qmm_half *)at(&s), p.z = (const qmm_half *)at(z);
            p.Y = (qmm_half *)y.mutable_data_ptr();
            p.bias = (const qmm_half *)at(bias), p.mul = (const qmm_half *)at(mul), p.residual = (const qmm_half *)at(res);
            p.M = M, p.K = K, p.N = N, p.G = G, p.bits = (int)bits, p.act = (int)act;
            at::Tensor space;
            if ((p.workspace_bytes = lib.linear_workspace(&p)) > 0) {
                space = scratch(p.workspace_bytes, X);
                p.workspace = space.mutable_data_ptr();
            }
            on_device(index, [&](void *stream) { return lib.linear(&p, stream); });
        }
        return give(a[10], y);
    });
}

// (q, k, v, k_cache, v_cache, slots, positions, rope, pairs, k_scale, v_scale, out)
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        count(n, 12);
        const at::Tensor *q = maybe(a[0], "q"), *positions = maybe(a[6], "positions"), *rope = maybe(a[7], "rope"),
                         *k_scale = maybe(a[9], "k_scale"), *v_scale = maybe(a[10], "v_scale"), *out = maybe(a[11], "out");
        const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache"),
                         &slots = tensor(a[5], "slots");
        qmm_kv_append_args p{};
        int index;
        p.pairs = PyObject_IsTrue(a[8]);
        if (p.pairs < 0) throw Raised{};
        p.dtype = leading(k, "k", index);
        const at::ScalarType type = k.scalar_type();
        p.T = k.size(0), p.Hkv = k.size(1), p.D = k.size(2);
        rows(k, "k", type, k.sizes(), index, p.k_stride);
        rows(v, "v", type, k.sizes(), index, p.v_stride);
        at::Tensor y;
        if (q) {
            if (q->dim() != 3) bad_value("q must be [tokens, heads, D]");
            p.Hq = q->size(1);
            rows(*q, "q", type, {p.T, p.Hq, p.D}, index, p.q_stride);
            if (out) rows(*out, "out", type, {p.T, p.Hq, p.D}, index, p.out_stride);
            y = out ? *out : at::empty({p.T, p.Hq, p.D}, q->options());
            p.out_stride[0] = y.stride(0), p.out_stride[1] = y.stride(1);
            p.q = at(q), p.out = y.mutable_data_ptr();
        } else if (out) {
            bad_value("out without q");
        }
        p.cache_dtype = caches(kc, vc, type, p.dtype, index, k_scale, v_scale, p.k_cache_stride, p.v_cache_stride);
        if (kc.size(1) != p.Hkv || kc.size(3) != p.D)
            bad_value("k_cache has shape " + show(kc.sizes()) + ", expected [pages, " + std::to_string(p.Hkv) + ", page, " + std::to_string(p.D) + "]");
        p.pages = kc.size(0), p.page = kc.size(2);
        dense(slots, "slots", at::kLong, {p.T}, index);
        if (rope) {
            if (!positions) bad_value("rope needs positions");
            if (rope->dim() != 2) bad_value("rope must be [rows, rot]");
            p.table_rows = rope->size(0), p.rot = rope->size(1);
            dense(*rope, "rope", at::kFloat, rope->sizes(), index);
            dense(*positions, "positions", at::kInt, {p.T}, index);
        } else if (positions) {
            bad_value("positions without rope");
        }
        p.k = at(&k), p.v = at(&v), p.k_cache = kc.mutable_data_ptr(), p.v_cache = vc.mutable_data_ptr();
        p.slots = (const int64_t *)at(&slots), p.positions = (const int32_t *)at(positions), p.rope = (const float *)at(rope);
        p.k_scale = (const float *)at(k_scale), p.v_scale = (const float *)at(v_scale);
        on_device(index, [&](void *stream) { return lib.kv_append(&p, stream); });
        if (!q) Py_RETURN_NONE;
        return give(a[11], y);
    });
}

// (q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q, max_kv, scale, window, k_scale, v_scale, out, lse)
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        count(n, 14);
        const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"), &table = tensor(a[3], "page_table"),
                         &cu = tensor(a[4], "cu_q"), &lens = tensor(a[5], "kv_lens");
        const at::Tensor *k_scale = maybe(a[10], "k_scale"), *v_scale = maybe(a[11], "v_scale"), *out = maybe(a[12], "out"), *lse = maybe(a[13], "lse");
        qmm_attention_args p{};
        int index;
        p.dtype = leading(q, "q", index);
        const at::ScalarType type = q.scalar_type();
        p.T = q.size(0), p.Hq = q.size(1), p.D = q.size(2);
        rows(q, "q", type, q.sizes(), index, p.q_stride);
        p.cache_dtype = caches(kc, vc, type, p.dtype, index, k_scale, v_scale, p.k_cache_stride, p.v_cache_stride);
        if (kc.size(3) != p.D) bad_value("k_cache has shape " + show(kc.sizes()) + ", expected [pages, heads, page, " + std::to_string(p.D) + "]");
        p.pages = kc.size(0), p.Hkv = kc.size(1), p.page = kc.size(2);
        if (table.dim() != 2) bad_value("page_table must be [sequences, width]");
        typed(table, "page_table", at::kInt);
        same_device(table, "page_table", index);
        p.B = table.size(0), p.width = table.size(1), p.table_stride = table.stride(0);
        if (table.stride(1) != 1 && p.width > 1) bad_value("page_table: the ids of a sequence must stand side by side");
        dense(cu, "cu_q", at::kInt, {p.B + 1}, index);
        dense(lens, "kv_lens", at::kInt, {p.B}, index);
        if (out) rows(*out, "out", type, q.sizes(), index, p.out_stride);
        const at::Tensor y = out ? *out : at::empty({p.T, p.Hq, p.D}, q.options());
        p.out_stride[0] = y.stride(0), p.out_stride[1] = y.stride(1);
        if (lse) dense(*lse, "lse", at::kFloat, {p.T, p.Hq}, index);
        p.max_q = integer(a[6], "max_q"), p.max_kv = integer(a[7], "max_kv"), p.window = integer(a[9], "window");
        p.scale = a[8] == Py_None ? 1.0 / std::sqrt((double)p.D) : PyFloat_AsDouble(a[8]);
        if (PyErr_Occurred()) throw Raised{};
        p.q = at(&q), p.k_cache = at(&kc), p.v_cache = at(&vc), p.out = y.mutable_data_ptr();
        p.lse = lse ? (float *)lse->mutable_data_ptr() : nullptr;
        p.page_table = (const int32_t *)at(&table), p.cu_q = (const int32_t *)at(&cu), p.kv_lens = (const int32_t *)at(&lens);
        p.k_scale = (const float *)at(k_scale), p.v_scale = (const float *)at(v_scale);
        at::Tensor space;
        if ((p.workspace_bytes = lib.attention_workspace(&p)) > 0) {
            space = scratch(p.workspace_bytes, q);
            p.workspace = space.mutable_data_ptr();
        }
        on_device(index, [&](void *stream) { return lib.attention(&p, stream); });
        return give(a[12], y);
    });
}

// (addresses of the five entry points, raise_status, raw_stream, get_device, set_device)
PyObject *connect(PyObject *, PyObject *args)
{
    unsigned long long f[5];
    PyObject *o[4];
    if (!PyArg_ParseTuple(args, "KKKKKOOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &o[0], &o[1], &o[2], &o[3])) return nullptr;
    lib.linear = reinterpret_cast<decltype(lib.linear)>(f[0]);
    lib.linear_workspace = reinterpret_cast<decltype(lib.linear_workspace)>(f[1]);
    lib.kv_append = reinterpret_cast<decltype(lib.kv_append)>(f[2]);
    lib.attention = reinterpret_cast<decltype(lib.attention)>(f[3]);
    lib.attention_workspace = reinterpret_cast<decltype(lib.attention_workspace)>(f[4]);
    for (PyObject *x : o) Py_INCREF(x);
    raise_status = o[0], raw_stream = o[1], get_device = o[2], set_device = o[3];
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"connect", connect, METH_VARARGS, nullptr},
    {"linear", (PyCFunction)(void *)linear, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void *)kv_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void *)paged_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
