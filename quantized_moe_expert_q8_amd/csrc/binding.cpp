// Torch side of the operators around the expert layer: checks of the tensors,
// outputs that the caller did not give, and the call into the C library, in
// C++.  Their kernels take 3 to 6 us for a few tokens, where checks of up to 13
// tensors in Python and a ctypes call of 16 to 22 arguments took longer than
// the kernel: eager calls one after another took 8.1 us for rms_norm_q8 of one
// row of 4096 (now 3.9, its kernel's time) and 11.5 us for logits_process of 5 x
// 131072 (now 6.7).
//
// The library's functions come as addresses (bind), so whatever file ctypes has
// loaded serves these calls too.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moeq8.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Library {
    decltype(&::rms_norm_q8) rms_norm_q8;
    decltype(&::i8_quantize_rows) i8_quantize_rows;
    decltype(&::gemm_i8) gemm_i8;
    decltype(&::logits_process) logits_process;
};
Library lib{};
PyObject* fail = nullptr;                         // raises for (name, status)
PyTypeObject* norm_type = nullptr;                // the tuple that rms_norm_q8 returns

std::string type_name(ScalarType t) { return std::string("torch.") + torch::getTHPDtype(t)->name; }

bool given(PyObject* o) { return o != Py_None; }

// ---- checks: one condition where all is well, the reason found afterwards ----

[[noreturn]] void refuse(PyObject* o, const char* name, ScalarType dtype, int64_t dev, at::IntArrayRef shape) {
    TORCH_CHECK_VALUE(THPVariable_Check(o) && THPVariable_Unpack(o).get_device() == dev, name,
                      " must be a device tensor, on the same device as the others");
    const Tensor& t = THPVariable_Unpack(o);
    TORCH_CHECK_TYPE(t.scalar_type() == dtype, name, " must be ", type_name(dtype), ", got ", type_name(t.scalar_type()));
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must be ", shape, ", got ", t.sizes());
    TORCH_CHECK_VALUE(false, name, " must have unit inner stride");
}

// A matrix [rows, cols] of rows whose elements lie together, and its row stride.
int64_t matrix(PyObject* o, const char* name, ScalarType dtype, int64_t dev, int64_t rows, int64_t cols) {
    if (THPVariable_Check(o)) {
        const Tensor& t = THPVariable_Unpack(o);
        if (t.dim() == 2 && t.scalar_type() == dtype && t.get_device() == dev && t.size(0) == rows && t.size(1) == cols &&
            (cols <= 1 || t.stride(1) == 1))
            return rows > 1 ? t.stride(0) : cols;
    }
    refuse(o, name, dtype, dev, {rows, cols});
}

// The address of a contiguous vector of n elements.
void* vector(PyObject* o, const char* name, ScalarType dtype, int64_t dev, int64_t n) {
    if (THPVariable_Check(o)) {
        const Tensor& t = THPVariable_Unpack(o);
        if (t.dim() == 1 && t.scalar_type() == dtype && t.get_device() == dev && t.size(0) == n &&
            (n <= 1 || t.stride(0) == 1))
            return t.data_ptr();
    }
    refuse(o, name, dtype, dev, {n});
}
void* vector_or_null(PyObject* o, const char* name, ScalarType dtype, int64_t dev, int64_t n) {
    return given(o) ? vector(o, name, dtype, dev, n) : nullptr;
}

// The 2-D device tensor a call goes by.
const Tensor& first(PyObject* o, const char* name) {
    TORCH_CHECK_VALUE(THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(), name, " must be a device tensor");
    const Tensor& t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(t.dim() == 2, name, " must be 2-D, got ", t.sizes());
    return t;
}

int32_t dtype_code(const Tensor& t, const char* name) {
    switch (t.scalar_type()) {
        case ScalarType::Float: return MOEQ8_F32;
        case ScalarType::Half: return MOEQ8_F16;
        case ScalarType::BFloat16: return MOEQ8_BF16;
        default: break;
    }
    TORCH_CHECK_TYPE(false, name, " must be a float32, float16 or bfloat16 tensor");
}

int64_t count_of(PyObject* o, const char* name) {
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a device tensor, on the same device as the others");
    return THPVariable_Unpack(o).numel();
}

// An object held for the length of a call.
struct Held {
    PyObject* o;
    explicit Held(PyObject* p) : o(p) {}
    Held(Held&& h) noexcept : o(h.o) { h.o = nullptr; }
    Held(const Held&) = delete;
    ~Held() { Py_XDECREF(o); }
    PyObject* give() { PyObject* p = o; o = nullptr; return p; }
    void* data() const { return o == Py_None ? nullptr : THPVariable_Unpack(o).data_ptr(); }
};

Held keep(PyObject* o) { Py_INCREF(o); return Held(o); }

// The output the caller gave, or a new one.
Held given_or_new(PyObject* o, at::IntArrayRef shape, const Tensor& like, ScalarType dtype) {
    if (given(o)) return keep(o);
    PyObject* made = THPVariable_Wrap(at::empty(shape, like.options().dtype(dtype)));
    if (!made) throw python_error();
    return Held(made);
}

void* stream_of(int64_t dev) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }

template <typename F>
void run(const char* name, F call) {
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = call();
    Py_END_ALLOW_THREADS
    if (status == MOEQ8_OK) return;
    Py_XDECREF(PyObject_CallFunction(fail, "si", name, status));
    throw python_error();
}

bool arguments(const char* name, Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
    return false;
}

ScalarType type_of(PyObject* o) {
    TORCH_CHECK_TYPE(THPDtype_Check(o), "not a torch dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

const char* text(PyObject* o) {
    const char* s = PyUnicode_AsUTF8(o);
    if (!s) throw python_error();
    return s;
}

// ---- entry points ---------------------------------------------------------------

PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments("bind", n, 6)) return nullptr;
    TORCH_CHECK_TYPE(PyCallable_Check(a[4]) && PyType_Check(a[5]) &&
                         PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(a[5]), &PyTuple_Type),
                     "bind takes four addresses, a callable and a tuple type");
    auto address = [&](int i) {
        void* p = PyLong_AsVoidPtr(a[i]);
        if (!p && PyErr_Occurred()) throw python_error();
        return p;
    };
    lib.rms_norm_q8 = reinterpret_cast<decltype(lib.rms_norm_q8)>(address(0));
    lib.i8_quantize_rows = reinterpret_cast<decltype(lib.i8_quantize_rows)>(address(1));
    lib.gemm_i8 = reinterpret_cast<decltype(lib.gemm_i8)>(address(2));
    lib.logits_process = reinterpret_cast<decltype(lib.logits_process)>(address(3));
    Py_INCREF(a[4]);
    Py_INCREF(a[5]);
    Py_XDECREF(fail);
    Py_XDECREF(reinterpret_cast<PyObject*>(norm_type));
    fail = a[4];
    norm_type = reinterpret_cast<PyTypeObject*>(a[5]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// matrix(tensor, name, dtype, device index, rows, cols) -> row stride
PyObject* py_matrix(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments("matrix", n, 6)) return nullptr;
    return PyLong_FromLongLong(matrix(a[0], text(a[1]), type_of(a[2]), integer(a[3]), integer(a[4]), integer(a[5])));
    END_HANDLE_TH_ERRORS
}

// vector(tensor, name, dtype, device index, n) -> address
PyObject* py_vector(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments("vector", n, 5)) return nullptr;
    return PyLong_FromVoidPtr(vector(a[0], text(a[1]), type_of(a[2]), integer(a[3]), integer(a[4])));
    END_HANDLE_TH_ERRORS
}

// rms_norm_q8(x, w, eps, residual, residual_out, fmt, q, scale, xq) -> (q, scale, xq, residual_out)
PyObject* py_rms_norm_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments("rms_norm_q8", n, 9)) return nullptr;
    PyObject *px = a[0], *pres = a[3], *pout = a[4];
    const Tensor& x = first(px, "x");
    const int32_t code = dtype_code(x, "x");
    const char* fmt = PyUnicode_Check(a[5]) ? text(a[5]) : "";
    const bool both = !strcmp(fmt, "both"), i8 = both || !strcmp(fmt, "i8"), q8_1 = both || !strcmp(fmt, "q8_1");
    if (!i8 && !q8_1) {
        PyErr_Format(PyExc_ValueError, "fmt must be one of ('i8', 'q8_1', 'both'), got %R", a[5]);
        return nullptr;
    }
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const int64_t dev = x.get_device(), rows = x.size(0), k = x.size(1);
    const ScalarType t = x.scalar_type();
    const int64_t xs = matrix(px, "x", t, dev, rows, k);
    const void* w = vector(a[1], "w", t, dev, k);
    int64_t rs = 0, ros = 0, qs = 0;
    Held residual = keep(Py_None), q = keep(Py_None), scale = keep(Py_None), xq = keep(Py_None);
    if (given(pres)) {
        rs = matrix(pres, "residual", t, dev, rows, k);
        Held r = given_or_new(pout, {rows, k}, x, t);
        ros = matrix(r.o, "residual_out", t, dev, rows, k);
        std::swap(residual.o, r.o);
    } else {
        TORCH_CHECK_VALUE(!given(pout), "residual_out without a residual");
    }
    if (i8) {
        Held c = given_or_new(a[6], {rows, k}, x, ScalarType::Char);
        Held s = given_or_new(a[7], {rows}, x, ScalarType::Float);
        qs = matrix(c.o, "q", ScalarType::Char, dev, rows, k);
        vector(s.o, "scale", ScalarType::Float, dev, rows);
        std::swap(q.o, c.o);
        std::swap(scale.o, s.o);
    }
    if (q8_1) {
        TORCH_CHECK_VALUE(k % 32 == 0, "q8_1 rows need k to be a multiple of 32, got ", k);
        const int64_t bytes = k / 32 * 36;
        Held c = given_or_new(a[8], {rows, bytes}, x, ScalarType::Byte);
        TORCH_CHECK_VALUE(matrix(c.o, "xq", ScalarType::Byte, dev, rows, bytes) == bytes, "xq rows must be contiguous");
        std::swap(xq.o, c.o);
    }
    if (rows) {
        const void* pr = given(pres) ? THPVariable_Unpack(pres).data_ptr() : nullptr;
        void *po = residual.data(), *pq = q.data(), *ps = scale.data(), *pxq = xq.data(), *stream = stream_of(dev);
        const void* xp = x.data_ptr();
        run("rms_norm_q8", [=] {
            return lib.rms_norm_q8(xp, xs, pr, rs, po, ros, w, code, rows, k, eps, (int8_t*)pq, qs, (float*)ps, pxq, stream);
        });
    }
    // a NamedTuple of Python, made as the tuple it is
    PyObject* values = PyTuple_New(4);
    if (!values) return nullptr;
    PyTuple_SET_ITEM(values, 0, q.give());
    PyTuple_SET_ITEM(values, 1, scale.give());
    PyTuple_SET_ITEM(values, 2, xq.give());
    PyTuple_SET_ITEM(values, 3, residual.give());
    Held args(PyTuple_Pack(1, values));
    Py_DECREF(values);
    return args.o ? PyTuple_Type.tp_new(norm_type, args.o, nullptr) : nullptr;
    END_HANDLE_TH_ERRORS
}

// i8_quantize_rows(x, q, scale) -> (q, scale)
PyObject* py_i8_quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments("i8_quantize_rows", n, 3)) return nullptr;
    const Tensor& x = first(a[0], "x");
    const int32_t code = dtype_code(x, "x");
    const int64_t dev = x.get_device(), rows = x.size(0), k = x.size(1);
    const int64_t xs = matrix(a[0], "x", x.scalar_type(), dev, rows, k);
    Held q = given_or_new(a[1], {rows, k}, x, ScalarType::Char);
    Held scale = given_or_new(a[2], {rows}, x, ScalarType::Float);
    const int64_t qs = matrix(q.o, "q", ScalarType::Char, dev, rows, k);
    void* ps = vector(scale.o, "scale", ScalarType::Float, dev, rows);
    if (rows) {
        const void* xp = x.data_ptr();
        void *pq = q.data(), *stream = stream_of(dev);
        run("i8_quantize_rows",
            [=] { return lib.i8_quantize_rows(xp, code, rows, k, xs, (int8_t*)pq, qs, (float*)ps, stream); });
    }
    return PyTuple_Pack(2, q.o, scale.o);
    END_HANDLE_TH_ERRORS
}

// gemm_i8(a, sa, b, sb, bias, out, out_dtype) -> out
PyObject* py_gemm_i8(PyObject*, PyObject* const* p, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (!arguments("gemm_i8", count, 7)) return nullptr;
    const Tensor &a = first(p[0], "a"), &b = first(p[2], "b");
    const int64_t dev = a.get_device(), m = a.size(0), k = a.size(1), n = b.size(0);
    const int64_t as = matrix(p[0], "a", ScalarType::Char, dev, m, k);
    const int64_t bs = matrix(p[2], "b", ScalarType::Char, dev, n, k);
    const void* sa = vector(p[1], "sa", ScalarType::Float, dev, m);
    const void* sb = vector(p[3], "sb", ScalarType::Float, dev, n);
    const void* bias = vector_or_null(p[4], "bias", ScalarType::Float, dev, n);
    Held out = given_or_new(p[5], {m, n}, a, given(p[5]) ? ScalarType::Float : type_of(p[6]));
    TORCH_CHECK_TYPE(THPVariable_Check(out.o), "out must be a float32, float16 or bfloat16 tensor");
    const Tensor& o = THPVariable_Unpack(out.o);
    const int32_t code = dtype_code(o, "out");
    const int64_t os = matrix(out.o, "out", o.scalar_type(), dev, m, n);
    if (m && n) {
        const void *pa = a.data_ptr(), *pb = b.data_ptr();
        void *po = out.data(), *stream = stream_of(dev);
        run("gemm_i8", [=] {
            return lib.gemm_i8((const int8_t*)pa, as, (const float*)sa, (const int8_t*)pb, bs, (const float*)sb,
                               (const float*)bias, m, n, k, code, po, os, stream);
        });
    }
    return out.give();
    END_HANDLE_TH_ERRORS
}

// logits_process(logits, tokens, begin, end, prompt_end, repetition, frequency, presence, bias_ids, bias_values,
//                bias_offsets, mask, out) -> out
PyObject* py_logits_process(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments("logits_process", n, 13)) return nullptr;
    const Tensor& z = first(a[0], "logits");
    const int32_t code = dtype_code(z, "logits");
    const ScalarType t = z.scalar_type();
    const int64_t dev = z.get_device(), rows = z.size(0), vocab = z.size(1);
    const int64_t zs = matrix(a[0], "logits", t, dev, rows, vocab);
    Held out = given_or_new(a[12], {rows, vocab}, z, t);
    const int64_t os = matrix(out.o, "out", t, dev, rows, vocab);
    const void *tokens = nullptr, *begin = nullptr, *end = nullptr, *prompt_end = nullptr, *rep = nullptr, *freq = nullptr,
               *pres = nullptr, *ids = nullptr, *values = nullptr, *offsets = nullptr, *mask = nullptr;
    int64_t n_tokens = 0, n_bias = 0, ms = 0;
    if (given(a[1])) {
        TORCH_CHECK_VALUE(given(a[2]) && given(a[3]), "tokens need begin and end");
        n_tokens = count_of(a[1], "tokens");
        tokens = vector(a[1], "tokens", ScalarType::Int, dev, n_tokens);
        begin = vector(a[2], "begin", ScalarType::Long, dev, rows);
        end = vector(a[3], "end", ScalarType::Long, dev, rows);
        prompt_end = vector_or_null(a[4], "prompt_end", ScalarType::Long, dev, rows);
        rep = vector_or_null(a[5], "repetition", ScalarType::Float, dev, rows);
        freq = vector_or_null(a[6], "frequency", ScalarType::Float, dev, rows);
        pres = vector_or_null(a[7], "presence", ScalarType::Float, dev, rows);
        if (!n_tokens) tokens = begin = end = prompt_end = rep = freq = pres = nullptr;     // an empty list has no address
    } else {
        for (int i = 2; i < 8; ++i) TORCH_CHECK_VALUE(!given(a[i]), "penalties need tokens");
    }
    TORCH_CHECK_VALUE(given(a[8]) == given(a[9]) && given(a[8]) == given(a[10]),
                      "bias_ids, bias_values and bias_offsets go together");
    if (given(a[8])) {
        n_bias = count_of(a[8], "bias_ids");
        ids = vector(a[8], "bias_ids", ScalarType::Int, dev, n_bias);
        values = vector(a[9], "bias_values", ScalarType::Float, dev, n_bias);
        offsets = vector(a[10], "bias_offsets", ScalarType::Long, dev, rows + 1);
        if (!n_bias) ids = values = offsets = nullptr;
    }
    if (given(a[11])) {
        ms = matrix(a[11], "mask", ScalarType::Int, dev, rows, (vocab + 31) / 32);
        mask = THPVariable_Unpack(a[11]).data_ptr();
    }
    if (rows && vocab) {
        const void* pz = z.data_ptr();
        void *po = out.data(), *stream = stream_of(dev);
        run("logits_process", [=] {
            return lib.logits_process(pz, zs, code, rows, vocab, (const int32_t*)tokens, n_tokens, (const int64_t*)begin,
                                      (const int64_t*)end, (const int64_t*)prompt_end, (const float*)rep, (const float*)freq,
                                      (const float*)pres, (const int32_t*)ids, (const float*)values, n_bias,
                                      (const int64_t*)offsets, (const int32_t*)mask, ms, po, os, stream);
        });
    }
    return out.give();
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<py_bind>("bind"), method<py_matrix>("matrix"), method<py_vector>("vector"),
                         method<py_rms_norm_q8>("rms_norm_q8"), method<py_i8_quantize_rows>("i8_quantize_rows"),
                         method<py_gemm_i8>("gemm_i8"), method<py_logits_process>("logits_process"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
