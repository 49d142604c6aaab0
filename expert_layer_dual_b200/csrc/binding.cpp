// binding.cpp -- argument marshalling of the training entry points for Python:
// the checks of the tensors (shape, type, contiguity, device) and the call of the
// C ABI in one native step.  Written against CPython and the tensor object only;
// no arithmetic, no CUDA call of its own.  In Python a call's ten to fifteen
// tensors took longer to check than a small kernel to run (8 us against 4).
//
// Every function takes the current device's index and stream handle first, then
// the tensors and numbers of the entry point's Python wrapper, and returns the
// entry point's status.  A tensor that is not what the call needs raises
// ValueError; nothing is launched then.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe.h"

namespace {

struct Args {
    PyObject* const* a;
    int64_t dev;
    void* stream;
    bool ok = true;

    bool open(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) {
        if (n != want) {
            PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
            return false;
        }
        a = args;
        dev = PyLong_AsLongLong(args[0]);
        stream = PyLong_AsVoidPtr(args[1]);
        return !PyErr_Occurred();
    }

    const at::Tensor* tensor(int i, const char* name) {
        if (!ok) return nullptr;
        if (!THPVariable_Check(a[i])) {
            PyErr_Format(PyExc_ValueError, "%s: not a tensor", name);
            ok = false;
            return nullptr;
        }
        const at::Tensor& t = THPVariable_Unpack(a[i]);
        if (t.is_neg() || t._is_zerotensor()) {  // their memory does not hold their values
            PyErr_Format(PyExc_ValueError, "%s: a negated view or a zero without memory; resolve it first", name);
            ok = false;
            return nullptr;
        }
        return &t;
    }

    int64_t integer(int i) {
        if (!ok) return 0;
        const int64_t v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) ok = false;
        return v;
    }
    float real(int i) {
        if (!ok) return 0.0f;
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) ok = false;
        return static_cast<float>(v);
    }
    bool none(int i) const { return a[i] == Py_None; }

    void refuse(const char* name, const at::Tensor& t, const char* want) {
        const std::string has = c10::str(t.sizes(), " ", t.scalar_type(), " on ", t.device(),
                                         t.is_contiguous() ? ", contiguous" : ", not contiguous");
        PyErr_Format(PyExc_ValueError, "%s: %s; expected %s, contiguous, on cuda:%lld, the current CUDA device",
                     name, has.c_str(), want, static_cast<long long>(dev));
        ok = false;
    }

    // The address of tensor i if it is contiguous, of one of the types and on the
    // current device, with the given sizes (rank 0: any shape of `elements`).
    template <typename Type>
    const void* data(int i, const char* name, std::initializer_list<int64_t> sizes, Type is_type,
                     const char* type_name, int64_t elements = -1) {
        const at::Tensor* t = tensor(i, name);
        if (t == nullptr) return nullptr;
        bool fits = is_type(t->scalar_type()) && t->is_cuda() && t->get_device() == dev && t->is_contiguous();
        if (elements >= 0)
            fits = fits && t->numel() == elements;
        else
            fits = fits && t->sizes() == at::IntArrayRef(sizes);
        if (!fits) {
            const std::string want = elements >= 0
                                         ? c10::str(elements, " elements of ", type_name)
                                         : c10::str(at::IntArrayRef(sizes), " ", type_name);
            refuse(name, *t, want.c_str());
            return nullptr;
        }
        return t->const_data_ptr();
    }
    static bool f32(at::ScalarType s) { return s == at::kFloat; }
    static bool i32(at::ScalarType s) { return s == at::kInt; }
    static bool codes(at::ScalarType s) { return s == at::kByte || s == at::kFloat8_e4m3fn; }
    static bool bf16(at::ScalarType s) { return s == at::kBFloat16 || s == at::kUInt16; }
    static bool halves(at::ScalarType s) { return bf16(s) || s == at::kShort; }
    static bool bytes(at::ScalarType s) { return codes(s) || s == at::kChar; }
    static bool flags(at::ScalarType s) { return s == at::kByte || s == at::kBool; }
    static bool output(at::ScalarType s) { return bf16(s) || s == at::kHalf || s == at::kFloat; }

    const float* floats(int i, const char* name, std::initializer_list<int64_t> sizes) {
        return static_cast<const float*>(data(i, name, sizes, f32, "float32"));
    }
    const float* floats_n(int i, const char* name, int64_t n) {
        return static_cast<const float*>(data(i, name, {}, f32, "float32", n));
    }
    const int32_t* ints_n(int i, const char* name, int64_t n) {
        return static_cast<const int32_t*>(data(i, name, {}, i32, "int32", n));
    }
    // An output: `p` as the checks above gave it for tensor i, with storage of its own (a
    // lazily cloned tensor still shares its source's).
    template <typename T>
    T* written(int i, const T* p) {
        if (!ok || p == nullptr) return nullptr;
        return static_cast<T*>(THPVariable_Unpack(a[i]).mutable_data_ptr());
    }
    const uint8_t* e4m3(int i, const char* name, std::initializer_list<int64_t> sizes) {
        return static_cast<const uint8_t*>(data(i, name, sizes, codes, "uint8 or float8_e4m3fn"));
    }
    // Sizes 0 and 1 of a matrix (other ranks are refused).
    bool matrix(int i, const char* name, int64_t* rows, int64_t* cols) {
        const at::Tensor* t = tensor(i, name);
        if (t == nullptr) return false;
        if (t->dim() != 2) {
            refuse(name, *t, "a matrix");
            return false;
        }
        *rows = t->size(0);
        *cols = t->size(1);
        return true;
    }
    // Any contiguous tensor on the current device.
    const void* buffer(int i, const char* name, size_t* bytes = nullptr) {
        const at::Tensor* t = tensor(i, name);
        if (t == nullptr) return nullptr;
        if (!t->is_cuda() || t->get_device() != dev || !t->is_contiguous()) {
            refuse(name, *t, "a buffer");
            return nullptr;
        }
        if (bytes != nullptr) *bytes = t->nbytes();
        return t->const_data_ptr();
    }
    // Tensor i has to hold `elements` or more of one of the types, in any shape (None: none).
    template <typename Type>
    void room(int i, const char* name, Type is_type, const char* type_name, int64_t elements) {
        if (none(i) && elements == 0) return;
        const at::Tensor* t = tensor(i, name);
        if (t == nullptr || (is_type(t->scalar_type()) && t->numel() >= elements)) return;
        const std::string want = c10::str(elements, " elements or more of ", type_name);
        refuse(name, *t, want.c_str());
    }
    // The address of a contiguous tensor that the current device reaches: its own memory,
    // pinned host memory, another device's with peer access.
    const void* reachable(int i, const char* name) { return reach(i, name, false); }
    void* reachable_output(int i, const char* name) { return const_cast<void*>(reach(i, name, true)); }
    const void* reach(int i, const char* name, bool write) {
        const at::Tensor* t = tensor(i, name);
        if (t == nullptr) return nullptr;
        if (t->is_cuda() && t->get_device() == dev) {
            const void* p = buffer(i, name);
            return write ? written(i, p) : p;
        }
        const void* p = nullptr;
        if (t->is_contiguous()) p = moe_device_address(write ? t->mutable_data_ptr() : t->const_data_ptr());
        if (p == nullptr) refuse(name, *t, "a buffer that the device reaches");
        return p;
    }
    void* workspace(int i, size_t* bytes) { return written(i, buffer(i, "workspace", bytes)); }
    static bool fits_int(std::initializer_list<int64_t> v) {
        for (int64_t x : v)
            if (x < 0 || x > INT32_MAX) return false;
        return true;
    }
    // The entry point's status, called without the interpreter lock: a launch waits while the
    // stream's queue is full, and what empties it may be a Python callback in the stream.
    // The tensors stay alive: the caller holds the arguments.
    template <typename Call>
    PyObject* status(Call call) {
        if (!ok) return nullptr;
        struct Unlocked {
            PyThreadState* thread = PyEval_SaveThread();
            ~Unlocked() { PyEval_RestoreThread(thread); }
        };
        moe_status s;
        {
            Unlocked u;
            s = call();
        }
        return PyLong_FromLong(s);
    }
};

// [G] matrices [N][K] with or without the leading G; several need offsets.
bool weight_shape(Args& c, int i, const char* name, bool grouped, int64_t* G, int64_t* N, int64_t* K) {
    const at::Tensor* t = c.tensor(i, name);
    if (t == nullptr) return false;
    if (t->dim() != 2 && t->dim() != 3) {
        c.refuse(name, *t, "[N, K] or [G, N, K]");
        return false;
    }
    *G = t->dim() == 3 ? t->size(0) : 1;
    *N = t->size(-2);
    *K = t->size(-1);
    if (!grouped && *G != 1) {
        PyErr_SetString(PyExc_ValueError, "several weight matrices need offsets");
        return c.ok = false;
    }
    return true;
}

// (dev, stream, logits, ids, mask, coef, loss, counts, prob_mean, tokens, ws)
PyObject* balance_loss(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args c;
    int64_t T, E, T2, k;
    size_t bytes = 0;
    if (!c.open(args, n, 11) || !c.matrix(2, "logits", &T, &E) || !c.matrix(3, "ids", &T2, &k)) return nullptr;
    const float* logits = c.floats(2, "logits", {T, E});
    const int32_t* ids = static_cast<const int32_t*>(c.data(3, "ids", {T, k}, Args::i32, "int32"));
    const uint8_t* mask =
        c.none(4) ? nullptr : static_cast<const uint8_t*>(c.data(4, "mask", {}, Args::flags, "uint8 or bool", T));
    const float coef = c.real(5);
    float* loss = c.written(6, c.floats_n(6, "loss", 1));
    int32_t* counts = c.written(7, c.ints_n(7, "counts", E));
    float* mean = c.written(8, c.floats_n(8, "prob_mean", E));
    int32_t* tokens = c.written(9, c.ints_n(9, "tokens", 1));
    void* ws = c.workspace(10, &bytes);
    if (!c.ok) return nullptr;
    if (!Args::fits_int({T, E, k})) return PyLong_FromLong(MOE_ERR_UNSUPPORTED);
    return c.status([&] {
        return moe_balance_loss(logits, ids, mask, (int32_t)T, (int32_t)E, (int32_t)k, coef, loss, counts,
                                mean, tokens, ws, bytes, c.stream);
    });
}

// (dev, stream, logits, ids, w, dw, mask, renormalize, dloss, coef, counts, tokens, dlogits)
PyObject* route_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args c;
    int64_t T, E, T2, k;
    if (!c.open(args, n, 13) || !c.matrix(2, "logits", &T, &E) || !c.matrix(3, "ids", &T2, &k)) return nullptr;
    const float* logits = c.floats(2, "logits", {T, E});
    const int32_t* ids = static_cast<const int32_t*>(c.data(3, "ids", {T, k}, Args::i32, "int32"));
    const float *w = nullptr, *dw = nullptr, *dloss = nullptr;
    const int32_t *counts = nullptr, *tokens = nullptr;
    if (!c.none(5)) {
        w = c.floats(4, "w", {T, k});
        dw = c.floats(5, "dw", {T, k});
    }
    const uint8_t* mask =
        c.none(6) ? nullptr : static_cast<const uint8_t*>(c.data(6, "mask", {}, Args::flags, "uint8 or bool", T));
    const int renormalize = PyObject_IsTrue(args[7]);
    if (!c.none(8)) {
        dloss = c.floats_n(8, "dloss", 1);
        counts = c.ints_n(10, "counts", E);
        tokens = c.ints_n(11, "tokens", 1);
    }
    const float coef = c.real(9);
    float* dlogits = c.written(12, c.floats(12, "dlogits", {T, E}));
    if (!c.ok || renormalize < 0) return nullptr;
    if (!Args::fits_int({T, E, k})) return PyLong_FromLong(MOE_ERR_UNSUPPORTED);
    return c.status([&] {
        return moe_route_backward(logits, ids, w, dw, mask, (int32_t)T, (int32_t)E, (int32_t)k, renormalize,
                                  dloss, coef, counts, tokens, dlogits, c.stream);
    });
}

// (dev, stream, codes, scales, weight codes, weight scales, offsets, output, ws)
template <bool INPUT>
PyObject* product(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args c;
    int64_t M, cols, G, N, K;
    size_t bytes = 0;
    if (!c.open(args, n, 9) || !c.matrix(2, "codes", &M, &cols) ||
        !weight_shape(c, 4, "weight codes", !c.none(6), &G, &N, &K))
        return nullptr;
    const int64_t in = INPUT ? N : K, out_cols = INPUT ? K : N;
    const uint8_t* a = c.e4m3(2, "codes", {M, in});
    const float* as = c.floats(3, "scales", {M, in / 128});
    const bool grouped = c.ok && c.tensor(4, "weight codes")->dim() == 3;
    const uint8_t* w = grouped ? c.e4m3(4, "weight codes", {G, N, K}) : c.e4m3(4, "weight codes", {N, K});
    const float* wsc = grouped ? c.floats(5, "weight scales", {G, N / 128, K / 128})
                               : c.floats(5, "weight scales", {N / 128, K / 128});
    const int32_t* offsets = c.none(6) ? nullptr : c.ints_n(6, "offsets", G + 1);
    void* out = c.written(
        7, c.data(7, "output", {M, out_cols}, Args::output, "bfloat16, uint16, float16 or float32"));
    void* ws = c.workspace(8, &bytes);
    if (!c.ok) return nullptr;
    if (!Args::fits_int({G, M, N, K})) return PyLong_FromLong(MOE_ERR_UNSUPPORTED);
    const at::ScalarType type = c.tensor(7, "output")->scalar_type();
    const int32_t out_type = type == at::kFloat ? MOE_OUT_F32 : type == at::kHalf ? MOE_OUT_F16 : MOE_OUT_BF16;
    return c.status([&] {
        return (INPUT ? moe_gemm_fp8_dgrad : moe_gemm_fp8)(a, as, w, wsc, offsets, (int32_t)G, (int32_t)M,
                                                            (int32_t)N, (int32_t)K, out, out_type, ws, bytes,
                                                            c.stream);
    });
}

// (dev, stream, x, codes, scales): x gives the sizes; the buffers may have any shape, hold
// more than is written, and lie in any memory that the device reaches.
PyObject* quantize_act(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args c;
    int64_t M, cols;
    if (!c.open(args, n, 5) || !c.matrix(2, "x", &M, &cols)) return nullptr;
    c.room(2, "x", Args::halves, "bfloat16, uint16 or int16", M * cols);
    c.room(3, "codes", Args::bytes, "uint8, int8 or float8_e4m3fn", M * cols);
    c.room(4, "scales", Args::f32, "float32", M * (cols / 128));
    const void* x = nullptr;
    void *q = nullptr, *s = nullptr;
    if (M * cols > 0) {  // else nothing is asked of the buffers
        x = c.reachable(2, "x");
        q = c.reachable_output(3, "codes");
        s = c.reachable_output(4, "scales");
    }
    if (!c.ok) return nullptr;
    if (!Args::fits_int({cols})) return PyLong_FromLong(MOE_ERR_UNSUPPORTED);
    return c.status([&] {
        return moe_quantize_act_fp8(static_cast<const uint16_t*>(x), M, (int32_t)cols,
                                    static_cast<uint8_t*>(q), static_cast<float*>(s), c.stream);
    });
}

// (dev, stream, x, offsets, codes, scales)
PyObject* quantize_tokens(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args c;
    int64_t M, cols, G = 1;
    if (!c.open(args, n, 6) || !c.matrix(2, "x", &M, &cols)) return nullptr;
    if (!c.none(3)) {
        const at::Tensor* t = c.tensor(3, "offsets");
        if (t == nullptr) return nullptr;
        G = t->numel() - 1;
    }
    if (!Args::fits_int({M, cols, G})) return PyLong_FromLong(MOE_ERR_UNSUPPORTED);
    const int64_t R = moe_fp8_token_rows((int32_t)M, (int32_t)G);
    const void* x = c.data(2, "x", {M, cols}, Args::bf16, "bfloat16 or uint16");
    const int32_t* offsets = c.none(3) ? nullptr : c.ints_n(3, "offsets", G + 1);
    uint8_t* q = c.written(4, c.e4m3(4, "codes", {cols, R}));
    float* s = c.written(5, c.floats(5, "scales", {R / 128, cols}));
    if (!c.ok) return nullptr;
    return c.status([&] {
        return moe_quantize_fp8_tokens(static_cast<const uint16_t*>(x), offsets, (int32_t)G, (int32_t)M,
                                       (int32_t)cols, q, s, c.stream);
    });
}

// (dev, stream, dy codes, dy scales, x codes, x scales, offsets, M, dw, accumulate, ws)
PyObject* wgrad(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args c;
    int64_t G, N, K;
    size_t bytes = 0;
    if (!c.open(args, n, 11) || !weight_shape(c, 8, "dw", !c.none(6), &G, &N, &K)) return nullptr;
    const int64_t M = c.integer(7);
    if (!c.ok) return nullptr;
    if (!Args::fits_int({G, M, N, K})) return PyLong_FromLong(M < 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
    const int64_t R = moe_fp8_token_rows((int32_t)M, (int32_t)G);
    const uint8_t* dy = c.e4m3(2, "dy codes", {N, R});
    const float* dys = c.floats(3, "dy scales", {R / 128, N});
    const uint8_t* x = c.e4m3(4, "x codes", {K, R});
    const float* xs = c.floats(5, "x scales", {R / 128, K});
    const int32_t* offsets = c.none(6) ? nullptr : c.ints_n(6, "offsets", G + 1);
    float* dw = c.written(8, c.floats_n(8, "dw", G * N * K));
    const int accumulate = PyObject_IsTrue(args[9]);
    void* ws = c.workspace(10, &bytes);
    if (!c.ok || accumulate < 0) return nullptr;
    return c.status([&] {
        return moe_gemm_fp8_wgrad(dy, dys, x, xs, offsets, (int32_t)G, (int32_t)M, (int32_t)N, (int32_t)K, dw,
                                  accumulate, ws, bytes, c.stream);
    });
}

// No C++ exception leaves an entry (a tensor without plain storage throws in its
// accessors).
using Entry = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
template <Entry F>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    try {
        return F(self, args, n);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
}

template <Entry F>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<F>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<balance_loss>("balance_loss"),
                         method<route_backward>("route_backward"),
                         method<product<false>>("gemm_fp8"),
                         method<product<true>>("gemm_fp8_dgrad"),
                         method<quantize_act>("quantize_act_fp8"),
                         method<quantize_tokens>("quantize_fp8_tokens"),
                         method<wgrad>("gemm_fp8_wgrad"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__moe_binding() { return PyModule_Create(&module); }
