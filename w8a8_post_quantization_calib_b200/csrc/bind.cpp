// bind.cpp -- the calls of the 4-bit formats and of the key/value cache for
// PyTorch tensors (module _sqbind): checks tensors, takes the current stream
// and calls the C ABI.  Written natively because these calls are made once a
// layer and token in a decode step: with the checks in Python a cache write
// took 12 us of the host's time, of which the launch is 4.
//
// Positional arguments only; the Python functions of the package give them
// names and defaults.  Every function returns None or raises: TypeError (not a
// CUDA tensor, wrong type), ValueError (shape, device, contiguity), and, through
// the package's SQError, any status that the C ABI returns.  A tensor that is
// not on a GPU, and an operand of the wrong type beside another one, raise an
// error that is both: the package's other calls raise TypeError there, these
// raised ValueError before.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/headeronly/version.h>

#include <string>

#include "sq.h"

namespace {

PyObject *g_error = nullptr;       // SQError(function, status)
PyObject *g_kind_error = nullptr;  // TypeError and ValueError

struct Raised {};                  // a Python exception is set

[[noreturn]] void raise(PyObject *type, const std::string &msg)
{
    PyErr_SetString(type, msg.c_str());
    throw Raised();
}

std::string shape_of(const at::Tensor &t)
{
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

// The arguments of one call: tensors have to be on the current device.
class Call {
public:
    Call(const char *name, PyObject *const *args, Py_ssize_t given, Py_ssize_t want)
        : name_(name), args_(args)
    {
        if (given != want) raise(PyExc_TypeError, std::string(name) + " takes " + std::to_string(want) + " arguments");
    }

    bool none(int i) const { return args_[i] == Py_None; }

    const at::Tensor &tensor(int i, const char *what) const
    {
        if (!THPVariable_Check(args_[i])) raise(PyExc_TypeError, std::string(what) + " must be a CUDA tensor");
        const at::Tensor &t = THPVariable_Unpack(args_[i]);
        if (!t.is_cuda()) raise(g_kind_error, std::string(what) + " must be a CUDA tensor, got one on " + t.device().str());
        if (t.device().index() != device())
            raise(PyExc_ValueError, std::string("every tensor must be on the current device cuda:") + std::to_string(device()) + ", got " +
                                        what + " on " + t.device().str());
        return t;
    }

    // tensor of a type
    const at::Tensor &typed(int i, const char *what, at::ScalarType type) const
    {
        const at::Tensor &t = tensor(i, what);
        if (t.scalar_type() != type)
            raise(g_kind_error, std::string(what) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
        return t;
    }

    // contiguous tensor of a type
    const at::Tensor &dense(int i, const char *what, at::ScalarType type) const
    {
        const at::Tensor &t = tensor(i, what);
        if (t.scalar_type() != type) raise(PyExc_TypeError, std::string(what) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
        if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(what) + " must be contiguous");
        return t;
    }

    // pointer of an optional fp32 vector of n elements
    const float *floats(int i, int64_t n, const char *what) const
    {
        if (none(i)) return nullptr;
        const at::Tensor &t = dense(i, what, at::kFloat);
        if (t.numel() != n) raise(PyExc_ValueError, std::string(what) + " must hold " + std::to_string(n) + " elements, got " + std::to_string(t.numel()));
        return static_cast<const float *>(t.data_ptr());
    }

    int64_t integer(int i) const
    {
        const long long v = PyLong_AsLongLong(args_[i]);
        if (v == -1 && PyErr_Occurred()) throw Raised();
        return v;
    }

    double number(int i) const
    {
        const double v = PyFloat_AsDouble(args_[i]);
        if (v == -1.0 && PyErr_Occurred()) throw Raised();
        return v;
    }

    // the current stream (None), an object with cuda_stream, or its address
    sq_stream stream(int i) const
    {
        if (none(i)) return c10::cuda::getCurrentCUDAStream(device()).stream();
        PyObject *o = args_[i];
        PyObject *attr = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : Py_NewRef(o);
        void *p = attr != nullptr ? PyLong_AsVoidPtr(attr) : nullptr;
        Py_XDECREF(attr);
        if (PyErr_Occurred()) throw Raised();
        return p;
    }

    // Calls f(args...) without the interpreter's lock (a launch can wait for
    // room in the stream's queue); returns None or raises its status.
    template <typename F, typename... Args> PyObject *call(F f, Args... args) const
    {
        PyThreadState *state = PyEval_SaveThread();
        const sq_status st = f(args...);
        PyEval_RestoreThread(state);
        if (st == SQ_OK) Py_RETURN_NONE;
        if (g_error == nullptr) raise(PyExc_RuntimeError, std::string(name_) + " returned status " + std::to_string(st));
        PyObject *e = PyObject_CallFunction(g_error, "si", name_, static_cast<int>(st));
        if (e != nullptr) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        throw Raised();
    }

private:
    int device() const
    {
        if (dev_ < 0) dev_ = c10::cuda::current_device();
        return dev_;
    }

    const char *name_;
    PyObject *const *args_;
    mutable int dev_ = -1;
};

sq_dtype dtype_of(const at::Tensor &t)
{
    switch (t.scalar_type()) {
    case at::kFloat: return SQ_F32;
    case at::kHalf: return SQ_F16;
    case at::kBFloat16: return SQ_BF16;
    default: raise(PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
    }
}

sq_fp4_format fp4_format(int64_t v)
{
    if (v != SQ_MXFP4 && v != SQ_NVFP4) raise(PyExc_ValueError, "format must be MXFP4 or NVFP4");
    return static_cast<sq_fp4_format>(v);
}

sq_kv_format kv_format(int64_t v)
{
    if (v != SQ_KV_INT8 && v != SQ_KV_FP8 && v != SQ_KV_MXFP4) raise(PyExc_ValueError, "format must be KV_INT8, KV_FP8 or KV_MXFP4");
    return static_cast<sq_kv_format>(v);
}

const at::Tensor &matrix(const at::Tensor &t, const char *what)
{
    if (t.dim() != 2) raise(PyExc_ValueError, std::string(what) + " must be 2-D, got " + shape_of(t));
    return t;
}

struct Operand {
    uint8_t *q, *sf;
};

// codes uint8 [rows, 16 ceil(K / 32)] and at least their scales' bytes
Operand operand(const Call &c, int i, int64_t rows, int64_t K, sq_fp4_format fmt, const char *what)
{
    const at::Tensor &q = c.dense(i, what, at::kByte), &sf = c.dense(i + 1, "scales", at::kByte);
    const int64_t row = static_cast<int64_t>(sq_fp4_code_bytes(K));
    if (q.dim() != 2 || q.size(0) != rows || q.size(1) != row)
        raise(PyExc_ValueError, std::string(what) + " must be [" + std::to_string(rows) + ", " + std::to_string(row) + "], got " + shape_of(q));
    const int64_t need = static_cast<int64_t>(sq_fp4_scale_bytes(fmt, rows, K));
    if (sf.numel() < need)
        raise(PyExc_ValueError, std::string(what) + ": the scales must hold " + std::to_string(need) + " bytes, got " + std::to_string(sf.numel()));
    return {static_cast<uint8_t *>(q.data_ptr()), static_cast<uint8_t *>(sf.data_ptr())};
}

// (act_max, w_max, alpha, s, g_act, g_w, stream)
PyObject *smooth_scales_nvfp4(const Call &c)
{
    const at::Tensor &am = c.dense(0, "act_max", at::kFloat);
    const int64_t K = am.numel();
    if (c.none(1) || c.none(3)) raise(PyExc_TypeError, "w_max and s must be CUDA tensors");
    return c.call(sq_smooth_scales_nvfp4, static_cast<const float *>(am.data_ptr()), c.floats(1, K, "w_max"), K,
                                         static_cast<float>(c.number(2)), const_cast<float *>(c.floats(3, K, "s")),
                                         const_cast<float *>(c.floats(4, 1, "g_act")),
                                         const_cast<float *>(c.floats(5, 1, "g_w")), c.stream(6));
}

// (w, s, fmt, wq4, w_sf, g, stream)
PyObject *quant_weight_fp4(const Call &c)
{
    const at::Tensor &w = matrix(c.tensor(0, "w"), "w");
    const int64_t N = w.size(0), K = w.size(1);
    const sq_dtype dt = dtype_of(w);
    if (!w.is_contiguous()) raise(PyExc_ValueError, "w must be contiguous");
    const sq_fp4_format fmt = fp4_format(c.integer(2));
    const Operand o = operand(c, 3, N, K, fmt, "weight codes");
    return c.call(sq_quant_weight_fp4, w.data_ptr(), dt, N, K, c.floats(1, K, "s"), fmt, c.floats(5, 1, "g"), o.q, o.sf, c.stream(6));
}

// (x, s, fmt, xq4, x_sf, g, stream)
PyObject *smooth_quant_act_fp4(const Call &c)
{
    const at::Tensor &x = matrix(c.tensor(0, "x"), "x");
    const int64_t M = x.size(0), K = x.size(1);
    const sq_dtype dt = dtype_of(x);
    if (K > 1 && x.stride(1) != 1) raise(PyExc_ValueError, "x rows must be contiguous");
    int64_t ld = x.stride(0);
    if (M <= 1) ld = K;
    else if (ld < K) raise(PyExc_ValueError, "x rows must not overlap");
    const sq_fp4_format fmt = fp4_format(c.integer(2));
    const Operand o = operand(c, 3, M, K, fmt, "activation codes");
    return c.call(sq_smooth_quant_act_fp4, x.data_ptr(), dt, M, K, ld, c.floats(1, K, "s"), fmt, c.floats(5, 1, "g"), o.q, o.sf, c.stream(6));
}

// (q4, sf, fmt, out, g, stream)
PyObject *dequant_fp4(const Call &c)
{
    const at::Tensor &out = matrix(c.tensor(3, "out"), "out");
    const int64_t rows = out.size(0), K = out.size(1);
    const sq_dtype dt = dtype_of(out);
    if (!out.is_contiguous()) raise(PyExc_ValueError, "out must be contiguous");
    const sq_fp4_format fmt = fp4_format(c.integer(2));
    const Operand o = operand(c, 0, rows, K, fmt, "codes");
    return c.call(sq_dequant_fp4, o.q, o.sf, fmt, rows, K, c.floats(4, 1, "g"), dt, out.data_ptr(), c.stream(5));
}

// (xq4, x_sf, wq4, w_sf, fmt, y, bias, g_act, g_w, stream)
PyObject *linear_fp4(const Call &c)
{
    const at::Tensor &y = matrix(c.tensor(5, "y"), "y"), &wq = matrix(c.tensor(2, "weight codes"), "weight codes");
    const int64_t M = y.size(0), N = y.size(1), K = 2 * wq.size(1);
    const sq_dtype dt = dtype_of(y);
    if (!y.is_contiguous()) raise(PyExc_ValueError, "y must be contiguous");
    const sq_fp4_format fmt = fp4_format(c.integer(4));
    const Operand x = operand(c, 0, M, K, fmt, "activation codes"), w = operand(c, 2, N, K, fmt, "weight codes");
    const void *bias = nullptr;
    if (!c.none(6)) {
        const at::Tensor &b = c.typed(6, "bias", y.scalar_type());
        if (b.numel() != N || !b.is_contiguous())
            raise(PyExc_ValueError, std::string("bias must be a contiguous ") + c10::toString(y.scalar_type()) + " tensor of " + std::to_string(N) + " elements");
        bias = b.data_ptr();
    }
    return c.call(sq_linear_fp4, x.q, x.sf, w.q, w.sf, fmt, M, N, K, c.floats(7, 1, "g_act"), c.floats(8, 1, "g_w"), bias, dt,
                                y.data_ptr(), c.stream(9));
}

struct Cache {
    void *p[4];                    // k codes, k scales, v codes, v scales
    int64_t pages, page_size;
};

// the four cache tensors from argument i on
Cache cache(const Call &c, int i, sq_kv_format fmt, int64_t H, int64_t D)
{
    const int64_t rb = static_cast<int64_t>(sq_kv_row_bytes(fmt, D)), sb = static_cast<int64_t>(sq_kv_scale_bytes(fmt, D));
    if (rb == 0) raise(PyExc_ValueError, "no cache rows of " + std::to_string(D) + " elements");
    static const char *const names[4] = {"k_cache", "k_scale", "v_cache", "v_scale"};
    Cache r{};
    for (int n = 0; n < 4; ++n) {
        const bool scale = n & 1;
        const at::ScalarType type = scale ? (fmt == SQ_KV_MXFP4 ? at::kByte : at::kFloat) : fmt == SQ_KV_INT8 ? at::kChar : at::kByte;
        const at::Tensor &t = c.typed(i + n, names[n], type);
        if (n == 0) {
            if (t.dim() != 4) raise(PyExc_ValueError, "k_cache must be 4-D, got " + shape_of(t));
            r.pages = t.size(0);
            r.page_size = t.size(1);
        }
        const int64_t last = !scale ? rb : fmt == SQ_KV_MXFP4 ? sb : 0;           // 0: no such dimension
        if (!t.is_contiguous() || t.dim() != (last ? 4 : 3) || t.size(0) != r.pages ||
            t.size(1) != r.page_size || t.size(2) != H || (last && t.size(3) != last))
            raise(PyExc_ValueError, std::string(names[n]) + " must be a contiguous " + c10::toString(type) + " tensor [" + std::to_string(r.pages) +
                                        ", " + std::to_string(r.page_size) + ", " + std::to_string(H) + (last ? ", " + std::to_string(last) : "") +
                                        "], got " + c10::toString(t.scalar_type()) + " " + shape_of(t));
        r.p[n] = t.data_ptr();
    }
    return r;
}

// (k, v, slots, fmt, k_cache, k_scale, v_cache, v_scale, stream)
PyObject *kv_cache_write(const Call &c)
{
    const at::Tensor &k = c.tensor(0, "k"), &v = c.tensor(1, "v");
    if (k.dim() != 3) raise(PyExc_ValueError, "k must be 3-D, got " + shape_of(k));
    if (v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type()) raise(PyExc_ValueError, "k and v must match");
    const int64_t T = k.size(0), H = k.size(1), D = k.size(2);
    const sq_dtype dt = dtype_of(k);
    int64_t ld[2];
    for (int n = 0; n < 2; ++n) {
        const at::Tensor &x = n ? v : k;
        const char *what = n ? "v" : "k";
        if ((D > 1 && x.stride(2) != 1) || (H > 1 && x.stride(1) != D))
            raise(PyExc_ValueError, std::string("the heads of a token of ") + what + " must be contiguous");
        if (T > 1 && x.stride(0) < H * D) raise(PyExc_ValueError, std::string("the tokens of ") + what + " must not overlap");
        ld[n] = T > 1 ? x.stride(0) : H * D;
    }
    const at::Tensor &slots = c.typed(2, "slots", at::kLong);
    if (slots.dim() != 1 || slots.size(0) != T || !slots.is_contiguous())
        raise(PyExc_ValueError, "slots must be a contiguous int64 tensor [" + std::to_string(T) + "]");
    const sq_kv_format fmt = kv_format(c.integer(3));
    const Cache a = cache(c, 4, fmt, H, D);
    return c.call(sq_kv_cache_write, k.data_ptr(), v.data_ptr(), dt, T, H, D, ld[0], ld[1], static_cast<const int64_t *>(slots.data_ptr()),
                                    fmt, a.pages * a.page_size, a.p[0], a.p[1], a.p[2], a.p[3], c.stream(8));
}

// (fmt, k_cache, k_scale, v_cache, v_scale, table, cu_rows, k_out, v_out, starts, stream)
PyObject *kv_cache_read(const Call &c)
{
    const at::Tensor &ko = c.tensor(7, "k_out"), &vo = c.tensor(8, "v_out");
    if (ko.dim() != 3) raise(PyExc_ValueError, "k_out must be 3-D, got " + shape_of(ko));
    if (vo.sizes() != ko.sizes() || vo.scalar_type() != ko.scalar_type()) raise(PyExc_ValueError, "k_out and v_out must match");
    if (!ko.is_contiguous() || !vo.is_contiguous()) raise(PyExc_ValueError, "k_out and v_out must be contiguous");
    const int64_t total = ko.size(0), H = ko.size(1), D = ko.size(2);
    const sq_dtype dt = dtype_of(ko);
    const sq_kv_format fmt = kv_format(c.integer(0));
    const Cache a = cache(c, 1, fmt, H, D);
    const at::Tensor &table = matrix(c.typed(5, "table", at::kInt), "table");
    const int64_t B = table.size(0), pages = table.size(1);
    auto ints = [](const at::Tensor &t, int64_t dim, int64_t n, const char *what) {
        if (!t.is_contiguous() || t.dim() != dim || t.numel() != n)
            raise(PyExc_ValueError, std::string(what) + " must be a contiguous int32 tensor of " + std::to_string(n) + " elements, got " +
                                        c10::toString(t.scalar_type()) + " " + shape_of(t));
        return static_cast<const int32_t *>(t.data_ptr());
    };
    const int32_t *tab = ints(table, 2, B * pages, "table"), *cu = ints(c.typed(6, "cu_rows", at::kInt), 1, B + 1, "cu_rows");
    const int32_t *starts = c.none(9) ? nullptr : ints(c.typed(9, "starts", at::kInt), 1, B, "starts");
    return c.call(sq_kv_cache_read, fmt, a.p[0], a.p[1], a.p[2], a.p[3], a.pages, a.page_size, H, D, tab, B, pages, cu, starts, total, dt,
                                   ko.data_ptr(), vo.data_ptr(), c.stream(10));
}

// No C++ exception leaves a call.
template <PyObject *(*F)(const Call &), int N>
PyObject *entry(const char *name, PyObject *const *args, Py_ssize_t given)
{
    try {
        return F(Call(name, args, given, N));
    } catch (const Raised &) {
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define SQ_ENTRY(fn, n) \
    PyObject *py_##fn(PyObject *, PyObject *const *args, Py_ssize_t given) { return entry<fn, n>("sq_" #fn, args, given); }
SQ_ENTRY(smooth_scales_nvfp4, 7)
SQ_ENTRY(quant_weight_fp4, 7)
SQ_ENTRY(smooth_quant_act_fp4, 7)
SQ_ENTRY(dequant_fp4, 6)
SQ_ENTRY(linear_fp4, 10)
SQ_ENTRY(kv_cache_write, 9)
SQ_ENTRY(kv_cache_read, 11)
#undef SQ_ENTRY

PyObject *py_set_error(PyObject *, PyObject *cls)
{
    Py_XSETREF(g_error, Py_NewRef(cls));
    Py_RETURN_NONE;
}

#define SQ_METHOD(fn) {#fn, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##fn)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SQ_METHOD(smooth_scales_nvfp4), SQ_METHOD(quant_weight_fp4), SQ_METHOD(smooth_quant_act_fp4),
                         SQ_METHOD(dequant_fp4),         SQ_METHOD(linear_fp4),       SQ_METHOD(kv_cache_write),
                         SQ_METHOD(kv_cache_read),       {"set_error", py_set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
#undef SQ_METHOD

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sqbind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sqbind()
{
    if (g_kind_error == nullptr) {
        PyObject *bases = PyTuple_Pack(2, PyExc_TypeError, PyExc_ValueError);
        if (bases == nullptr) return nullptr;
        g_kind_error = PyErr_NewException("w8a8_post_quantization_calib_b200._sqbind.TensorKindError", bases, nullptr);
        Py_DECREF(bases);
        if (g_kind_error == nullptr) return nullptr;
    }
    PyObject *m = PyModule_Create(&module);
    if (m != nullptr && (PyModule_AddStringConstant(m, "TORCH_VERSION", TORCH_VERSION) != 0 ||
                         PyModule_AddObjectRef(m, "TensorKindError", g_kind_error) != 0))
        Py_CLEAR(m);
    return m;
}
