// Python module _calls: the ordinary calls of rms_norm, swiglu, grouped_gemm and
// gemm_f8, for single tokens, whose kernels take less time than Python's
// checks.  A call is made from here where every argument is as its wrapper
// documents it, dense tensors on the current device and no stream named;
// anything else returns None, and the wrapper goes on to say what is wrong or
// to make the call its own way.  So each function here checks what its wrapper
// checks, and never raises for an argument.
//
// One call with new outputs after another, by Python's checks and from here
// (3.6 to 4 us of it the library's call itself): rms_norm of 1 x 4096 with a
// residual 11.3 and 6.0 us, swiglu 9.1 and 5.2, gemm_f8 of 4 x 64 x 64 8.4 and
// 4.6.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "tdi8.h"

namespace {

struct Entries {
    decltype(&rmsnorm_quant_s8) norm_s8;
    decltype(&rmsnorm_quant_f8) norm_f8;
    decltype(&swiglu_quant_s8) act_s8;
    decltype(&swiglu_quant_f8) act_f8;
    decltype(&gemm_s8s8_grouped) grouped;
    decltype(&gemm_f8f8_block128) product_f8;
} entries;
PyObject *error_class;  // raised with a status

constexpr int64_t kBlock = 128;
using at::ScalarType;

// The library's number of a floating type, or -1.
int type_of(ScalarType t) {
    return t == ScalarType::Float ? TDI8_F32 : t == ScalarType::BFloat16 ? TDI8_BF16
                                           : t == ScalarType::Half       ? TDI8_F16
                                                                         : -1;
}

// A dense tensor on GPU `device` whose memory holds its values (no lazy
// negation), or null.
const at::Tensor *tensor(PyObject *o, int64_t device) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device || t.layout() != at::kStrided || t.is_neg())
        return nullptr;
    return &t;
}

// The leading dimension of a matrix with unit column stride, or -1.
int64_t matrix(const at::Tensor &t, ScalarType type, int64_t rows, int64_t cols) {
    if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols) return -1;
    if (cols > 1 && t.stride(1) != 1) return -1;
    if (rows <= 1) return cols > 1 ? cols : 1;
    return t.stride(0) < cols ? -1 : t.stride(0);
}
bool vector(const at::Tensor &t, ScalarType type, int64_t count) {
    return t.scalar_type() == type && t.dim() == 1 && t.size(0) == count && (count <= 1 || t.stride(0) == 1);
}
template <class... V>
bool fit(V... v) {
    return ((v <= INT_MAX) && ...);
}

// An argument that may be None: whether it is given; `ok` turns false where it
// is no such tensor.
bool optional(PyObject *o, int64_t device, const at::Tensor *&t, bool &ok) {
    t = o == Py_None ? nullptr : tensor(o, device);
    ok = ok && (t || o == Py_None);
    return t != nullptr;
}

// Whether a call may write the caller's tensor: not where autograd would take
// it for what it was.
bool writable(const at::Tensor &t) { return !t.requires_grad() || !at::GradMode::is_enabled(); }

struct Output {
    at::Tensor made;          // a new one
    PyObject *given = nullptr;
    void *data = nullptr;
    int64_t ld = 1;

    // The caller's, already checked.
    void take(PyObject *o, const at::Tensor &t, int64_t stride) {
        given = o;
        data = t.data_ptr();
        ld = stride;
    }
    void make(at::IntArrayRef shape, const at::Tensor &like, ScalarType type) {
        made = at::empty(shape, like.options().dtype(type));
        data = made.data_ptr();
        ld = shape.back() > 1 ? shape.back() : 1;
    }
    // The result.  The caller's tensor counts as written, for backward passes
    // that kept it.
    PyObject *object() {
        if (!given) return THPVariable_Wrap(std::move(made));
        const at::Tensor &t = THPVariable_Unpack(given);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
        Py_INCREF(given);
        return given;
    }
};

// out and scale of an 8-bit result of T x H: 1 made or taken, 0 not as documented.
bool eight_bit_out(bool f8, int64_t T, int64_t H, const at::Tensor &like, PyObject *out, PyObject *scale,
                   int64_t device, Output &q, Output &s) {
    const ScalarType type = f8 ? ScalarType::Float8_e4m3fn : ScalarType::Char;
    const int64_t blocks = (H + kBlock - 1) / kBlock;
    bool ok = true;
    const at::Tensor *tq, *ts;
    if (optional(out, device, tq, ok)) {
        const int64_t ld = matrix(*tq, type, T, H);
        if (ld < 0 || !writable(*tq)) return false;
        q.take(out, *tq, ld);
    }
    if (optional(scale, device, ts, ok)) {
        const int64_t ld = f8 ? matrix(*ts, ScalarType::Float, T, blocks) : 1;
        if (ld < 0 || (!f8 && !vector(*ts, ScalarType::Float, T)) || !writable(*ts)) return false;
        s.take(scale, *ts, ld);
    }
    if (!ok) return false;
    if (!tq) q.make({T, H}, like, type);
    if (!ts) {
        if (f8)
            s.make({T, blocks}, like, ScalarType::Float);
        else
            s.make({T}, like, ScalarType::Float);
    }
    return true;
}

// 0 for "s8", 1 for "f8", else -1.
int format_of(PyObject *o) {
    if (!PyUnicode_Check(o)) return -1;
    if (PyUnicode_CompareWithASCIIString(o, "s8") == 0) return 0;
    return PyUnicode_CompareWithASCIIString(o, "f8") == 0 ? 1 : -1;
}

struct Where {
    int64_t device;
    hipStream_t stream;
};
bool where(PyObject *device, PyObject *stream, Where &w) {
    w.device = PyLong_AsLongLong(device);
    w.stream = static_cast<hipStream_t>(PyLong_AsVoidPtr(stream));
    if (!PyErr_Occurred()) return true;
    PyErr_Clear();
    return false;
}

bool failed(int status) {
    if (status == TDI8_OK) return false;
    PyObject *number = PyLong_FromLong(status);
    if (number) PyErr_SetObject(error_class, number);
    Py_XDECREF(number);
    return true;
}

PyObject *pack(Output *first, int count) {
    PyObject *all = PyTuple_New(count);
    if (!all) return nullptr;
    for (int i = 0; i < count; ++i) {
        PyObject *o = first[i].object();
        if (!o) {
            Py_DECREF(all);
            return nullptr;
        }
        PyTuple_SET_ITEM(all, i, o);
    }
    return all;
}

// (x, weight, eps, residual, fmt, sum_out, out, scale, device, stream)
PyObject *rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    if (n != 10 || !where(a[8], a[9], w)) Py_RETURN_NONE;
    const at::Tensor *x = tensor(a[0], w.device), *weight = tensor(a[1], w.device), *residual, *given_sum;
    const int fmt = format_of(a[4]);
    bool ok = x && weight && fmt >= 0 && PyFloat_CheckExact(a[2]);
    const bool adds = optional(a[3], w.device, residual, ok);
    const bool in_place = optional(a[5], w.device, given_sum, ok);
    if (!ok || (in_place && !adds) || x->dim() != 2) Py_RETURN_NONE;
    const ScalarType dtype = x->scalar_type();
    const int type = type_of(dtype);
    const int64_t T = x->size(0), H = x->size(1);
    const int64_t ldx = matrix(*x, dtype, T, H), ldr = adds ? matrix(*residual, dtype, T, H) : 0;
    if (type < 0 || ldx < 0 || ldr < 0 || !vector(*weight, dtype, H)) Py_RETURN_NONE;
    Output o[3];  // q, scale, sum
    if (in_place) {
        const int64_t ld = matrix(*given_sum, dtype, T, H);
        if (ld < 0 || !writable(*given_sum)) Py_RETURN_NONE;
        o[2].take(a[5], *given_sum, ld);
    }
    if (!eight_bit_out(fmt == 1, T, H, *x, a[6], a[7], w.device, o[0], o[1])) Py_RETURN_NONE;
    if (adds && !in_place) o[2].make({T, H}, *x, dtype);
    if (!fit(T, H, ldx, ldr, o[0].ld, o[1].ld, o[2].ld)) Py_RETURN_NONE;
    const void *px = x->data_ptr(), *pr = adds ? residual->data_ptr() : nullptr, *pw = weight->data_ptr();
    const float eps = static_cast<float>(PyFloat_AS_DOUBLE(a[2]));
    const int ldsum = adds ? static_cast<int>(o[2].ld) : 0;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = fmt == 0
                 ? entries.norm_s8(type, T, H, px, ldx, pr, ldr, pw, eps, o[2].data, ldsum,
                                   static_cast<int8_t *>(o[0].data), o[0].ld, static_cast<float *>(o[1].data), w.stream)
                 : entries.norm_f8(type, T, H, px, ldx, pr, ldr, pw, eps, o[2].data, ldsum,
                                   static_cast<uint8_t *>(o[0].data), o[0].ld, static_cast<float *>(o[1].data),
                                   o[1].ld, w.stream);
    Py_END_ALLOW_THREADS
    return failed(status) ? nullptr : pack(o, adds ? 3 : 2);
    END_HANDLE_TH_ERRORS
}

// (gate, up, fmt, out, scale, device, stream)
PyObject *swiglu(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    if (n != 7 || !where(a[5], a[6], w)) Py_RETURN_NONE;
    const at::Tensor *gate = tensor(a[0], w.device), *up = tensor(a[1], w.device);
    const int fmt = format_of(a[2]);
    if (!gate || !up || fmt < 0 || gate->dim() != 2) Py_RETURN_NONE;
    const ScalarType dtype = gate->scalar_type();
    const int type = type_of(dtype);
    const int64_t T = gate->size(0), N = gate->size(1);
    const int64_t ldg = matrix(*gate, dtype, T, N), ldu = matrix(*up, dtype, T, N);
    Output o[2];
    if (type < 0 || ldg < 0 || ldu < 0 || !eight_bit_out(fmt == 1, T, N, *gate, a[3], a[4], w.device, o[0], o[1]) ||
        !fit(T, N, ldg, ldu, o[0].ld, o[1].ld))
        Py_RETURN_NONE;
    const void *pg = gate->data_ptr(), *pu = up->data_ptr();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = fmt == 0 ? entries.act_s8(type, T, N, pg, ldg, pu, ldu, static_cast<int8_t *>(o[0].data), o[0].ld,
                                       static_cast<float *>(o[1].data), w.stream)
                      : entries.act_f8(type, T, N, pg, ldg, pu, ldu, static_cast<uint8_t *>(o[0].data), o[0].ld,
                                       static_cast<float *>(o[1].data), o[1].ld, w.stream);
    Py_END_ALLOW_THREADS
    return failed(status) ? nullptr : pack(o, 2);
    END_HANDLE_TH_ERRORS
}

// The result of a product: the caller's or a new one of `dtype`; its type, or -1.
int product_out(PyObject *out, PyObject *dtype, int64_t M, int64_t N, const at::Tensor &like, int64_t device,
                Output &c) {
    bool ok = true;
    const at::Tensor *given;
    if (optional(out, device, given, ok)) {
        const int type = type_of(given->scalar_type());
        const int64_t ld = matrix(*given, given->scalar_type(), M, N);
        if (type < 0 || ld < 0 || !writable(*given)) return -1;
        c.take(out, *given, ld);
        return type;
    }
    if (!ok || !THPDtype_Check(dtype)) return -1;
    const ScalarType made = reinterpret_cast<THPDtype *>(dtype)->scalar_type;
    const int type = type_of(made);
    if (type >= 0) c.make({M, N}, like, made);
    return type;
}

// (A, a_scale, B, b_scale, offsets, rows, out, dtype, device, stream)
PyObject *grouped_gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    if (n != 10 || !where(a[8], a[9], w)) Py_RETURN_NONE;
    const at::Tensor *A = tensor(a[0], w.device), *sa = tensor(a[1], w.device), *B = tensor(a[2], w.device),
                     *sb = tensor(a[3], w.device), *offsets, *rows;
    bool ok = A && sa && B && sb;
    optional(a[4], w.device, offsets, ok);
    optional(a[5], w.device, rows, ok);
    if (!ok || A->dim() != 2 || B->scalar_type() != ScalarType::Char) Py_RETURN_NONE;
    const int64_t T = A->size(0), K = A->size(1), lda = matrix(*A, ScalarType::Char, T, K);
    const int one = B->dim() == 2 ? 1 : 0;  // (N, K): one group
    if (lda < 0 || B->dim() + one != 3 || B->size(2 - one) != K || (K > 1 && B->stride(2 - one) != 1)) Py_RETURN_NONE;
    const int64_t G = one ? 1 : B->size(0), N = B->size(1 - one);
    if (sb->scalar_type() != ScalarType::Float || sb->dim() + one != 2 || (!one && sb->size(0) != G) ||
        sb->size(1 - one) != N || !sb->is_contiguous() || !vector(*sa, ScalarType::Float, T))
        Py_RETURN_NONE;
    if (offsets ? !vector(*offsets, ScalarType::Int, G + 1) : G != 1) Py_RETURN_NONE;
    const int64_t M = rows ? rows->numel() : T;
    if (rows && !vector(*rows, ScalarType::Int, M)) Py_RETURN_NONE;
    const int64_t ldb = N > 1 ? B->stride(1 - one) : K > 1 ? K : 1, group_b = G > 1 ? B->stride(0) : 0;
    // (operands that the library refuses for how they lie, which Python puts into words)
    if (M > 0 && (T == 0 || ldb < K || (G > 1 && group_b < (N - 1) * ldb + K))) Py_RETURN_NONE;
    Output c;
    const int type = product_out(a[6], a[7], M, N, *A, w.device, c);
    if (type < 0 || !fit(G, M, N, K, lda, T, ldb, c.ld)) Py_RETURN_NONE;
    const int8_t *pa = static_cast<const int8_t *>(A->data_ptr()), *pb = static_cast<const int8_t *>(B->data_ptr());
    const float *psa = static_cast<const float *>(sa->data_ptr()), *psb = static_cast<const float *>(sb->data_ptr());
    const int32_t *prows = rows ? static_cast<const int32_t *>(rows->data_ptr()) : nullptr;
    const int32_t *poffsets = offsets ? static_cast<const int32_t *>(offsets->data_ptr()) : nullptr;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = entries.grouped(type, G, M, N, K, pa, lda, T, psa, prows, poffsets, pb, ldb, group_b, psb, c.data, c.ld,
                             w.stream);
    Py_END_ALLOW_THREADS
    return failed(status) ? nullptr : c.object();
    END_HANDLE_TH_ERRORS
}

// (A, a_scale, B, b_scale, out, dtype, device, stream)
PyObject *gemm_f8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    if (n != 8 || !where(a[6], a[7], w)) Py_RETURN_NONE;
    const at::Tensor *A = tensor(a[0], w.device), *sa = tensor(a[1], w.device), *B = tensor(a[2], w.device),
                     *sb = tensor(a[3], w.device);
    if (!A || !sa || !B || !sb || A->dim() != 2 || B->dim() != 2) Py_RETURN_NONE;
    const int64_t M = A->size(0), K = A->size(1), N = B->size(0);
    const int64_t kb = (K + kBlock - 1) / kBlock, nb = (N + kBlock - 1) / kBlock;
    const int64_t lda = matrix(*A, ScalarType::Float8_e4m3fn, M, K), ldb = matrix(*B, ScalarType::Float8_e4m3fn, N, K);
    const int64_t ldas = matrix(*sa, ScalarType::Float, M, kb), ldbs = matrix(*sb, ScalarType::Float, nb, kb);
    if (lda < 0 || ldb < 0 || ldas < 0 || ldbs < 0) Py_RETURN_NONE;
    Output c;
    const int type = product_out(a[4], a[5], M, N, *A, w.device, c);
    if (type < 0 || !fit(M, N, K, lda, ldas, ldb, ldbs, c.ld)) Py_RETURN_NONE;
    const uint8_t *pa = static_cast<const uint8_t *>(A->data_ptr()), *pb = static_cast<const uint8_t *>(B->data_ptr());
    const float *psa = static_cast<const float *>(sa->data_ptr()), *psb = static_cast<const float *>(sb->data_ptr());
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = entries.product_f8(type, M, N, K, pa, lda, psa, ldas, pb, ldb, psb, ldbs, c.data, c.ld, w.stream);
    Py_END_ALLOW_THREADS
    return failed(status) ? nullptr : c.object();
    END_HANDLE_TH_ERRORS
}

// (error class, addresses of the library's entry points in the order of Entries)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[6];
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "bind takes an exception class and six addresses");
        return nullptr;
    }
    for (int i = 0; i < 6; ++i) p[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (PyErr_Occurred()) return nullptr;
    entries = {reinterpret_cast<decltype(Entries::norm_s8)>(p[0]), reinterpret_cast<decltype(Entries::norm_f8)>(p[1]),
               reinterpret_cast<decltype(Entries::act_s8)>(p[2]),  reinterpret_cast<decltype(Entries::act_f8)>(p[3]),
               reinterpret_cast<decltype(Entries::grouped)>(p[4]),
               reinterpret_cast<decltype(Entries::product_f8)>(p[5])};
    Py_INCREF(a[0]);
    Py_XDECREF(error_class);
    error_class = a[0];
    Py_RETURN_NONE;
}

#define TDI8_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TDI8_METHOD(rms_norm), TDI8_METHOD(swiglu), TDI8_METHOD(grouped_gemm), TDI8_METHOD(gemm_f8),
                         TDI8_METHOD(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers it was built against.  Another's
// tensors may be laid out otherwise, so the package then leaves it alone.
PyMODINIT_FUNC PyInit__calls() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TDI8_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
