// The 8-bit helpers' common case in C++: torch tensors in, the library's call on
// the current stream, torch tensors out.  It exists because a call's checks,
// torch.empty and argument conversions in Python take 4 to 8 us, as long as the
// smallest kernels (1 x 4096 x 4096: 7.2 us a call so, 5.5 here; a store and read
// back of one token 12.9, 10.1).
//
// Each function checks what the Python helper of its name checks and returns None
// where anything is not as that asks (or the library refuses the call): the helper
// then goes its own way, which says what is wrong.  Nothing here computes.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include "mkp.h"

namespace {

using at::Tensor;

// One operand: its address and leading dimension.
struct View {
    void* p = nullptr;
    int64_t ld = 0;
};

const Tensor* tensor_of(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A matrix (vector: cols < 0) of these extents on GPU `gpu`, its last axis contiguous.
bool view(const Tensor* t, int gpu, at::ScalarType type, int64_t rows, int64_t cols, View& v) {
    if (t == nullptr || t->scalar_type() != type || !t->is_cuda() || t->get_device() != gpu || t->layout() != at::kStrided)
        return false;
    if (cols < 0) {
        if (t->dim() != 1 || t->size(0) != rows || (rows > 1 && t->stride(0) != 1)) return false;
        v.ld = 1;
    } else {
        if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols || (cols > 1 && t->stride(1) != 1)) return false;
        v.ld = rows > 1 ? t->stride(0) : cols;
    }
    v.p = t->data_ptr();
    return true;
}

// A quantised matrix's scales: a vector (group 0), or a matrix of them.
bool scales(const Tensor* t, int gpu, int64_t rows, int64_t cols, int64_t group, View& v) {
    if (group == 0) return view(t, gpu, at::kFloat, rows, -1, v);
    return view(t, gpu, at::kFloat, rows, (cols + group - 1) / group, v);
}

bool known_group(int64_t g) { return g == 0 || g == 32 || g == 64 || g == 128 || g == 256; }

// bf16 and binary32 by the library's codes.
bool real_code(const Tensor& t, int& code) {
    code = t.scalar_type() == at::kFloat ? MKP_F32 : MKP_BF16;
    return t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16;
}
at::ScalarType type_of(int64_t code) { return code == MKP_F32 ? at::kFloat : at::kBFloat16; }

// The GPU that t is on, if it is the current one; else -1.
int current_gpu(const Tensor* t, int64_t dims) {
    if (t == nullptr || !t->is_cuda() || t->dim() != dims) return -1;
    const int gpu = t->get_device();
    return gpu == c10::hip::current_device() ? gpu : -1;
}
void* stream_of(int gpu) { return (void*)c10::hip::getCurrentHIPStream(gpu).stream(); }

Tensor make(const Tensor& like, at::IntArrayRef size, at::ScalarType type) {
    return at::empty(size, at::TensorOptions().dtype(type).device(like.device()));
}

bool integer(PyObject* o, int64_t& v) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    v = x;
    return true;
}

// (x, group) -> (q, scale)
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t group;
    int code;
    View x;
    if (n != 2 || !integer(a[1], group) || !known_group(group)) Py_RETURN_NONE;
    const Tensor* t = tensor_of(a[0]);
    const int gpu = current_gpu(t, 2);
    if (gpu < 0 || !real_code(*t, code)) Py_RETURN_NONE;
    const int64_t M = t->size(0), K = t->size(1), groups = group ? (K + group - 1) / group : 1, ldq = (K + 15) / 16 * 16;
    if (K == 0 || !view(t, gpu, t->scalar_type(), M, K, x)) Py_RETURN_NONE;   // (no columns: the helper's own way)
    Tensor q = make(*t, {M, ldq}, at::kChar);
    Tensor s = group ? make(*t, {M, groups}, at::kFloat) : make(*t, {M}, at::kFloat);
    if (mkp_quantize_rows(M, K, x.p, x.ld, code, group, (int8_t*)q.data_ptr(), ldq, (float*)s.data_ptr(), groups > 0 ? groups : 1,
                          stream_of(gpu)) != MKP_OK)
        Py_RETURN_NONE;
    if (ldq != K) q = q.narrow(1, 0, K);
    PyObject* out = PyTuple_New(2);
    if (out == nullptr) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(q));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(s));
    return out;
    END_HANDLE_TH_ERRORS
}

// (q, scale, group, type code) -> y
PyObject* dequantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t group, code;
    View q, s;
    if (n != 4 || !integer(a[2], group) || !known_group(group) || !integer(a[3], code)) Py_RETURN_NONE;
    if (code != MKP_F32 && code != MKP_BF16) Py_RETURN_NONE;
    const Tensor* t = tensor_of(a[0]);
    const int gpu = current_gpu(t, 2);
    if (gpu < 0) Py_RETURN_NONE;
    const int64_t M = t->size(0), K = t->size(1);
    if (!view(t, gpu, at::kChar, M, K, q) || !scales(tensor_of(a[1]), gpu, M, K, group, s)) Py_RETURN_NONE;
    Tensor y = make(*t, {M, K}, type_of(code));
    if (mkp_dequantize_rows(M, K, (const int8_t*)q.p, q.ld, (const float*)s.p, s.ld, group, y.data_ptr(), K, (int)code,
                            stream_of(gpu)) != MKP_OK)
        Py_RETURN_NONE;
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// (x, w, w_scale, bias or None, activation code, x_scale or None, type code) -> y
PyObject* linear_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t act, code, bytes = 0;
    int x_code = MKP_I8;
    View x, w, ws, xs, b;
    if (n != 7 || !integer(a[4], act) || !integer(a[6], code)) Py_RETURN_NONE;
    if (code != MKP_F32 && code != MKP_BF16) Py_RETURN_NONE;
    const Tensor *t = tensor_of(a[0]), *wt = tensor_of(a[1]);
    const int gpu = current_gpu(t, 2);
    if (gpu < 0 || wt == nullptr || wt->dim() != 2) Py_RETURN_NONE;
    const int64_t M = t->size(0), K = t->size(1), N = wt->size(0);
    if (a[5] == Py_None ? !real_code(*t, x_code) : !view(tensor_of(a[5]), gpu, at::kFloat, M, -1, xs)) Py_RETURN_NONE;
    if (!view(t, gpu, a[5] == Py_None ? t->scalar_type() : at::kChar, M, K, x) || !view(wt, gpu, at::kChar, N, K, w) ||
        !view(tensor_of(a[2]), gpu, at::kFloat, N, -1, ws) || (a[3] != Py_None && !view(tensor_of(a[3]), gpu, at::kFloat, N, -1, b)))
        Py_RETURN_NONE;
    if (mkp_linear_i8_workspace(M, N, K, x.p, x.ld, x_code, (const int8_t*)w.p, w.ld, &bytes) != MKP_OK) Py_RETURN_NONE;
    Tensor y = make(*t, {M, N}, type_of(code)), work;
    if (bytes > 0) work = make(*t, {bytes}, at::kByte);
    if (mkp_linear_i8(M, N, K, x.p, x.ld, x_code, (const float*)xs.p, (const int8_t*)w.p, w.ld, (const float*)ws.p,
                      (const float*)b.p, (int)act, y.data_ptr(), N, (int)code, bytes > 0 ? work.data_ptr() : nullptr, bytes,
                      stream_of(gpu)) != MKP_OK)
        Py_RETURN_NONE;
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// (dy, x, x_scale, z, z_scale, z_group, activation code, need_dz, need_dw, need_dbias, type code) -> (dz, dw, dbias)
PyObject* linear_q8_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t group, act, need[3], code, bytes = 0;
    int dy_code;
    View dy, x, xs, z, zs;
    zs.ld = 1;
    if (n != 11 || !integer(a[5], group) || !integer(a[6], act) || !integer(a[10], code)) Py_RETURN_NONE;
    for (int i = 0; i < 3; ++i)
        if (!integer(a[7 + i], need[i])) Py_RETURN_NONE;
    if (code != MKP_F32 && code != MKP_BF16) Py_RETURN_NONE;
    const Tensor *t = tensor_of(a[0]), *xt = tensor_of(a[1]);
    const int gpu = current_gpu(t, 2);
    if (gpu < 0 || xt == nullptr || xt->dim() != 2 || !real_code(*t, dy_code)) Py_RETURN_NONE;
    const int64_t M = t->size(0), N = t->size(1), K = xt->size(1);
    if (!view(t, gpu, t->scalar_type(), M, N, dy) || !view(xt, gpu, at::kChar, M, K, x) ||
        !view(tensor_of(a[2]), gpu, at::kFloat, M, -1, xs))
        Py_RETURN_NONE;
    if (act == MKP_ACT_NONE) group = 0;
    else if (!known_group(group) || !view(tensor_of(a[3]), gpu, at::kChar, M, N, z) || !scales(tensor_of(a[4]), gpu, M, N, group, zs))
        Py_RETURN_NONE;
    if (mkp_linear_q8_backward_workspace(M, N, K, need[1] != 0, need[2] != 0, &bytes) != MKP_OK) Py_RETURN_NONE;
    Tensor dz, dw, db, work;
    if (need[0]) dz = make(*t, {M, N}, at::kBFloat16);
    if (need[1]) dw = make(*t, {N, K}, type_of(code));
    if (need[2]) db = make(*t, {N}, at::kFloat);
    if (bytes > 0) work = make(*t, {bytes}, at::kByte);
    auto at_of = [](const Tensor& v) { return v.defined() ? v.data_ptr() : nullptr; };
    if (mkp_linear_q8_backward(M, N, K, dy.p, dy.ld, dy_code, (const int8_t*)x.p, x.ld, (const float*)xs.p, (const int8_t*)z.p, z.ld,
                               (const float*)zs.p, zs.ld, group, (int)act, at_of(dz), N, at_of(dw), K, (int)code,
                               (float*)at_of(db), at_of(work), bytes, stream_of(gpu)) != MKP_OK)
        Py_RETURN_NONE;
    PyObject* out = PyTuple_New(3);
    if (out == nullptr) return nullptr;
    const Tensor* all[3] = {&dz, &dw, &db};
    for (int i = 0; i < 3; ++i) {
        PyObject* o = Py_None;
        if (all[i]->defined()) o = THPVariable_Wrap(*all[i]);
        else Py_INCREF(o);
        PyTuple_SET_ITEM(out, i, o);
    }
    return out;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"quantize_rows", (PyCFunction)(void (*)(void))quantize_rows, METH_FASTCALL, "quantize_rows"},
    {"dequantize_rows", (PyCFunction)(void (*)(void))dequantize_rows, METH_FASTCALL, "dequantize_rows"},
    {"linear_i8", (PyCFunction)(void (*)(void))linear_i8, METH_FASTCALL, "linear_i8"},
    {"linear_q8_backward", (PyCFunction)(void (*)(void))linear_q8_backward, METH_FASTCALL, "linear_q8_backward"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mkptorch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mkptorch(void) { return PyModule_Create(&module); }
