// Python module `_tensors`: the binding's short ways to PyTorch's tensors.
//
// look() reads what a call over many tensors needs of them. A model's gradients are dozens to hundreds; from Python each
// question to one of them (type, contiguous, address, length, device) costs some 75 ns: 62 gradients and as many
// results took 50 us of a call whose kernels take 12. Here the five cost some 10 ns together.
//
// The calls on matrices do what dense.py does with a call on the current stream whose operands are all in order: check
// them, allocate the results and a workspace, call the library. Anything else gets None, and dense.py does it or says
// what is wrong. Small ones take 7 to 8 us of the host's time instead of 20, gradients 15 instead of 30, 62 tensors
// clipped 14 instead of 27 (Python's checks and allocations and the driver's launches push one another out of the
// host's caches).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <exception>
#include <vector>

#include "tcl_dense.h"

namespace {

// look(tensors, name): (addresses, lengths, types, device) of a list of contiguous bf16 and fp32 tensors. The first three
// are bytes: uint64, int64 and int32 (TCL_OUT_F32 0, TCL_OUT_BF16 1) for each. device: the GPU's index, -1 for
// tensors that are not on one, -2 where they are not all on the same one.
PyObject* look(PyObject*, PyObject* args) {
    PyObject *list, *name;
    if (!PyArg_ParseTuple(args, "O!U", &PyList_Type, &list, &name)) return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(list);
    PyObject* const addresses = PyBytes_FromStringAndSize(nullptr, 8 * n);
    PyObject* const lengths = PyBytes_FromStringAndSize(nullptr, 8 * n);
    PyObject* const types = PyBytes_FromStringAndSize(nullptr, 4 * n);
    int device = -1;
    bool ok = addresses && lengths && types;
    try {
        for (Py_ssize_t i = 0; ok && i < n; ++i) {
            PyObject* const item = PyList_GET_ITEM(list, i);
            if (!THPVariable_Check(item)) {
                PyErr_Format(PyExc_TypeError, "%U must be tensors, not %s", name, Py_TYPE(item)->tp_name);
                ok = false;
                break;
            }
            const at::Tensor& t = THPVariable_Unpack(item);
            const at::ScalarType type = t.scalar_type();
            if (type != at::kFloat && type != at::kBFloat16) {
                PyErr_Format(PyExc_TypeError, "%U must be bfloat16 or float32, not %s", name, c10::toString(type));
                ok = false;
            } else if (!t.is_contiguous()) {
                PyErr_Format(PyExc_ValueError, "%U must be contiguous", name);
                ok = false;
            } else {
                reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(addresses))[i] = reinterpret_cast<uintptr_t>(t.const_data_ptr());
                reinterpret_cast<int64_t*>(PyBytes_AS_STRING(lengths))[i] = t.numel();
                reinterpret_cast<int32_t*>(PyBytes_AS_STRING(types))[i] = type == at::kBFloat16;
                const int on = t.is_cuda() ? t.get_device() : -1;
                device = i == 0 || on == device ? on : -2;
            }
        }
    } catch (const std::exception& e) {   // (a tensor without memory, a sparse one)
        PyErr_Format(PyExc_ValueError, "%U: %s", name, e.what());
        ok = false;
    }
    if (ok) return Py_BuildValue("(NNNi)", addresses, lengths, types, device);
    Py_XDECREF(addresses);
    Py_XDECREF(lengths);
    Py_XDECREF(types);
    return nullptr;
}

// The library's entries, by bind(gated_ffn, gated_ffn_grad, cross_entropy, cross_entropy_grad, clip_gradients).
struct {
    decltype(&tcl_gated_ffn) ffn;
    decltype(&tcl_gated_ffn_grad) ffn_grad;
    decltype(&tcl_cross_entropy) entropy;
    decltype(&tcl_cross_entropy_grad) entropy_grad;
    decltype(&tcl_clip_gradients) clip;
} lib;

PyObject* bind(PyObject*, PyObject* args) {
    unsigned long long a[5];
    if (!PyArg_ParseTuple(args, "KKKKK", &a[0], &a[1], &a[2], &a[3], &a[4])) return nullptr;
    lib = {reinterpret_cast<decltype(lib.ffn)>(a[0]), reinterpret_cast<decltype(lib.ffn_grad)>(a[1]),
           reinterpret_cast<decltype(lib.entropy)>(a[2]), reinterpret_cast<decltype(lib.entropy_grad)>(a[3]),
           reinterpret_cast<decltype(lib.clip)>(a[4])};
    Py_RETURN_NONE;
}

// A bf16 matrix with contiguous rows on the current GPU.
struct Mat {
    const at::Tensor* t;
    void* p;
    int rows, cols, ld;
};

struct Call {
    int device = -1;
    bool ok = true;

    const at::Tensor* tensor(PyObject* o) {
        if (!ok || !THPVariable_Check(o)) return fail();
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) return fail();
        if (device < 0) device = c10::cuda::current_device();
        return t.get_device() == device ? &t : fail();
    }
    Mat mat(PyObject* o) {
        Mat m = {};
        const at::Tensor* t = tensor(o);
        if (!t || t->scalar_type() != at::kBFloat16 || t->dim() != 2) {
            ok = false;
            return m;
        }
        const int64_t rows = t->size(0), cols = t->size(1), ld = rows > 1 ? t->stride(0) : (cols + 15) / 16 * 16;
        ok = cols >= 1 && (cols == 1 || t->stride(1) == 1) && ld >= cols && ld <= INT_MAX && rows <= INT_MAX;
        if (ok) m = {t, t->data_ptr(), static_cast<int>(rows), static_cast<int>(cols), static_cast<int>(ld)};
        return m;
    }
    // A contiguous vector of n values of a type (or of another one).
    const at::Tensor* vector(PyObject* o, int64_t n, at::ScalarType type, at::ScalarType other) {
        const at::Tensor* t = tensor(o);
        if (!t || (t->scalar_type() != type && t->scalar_type() != other) || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
            return fail();
        return t;
    }
    cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

  private:
    const at::Tensor* fail() {
        ok = false;
        return nullptr;
    }
};

at::Tensor empty(at::IntArrayRef size, const at::Tensor& like, at::ScalarType type) { return at::empty(size, like.options().dtype(type)); }

// f(workspace, its size) with `room` bytes, and once more with a larger one where it asks for that: its status.
template <class F>
int with_room(size_t room, const at::Tensor& like, F f) {
    at::Tensor space;
    size_t size = room;
    for (int again = 0;; ++again) {
        if (size) space = empty({static_cast<int64_t>(size)}, like, at::kByte);
        void* const p = size ? space.data_ptr() : nullptr;
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = f(p, &size);
        Py_END_ALLOW_THREADS
        if (st != TCL_ERR_WORKSPACE || again) return st;
    }
}

// gated_ffn(x, w_gate, w_up, w_down, act, keep): (out, kept values or None), a status, or None
PyObject* gated_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 6) Py_RETURN_NONE;
    Call c;
    const Mat x = c.mat(a[0]), g = c.mat(a[1]), u = c.mat(a[2]), d = c.mat(a[3]);
    const long act = PyLong_AsLong(a[4]);
    const bool keep = a[5] == Py_True;
    if (act < 0 && PyErr_Occurred()) return nullptr;
    if (!c.ok || act < 0 || (!keep && a[5] != Py_False) || g.cols != x.cols || u.cols != x.cols || u.rows != g.rows || d.rows != x.cols ||
        d.cols != g.rows)
        Py_RETURN_NONE;
    const int64_t pitch = (static_cast<int64_t>(g.rows) + 63) / 64 * 64;   // (rows on whole lines of 128 bytes)
    if (pitch > INT_MAX) Py_RETURN_NONE;
    const at::Tensor mid = empty({keep ? 3 : 1, x.rows, pitch}, *x.t, at::kBFloat16);
    const at::Tensor out = empty({x.rows, x.cols}, *x.t, at::kBFloat16);
    char* const h = static_cast<char*>(mid.data_ptr());
    const int64_t part = 2 * pitch * x.rows;
    const cudaStream_t stream = c.stream();
    const int st = with_room(0, out, [&](void* space, size_t* size) {
        return lib.ffn(x.rows, x.cols, g.rows, x.p, x.ld, g.p, g.ld, u.p, u.ld, d.p, d.ld, static_cast<int>(act), keep ? h + part : nullptr,
                       keep ? h + 2 * part : nullptr, h, static_cast<int>(pitch), out.data_ptr(), x.cols, space, size, stream);
    });
    if (st) return PyLong_FromLong(st);
    if (!keep) return THPVariable_Wrap(out);
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(mid));
    END_HANDLE_TH_ERRORS
}

// cross_entropy(x, w, targets): (loss, lse), a status, or None
PyObject* cross_entropy(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 3) Py_RETURN_NONE;
    Call c;
    const Mat x = c.mat(a[0]), w = c.mat(a[1]);
    const at::Tensor* y = c.vector(a[2], x.rows, at::kLong, at::kInt);
    if (!c.ok || w.cols != x.cols || w.rows < 1) Py_RETURN_NONE;
    const at::Tensor loss = empty({x.rows}, *x.t, at::kFloat), lse = empty({x.rows}, *x.t, at::kFloat);
    // (what operands on 16-byte pieces take: sums for each token and 64 words, for few tokens each warp of the GPU)
    const size_t words = (static_cast<size_t>(w.rows) + 63) / 64;
    const size_t room = x.rows * (8 * std::max<size_t>(words, x.rows <= 128 ? 1024 : 0) + 4) + 512;
    const cudaStream_t stream = c.stream();
    const int st = with_room(room, loss, [&](void* space, size_t* size) {
        return lib.entropy(x.rows, x.cols, w.rows, x.p, x.ld, w.p, w.ld, y->data_ptr(), static_cast<int>(y->element_size()),
                           static_cast<float*>(loss.data_ptr()), static_cast<float*>(lse.data_ptr()), space, size, stream);
    });
    if (st) return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", THPVariable_Wrap(loss), THPVariable_Wrap(lse));
    END_HANDLE_TH_ERRORS
}

// The weights' gradients' type: TCL_OUT_F32, TCL_OUT_BF16, or another number.
bool w_type(PyObject* o, int* code, at::ScalarType* type) {
    const long v = PyLong_AsLong(o);
    *code = static_cast<int>(v);
    *type = v == TCL_OUT_F32 ? at::kFloat : at::kBFloat16;
    return v == TCL_OUT_F32 || v == TCL_OUT_BF16;
}

// gated_ffn_grad(grad, x, w_gate, w_up, w_down, kept values, inner, act, w_type): (dx, dw_gate, dw_up, dw_down), a status, or None
PyObject* gated_ffn_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) Py_RETURN_NONE;
    Call c;
    const Mat gr = c.mat(a[0]), x = c.mat(a[1]), g = c.mat(a[2]), u = c.mat(a[3]), d = c.mat(a[4]);
    const at::Tensor* kept = c.tensor(a[5]);
    if (!c.ok || !PyLong_Check(a[6])) Py_RETURN_NONE;
    const long inner = PyLong_AsLong(a[6]), act = PyLong_AsLong(a[7]);
    int code;
    at::ScalarType type;
    const bool typed = w_type(a[8], &code, &type);
    if (PyErr_Occurred()) return nullptr;
    if (!typed || act < 0 || inner != g.rows || g.cols != x.cols || u.cols != x.cols || u.rows != g.rows || d.rows != x.cols ||
        d.cols != g.rows || gr.rows != x.rows || gr.cols != x.cols || kept->scalar_type() != at::kBFloat16 || kept->dim() != 3 ||
        kept->size(0) != 3 || kept->size(1) != x.rows || kept->size(2) < g.rows || kept->size(2) % 8 || kept->size(2) > INT_MAX ||
        !kept->is_contiguous() || reinterpret_cast<uintptr_t>(kept->data_ptr()) % 16)
        Py_RETURN_NONE;
    const int64_t pitch = kept->size(2), part = 2 * pitch * x.rows;
    const at::Tensor dx = empty({x.rows, x.cols}, *x.t, at::kBFloat16), dg = empty({g.rows, g.cols}, *x.t, type),
                     du = empty({g.rows, g.cols}, *x.t, type), dd = empty({d.rows, d.cols}, *x.t, type);
    const char* const h = static_cast<const char*>(kept->data_ptr());
    const size_t room = 2 * ((2 * static_cast<size_t>(x.rows) * ((g.rows + 63) / 64 * 64) + 255) / 256 * 256);   // (what most sizes take)
    const cudaStream_t stream = c.stream();
    const int st = with_room(room, dx, [&](void* space, size_t* size) {
        return lib.ffn_grad(x.rows, x.cols, g.rows, gr.p, gr.ld, x.p, x.ld, g.p, g.ld, u.p, u.ld, d.p, d.ld, static_cast<int>(act),
                            h + part, h + 2 * part, h, static_cast<int>(pitch), dx.data_ptr(), x.cols, dg.data_ptr(), x.cols,
                            du.data_ptr(), x.cols, dd.data_ptr(), g.rows, code, space, size, stream);
    });
    if (st) return PyLong_FromLong(st);
    return Py_BuildValue("(NNNN)", THPVariable_Wrap(dx), THPVariable_Wrap(dg), THPVariable_Wrap(du), THPVariable_Wrap(dd));
    END_HANDLE_TH_ERRORS
}

// cross_entropy_grad(x, w, targets, grad, w_type): (loss, lse, dx, dw), a status, or None
PyObject* cross_entropy_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5) Py_RETURN_NONE;
    Call c;
    const Mat x = c.mat(a[0]), w = c.mat(a[1]);
    const at::Tensor* y = c.vector(a[2], x.rows, at::kLong, at::kInt);
    const at::Tensor* gr = c.vector(a[3], x.rows, at::kFloat, at::kFloat);
    int code;
    at::ScalarType type;
    const bool typed = w_type(a[4], &code, &type);
    if (PyErr_Occurred()) return nullptr;
    if (!c.ok || !typed || w.cols != x.cols || w.rows < 1) Py_RETURN_NONE;
    const at::Tensor loss = empty({x.rows}, *x.t, at::kFloat), lse = empty({x.rows}, *x.t, at::kFloat),
                     dx = empty({x.rows, x.cols}, *x.t, at::kBFloat16), dw = empty({w.rows, w.cols}, *x.t, type);
    // (what most sizes take: exponentials, scaled rows of x, sums for each 64 words and two more values a token)
    const size_t words = (static_cast<size_t>(w.rows) + 63) / 64, tokens = x.rows;
    const size_t room = tokens && tokens * words <= 1u << 24 ? tokens * (136 * words + 128 * ((static_cast<size_t>(x.cols) + 63) / 64) + 8) + 1280 : 0;
    const cudaStream_t stream = c.stream();
    const int st = with_room(room, loss, [&](void* space, size_t* size) {
        return lib.entropy_grad(x.rows, x.cols, w.rows, x.p, x.ld, w.p, w.ld, y->data_ptr(), static_cast<int>(y->element_size()),
                                static_cast<const float*>(gr->data_ptr()), static_cast<float*>(loss.data_ptr()),
                                static_cast<float*>(lse.data_ptr()), dx.data_ptr(), x.cols, dw.data_ptr(), x.cols, code, space, size,
                                stream);
    });
    if (st) return PyLong_FromLong(st);
    return Py_BuildValue("(NNNN)", THPVariable_Wrap(loss), THPVariable_Wrap(lse), THPVariable_Wrap(dx), THPVariable_Wrap(dw));
    END_HANDLE_TH_ERRORS
}

// clip_grads(tensors, out or None, bound): the norm, a status, or None
PyObject* clip_grads(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 3 || !PyList_Check(a[0]) || (a[1] != Py_None && !PyList_Check(a[1])) || !PyFloat_Check(a[2])) Py_RETURN_NONE;
    const Py_ssize_t count = PyList_GET_SIZE(a[0]);
    if (count < 1 || count > INT_MAX || (a[1] != Py_None && PyList_GET_SIZE(a[1]) != count)) Py_RETURN_NONE;
    Call c;
    const at::Tensor* first = nullptr;
    std::vector<const void*> from(count);
    std::vector<void*> to(count);
    std::vector<long long> lengths(count);
    std::vector<int> types(count);
    for (Py_ssize_t i = 0; i < count; ++i) {
        const at::Tensor* t = c.tensor(PyList_GET_ITEM(a[0], i));
        if (!t || (t->scalar_type() != at::kFloat && t->scalar_type() != at::kBFloat16) || !t->is_contiguous()) Py_RETURN_NONE;
        first = t;
        from[i] = to[i] = t->data_ptr();
        lengths[i] = t->numel();
        types[i] = t->scalar_type() == at::kBFloat16 ? TCL_OUT_BF16 : TCL_OUT_F32;
        if (a[1] == Py_None) continue;
        const at::Tensor* o = c.tensor(PyList_GET_ITEM(a[1], i));
        if (!o || o->scalar_type() != t->scalar_type() || o->numel() != t->numel() || !o->is_contiguous()) Py_RETURN_NONE;
        to[i] = o->data_ptr();
    }
    const at::Tensor norm = empty({}, *first, at::kFloat);
    const float bound = static_cast<float>(PyFloat_AS_DOUBLE(a[2]));
    const cudaStream_t stream = c.stream();
    const size_t room = 16384 * (count / 256 + 2);   // (a sum for each block of the launches that they take)
    const int st = with_room(room, norm, [&](void* space, size_t* size) {
        return lib.clip(static_cast<int>(count), from.data(), to.data(), lengths.data(), types.data(), bound,
                        static_cast<float*>(norm.data_ptr()), space, size, stream);
    });
    if (st) return PyLong_FromLong(st);
    return THPVariable_Wrap(norm);
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef fast(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {{"look", look, METH_VARARGS, nullptr},
                         {"bind", bind, METH_VARARGS, nullptr},
                         fast<gated_ffn>("gated_ffn"),
                         fast<cross_entropy>("cross_entropy"),
                         fast<gated_ffn_grad>("gated_ffn_grad"),
                         fast<cross_entropy_grad>("cross_entropy_grad"),
                         fast<clip_grads>("clip_grads"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
