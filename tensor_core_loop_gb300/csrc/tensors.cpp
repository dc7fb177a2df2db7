// Python module `_tensors`: what a call over many PyTorch tensors needs of them, read in one call.
//
// A model's gradients are dozens to hundreds of tensors. From Python each question to one of them (type, contiguous,
// address, length, device) costs some 75 ns: 62 gradients and as many results took 50 us of a call whose kernels
// take 12. Here the five cost some 10 ns together.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

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

PyMethodDef methods[] = {{"look", look, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
