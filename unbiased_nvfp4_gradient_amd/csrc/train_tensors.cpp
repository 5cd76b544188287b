// train_tensors.cpp -- reads the addresses, sizes and types of a list of torch tensors for the C
// ABI's arrays, and counts a version of those that a call wrote.  Gradient clipping takes hundreds of tensors a call, and attribute by attribute
// from Python they cost more than the kernels: clipping 300 tensors into 300 others took 244 us a
// call, 40 us with the lists read here.
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <vector>

namespace {

const char *kind(const at::Tensor &t, int32_t *type)
{
    switch (t.scalar_type()) {
    case at::kFloat: *type = 0; return nullptr;          // NVFP4_F32
    case at::kBFloat16: *type = 1; return nullptr;       // NVFP4_BF16
    case at::kHalf: *type = 2; return nullptr;           // NVFP4_F16
    default: return c10::toString(t.scalar_type());
    }
}

template <typename X> PyObject *bytes_of(const std::vector<X> &v)
{
    return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(v.data()),
                                     (Py_ssize_t)(v.size() * sizeof(X)));
}

// table(tensors, name) -> (device index, addresses, sizes, types), the last three as bytes of
// void *, int64_t and int32_t.  ValueError where an entry is no contiguous floating tensor of
// one GPU; `name` is the list's in the message.
PyObject *table(PyObject *, PyObject *args)
{
    PyObject *list;
    const char *name;
    if (!PyArg_ParseTuple(args, "O!s", &PyList_Type, &list, &name)) return nullptr;
    try {
        const Py_ssize_t n = PyList_GET_SIZE(list);
        std::vector<void *> at(n);
        std::vector<int64_t> sizes(n);
        std::vector<int32_t> types(n);
        int device = -1;
        for (Py_ssize_t i = 0; i < n; ++i)
            if (PyObject *o = PyList_GET_ITEM(list, i); !THPVariable_Check(o))
                return PyErr_Format(PyExc_ValueError, "%s must hold torch tensors; got %s", name,
                                    Py_TYPE(o)->tp_name);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const at::Tensor &t = THPVariable_Unpack(PyList_GET_ITEM(list, i));
            if (!t.is_cuda() || (i && t.get_device() != device))
                return PyErr_Format(PyExc_ValueError, "%s must be on one GPU; got %s", name,
                                    t.device().str().c_str());
            device = (int)t.get_device();
            if (t.layout() != at::kStrided || !t.is_contiguous())
                return PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
            if (const char *other = kind(t, &types[i]))
                return PyErr_Format(PyExc_ValueError,
                                    "%s must be float32, bfloat16 or float16; got %s", name, other);
            at[i] = t.data_ptr();
            sizes[i] = t.numel();
        }
        return Py_BuildValue("iNNN", device, bytes_of(at), bytes_of(sizes), bytes_of(types));
    } catch (const std::exception &e) {
        return PyErr_Format(PyExc_ValueError, "%s holds a tensor without memory of its own: %s",
                            name, e.what());
    }
}

// written(tensors): the tensors that table() took have been written through their addresses.  Each
// counts a version, as with any operation in place, so that a backward pass that saved its old
// elements is refused (tensors of inference mode count none).
PyObject *written(PyObject *, PyObject *list)
{
    if (!PyList_Check(list)) return PyErr_Format(PyExc_TypeError, "written() takes a list");
    try {
        for (Py_ssize_t i = 0; i < PyList_GET_SIZE(list); ++i) {
            PyObject *o = PyList_GET_ITEM(list, i);
            if (!THPVariable_Check(o))
                return PyErr_Format(PyExc_TypeError, "written() takes tensors; got %s",
                                    Py_TYPE(o)->tp_name);
            const at::Tensor &t = THPVariable_Unpack(o);
            if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
        }
    } catch (const std::exception &e) {
        return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
    }
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"table", table, METH_VARARGS, "addresses, sizes and types of tensors"},
                         {"written", written, METH_O, "counts a version of each tensor"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
