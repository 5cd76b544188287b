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

// What adamw_step takes of each parameter: the layout of nvfp4_block.h's adamw_tensor.
struct AdamWTensor {
    void *param, *grad, *m, *v, *m_scale, *v_scale, *master;
    int64_t size;
    int32_t type, bits;
};

// A parameter's own tensors in the order of AdamWState, after the parameter and its gradient.
const char *const FIELDS[] = {"param", "grad", "m", "v", "m_scale", "v_scale", "master"};

// adamw(params, grads, states) -> (device index, adamw_tensor[] as bytes, the tensors that the step
// writes).  states holds tuples (m, v[, m_scale, v_scale[, master]]), None for what there is not.
// ValueError where a tensor does not fit its parameter.
PyObject *adamw(PyObject *, PyObject *args)
{
    PyObject *params, *grads, *states;
    if (!PyArg_ParseTuple(args, "O!O!O!", &PyList_Type, &params, &PyList_Type, &grads,
                          &PyList_Type, &states))
        return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(params);
    if (PyList_GET_SIZE(grads) != n || PyList_GET_SIZE(states) != n)
        return PyErr_Format(PyExc_ValueError,
                            "params, grads and states must be of one length; got %zd, %zd and %zd",
                            n, PyList_GET_SIZE(grads), PyList_GET_SIZE(states));
    PyObject *written = nullptr;
    try {
        std::vector<AdamWTensor> out(n);
        int device = -1;
        written = PyList_New(0);
        if (!written) return nullptr;
        const auto refuse = [&](PyObject *) {
            Py_DECREF(written);
            return nullptr;
        };
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject *state = PyList_GET_ITEM(states, i);
            if (!PyTuple_Check(state) || PyTuple_GET_SIZE(state) < 2 || PyTuple_GET_SIZE(state) > 5)
                return refuse(PyErr_Format(PyExc_ValueError, "states[%zd] must be a tuple (m, v"
                                           "[, m_scale, v_scale[, master]]); got %s", i,
                                           Py_TYPE(state)->tp_name));
            PyObject *given[7] = {PyList_GET_ITEM(params, i), PyList_GET_ITEM(grads, i)};
            for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(state); ++k)
                given[2 + k] = PyTuple_GET_ITEM(state, k);
            void *at[7] = {};
            int64_t numel = 0, blocks = 0;
            at::ScalarType type = at::kFloat;
            bool coded = false;
            for (int k = 0; k < 7; ++k) {
                const char *name = FIELDS[k];
                if (!given[k] || given[k] == Py_None) {
                    if (k < 4 || (coded && k < 6))
                        return refuse(PyErr_Format(PyExc_ValueError, "%s of parameter %zd is "
                                                   "missing", name, i));
                    continue;
                }
                if (!THPVariable_Check(given[k]))
                    return refuse(PyErr_Format(PyExc_ValueError, "%s of parameter %zd must be a "
                                               "torch tensor; got %s", name, i,
                                               Py_TYPE(given[k])->tp_name));
                const at::Tensor &t = THPVariable_Unpack(given[k]);
                if (!t.is_cuda() || (device >= 0 && t.get_device() != device))
                    return refuse(PyErr_Format(PyExc_ValueError, "params, grads and states must be "
                                               "on one GPU; got %s", t.device().str().c_str()));
                device = (int)t.get_device();
                if (t.layout() != at::kStrided || !t.is_contiguous())
                    return refuse(PyErr_Format(PyExc_ValueError, "%s of parameter %zd must be "
                                               "contiguous", name, i));
                bool fits = true;
                if (k == 0) {
                    if (const char *other = kind(t, &out[i].type))
                        return refuse(PyErr_Format(PyExc_ValueError, "params must be float32, "
                                                   "bfloat16 or float16; got %s", other));
                    type = t.scalar_type();
                    numel = t.numel();
                    blocks = (numel + 127) / 128;
                } else if (k == 1) {
                    fits = t.scalar_type() == type && t.numel() == numel;
                } else if (k == 2 || k == 3) {
                    if (k == 2) coded = t.scalar_type() == at::kByte;
                    fits = coded ? t.scalar_type() == at::kByte && t.dim() == 2 &&
                                       t.size(0) == blocks && t.size(1) == 128
                                 : t.scalar_type() == at::kFloat && t.numel() == numel;
                } else if (k < 6) {
                    fits = coded && t.scalar_type() == at::kByte && t.numel() == blocks;
                } else {
                    fits = type != at::kFloat && t.scalar_type() == at::kFloat &&
                           t.numel() == numel;
                }
                if (!fits)
                    return refuse(PyErr_Format(
                        PyExc_ValueError, "%s of parameter %zd, %s of %lld elements, does not fit "
                        "%lld elements of %s%s", name, i, c10::toString(t.scalar_type()),
                        (long long)t.numel(), (long long)numel, c10::toString(type),
                        coded ? " with moments in 8 bits" : ""));
                at[k] = t.data_ptr();
                if (k != 1 && PyList_Append(written, given[k]) < 0) return refuse(nullptr);
            }
            out[i] = {at[0], at[1], at[2], at[3], at[4], at[5], at[6], numel, out[i].type,
                      coded ? 8 : 32};
        }
        return Py_BuildValue("iNN", device, bytes_of(out), written);
    } catch (const std::exception &e) {
        Py_XDECREF(written);
        return PyErr_Format(PyExc_ValueError, "params, grads or states hold a tensor without memory "
                            "of its own: %s", e.what());
    }
}

PyMethodDef methods[] = {{"adamw", adamw, METH_VARARGS, "what an AdamW step takes of each parameter"},
                         {"table", table, METH_VARARGS, "addresses, sizes and types of tensors"},
                         {"written", written, METH_O, "counts a version of each tensor"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
