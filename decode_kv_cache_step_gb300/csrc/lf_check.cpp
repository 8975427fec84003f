// Argument checks of the Python binding in one call: what takes the interpreter
// half a microsecond per tensor (dtype, shape, device, layout, address) takes some
// 30 ns here. The binding works without this module; it is only faster with it.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

bool fits(const at::Tensor& t, PyObject* dtype, PyObject* shape) {
    if (!t.defined() || !t.is_cuda() || !THPDtype_Check(dtype) || !PyTuple_Check(shape)) return false;
    if (t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type) return false;
    if (PyTuple_GET_SIZE(shape) != t.dim()) return false;
    for (int64_t i = 0; i < t.dim(); ++i) {
        PyObject* n = PyTuple_GET_ITEM(shape, i);
        if (!PyLong_Check(n)) return false;
        const long long want = PyLong_AsLongLong(n);
        if (want == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
        if (want != t.size(i)) return false;
    }
    return t.is_contiguous();
}

// pointers(tensor, name, dtype, shape, ...): the data pointers of the tensors (None
// for None) if each is a contiguous CUDA tensor of its dtype and shape and all are
// on one device, else None. (The names are for the caller's own messages.)
PyObject* pointers(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n % 4 != 0) {
        PyErr_SetString(PyExc_TypeError, "pointers: four arguments per tensor");
        return nullptr;
    }
    PyObject* out = PyTuple_New(n / 4);
    if (!out) return nullptr;
    int device = -1;
    bool good = true;
    for (Py_ssize_t i = 0; good && i < n / 4; ++i) {
        PyObject* o = args[4 * i];
        PyObject* pointer = nullptr;
        if (o == Py_None) {
            Py_INCREF(Py_None);
            pointer = Py_None;
        } else if (THPVariable_Check(o)) {
            try {
                const at::Tensor& t = THPVariable_Unpack(o);
                if (fits(t, args[4 * i + 2], args[4 * i + 3]) && (device < 0 || device == t.get_device())) {
                    device = static_cast<int>(t.get_device());
                    pointer = PyLong_FromVoidPtr(t.data_ptr());
                }
            } catch (...) {  // tensors without a layout or an address
            }
        }
        if (pointer)
            PyTuple_SET_ITEM(out, i, pointer);
        else
            good = false;
    }
    if (good) return out;
    Py_DECREF(out);
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"pointers", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pointers)), METH_FASTCALL,
     "Data pointers of checked tensors, or None."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lf_check", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (The torch whose headers this was compiled against: the binding uses it with no
// other.)
PyMODINIT_FUNC PyInit__lf_check() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", LF_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
