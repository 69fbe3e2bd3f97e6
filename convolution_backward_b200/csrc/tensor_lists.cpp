// tensor_lists.cpp -- reads lists of tensors for the Python binding: a step over hundreds of
// tensors asks every one of them for its device, type, shape, layout and address, which took the
// interpreter 0.45 us a tensor (300 tensors: 137 us, beside 42 of the norm of their 120 M elements on the GPU)
// and takes 0.02 here.  It only looks, and counts changes: nothing is allocated, launched or kept.
#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <memory>
#include <new>
#include <utility>

namespace {

template <typename T>
T* address(PyObject* v)
{
    return reinterpret_cast<T*>(PyLong_AsVoidPtr(v));
}

// F with torch's exceptions (tensors under a function transform and symbolic sizes raise them where a size or an address
// is asked for) as Python's: one that left the module would end the process.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t count)
{
    try {
        return F(self, args, count);
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry()
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<F>));
}

PyObject* fail(PyObject* type, const char* what, const char* text)
{
    PyErr_Format(type, text, what);
    return nullptr;
}

// Whether a tensor's storage holds its elements: one that was released (as sharded training does), or a fake
// tensor's, has none, and the address is that of the offset.
bool held(const at::Tensor& t)
{
    if (t.numel() == 0) return true;
    const c10::Storage& s = t.storage();
    return s.data() != nullptr && s.nbytes() >= static_cast<size_t>(t.storage_offset() + t.numel()) * t.element_size();
}

int64_t type_of(const at::Tensor& t) { return t.is_contiguous() ? static_cast<int64_t>(t.scalar_type()) : -1; }

// read(tensors, like, what, addresses, elements) -> (type, device): fills the arrays at the two
// addresses (elements may be 0) from a list of contiguous CUDA tensors of one type (0 fp32, 1 bf16, 2 f16; -1: no
// tensor) and device.  like: None, or a list of tensors of the same length whose shapes they must have;
// then an entry may be None, and its address is 0.
PyObject* read(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    if (count != 5 || !PyList_Check(args[0]) || (args[1] != Py_None && !PyList_Check(args[1]))) {
        PyErr_SetString(PyExc_TypeError, "read(tensors: list, like: list or None, what, addresses, elements)");
        return nullptr;
    }
    PyObject* const list = args[0];
    PyObject* const like = args[1] == Py_None ? nullptr : args[1];
    const char* const what = PyUnicode_AsUTF8(args[2]);
    uint64_t* const at = address<uint64_t>(args[3]);
    int64_t* const elements = address<int64_t>(args[4]);
    if (!what || PyErr_Occurred()) return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(list);
    if (like && PyList_GET_SIZE(like) != n) {
        PyErr_Format(PyExc_ValueError, "expected %zd %s, got %zd", PyList_GET_SIZE(like), what, n);
        return nullptr;
    }
    int type = -1, device = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject* const o = PyList_GET_ITEM(list, i);
        if (like && o == Py_None) {
            at[i] = 0;
            if (elements) elements[i] = 0;
            continue;
        }
        if (!THPVariable_Check(o)) return fail(PyExc_TypeError, what, "%s must be tensors");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) return fail(PyExc_ValueError, what, "%s: tensors must be CUDA tensors (no CPU path)");
        if (t.layout() != c10::kStrided || !t.is_contiguous()) return fail(PyExc_ValueError, what, "%s: tensors must be contiguous");
        const c10::ScalarType s = t.scalar_type();
        const int code = s == c10::kFloat ? 0 : s == c10::kBFloat16 ? 1 : s == c10::kHalf ? 2 : -1;
        if (code < 0) return fail(PyExc_TypeError, what, "%s: unsupported dtype; use float32, bfloat16 or float16");
        if (type >= 0 && code != type) return fail(PyExc_TypeError, what, "%s must have one dtype");
        type = code;
        const int index = static_cast<int>(t.get_device());
        if (device >= 0 && index != device) return fail(PyExc_ValueError, what, "%s: all tensors of one call must be on the same CUDA device");
        device = index;
        if (like) {
            PyObject* const l = PyList_GET_ITEM(like, i);
            if (!THPVariable_Check(l) || !t.sizes().equals(THPVariable_Unpack(l).sizes()))
                return fail(PyExc_ValueError, what, "%s must have their parameters' shapes");
        }
        if (!held(t)) return fail(PyExc_ValueError, what, "%s: a tensor's storage does not hold its elements");
        at[i] = reinterpret_cast<uint64_t>(t.const_data_ptr());
        if (elements) elements[i] = t.numel();
    }
    return Py_BuildValue("(ii)", type, device);
}

// describe(tensors, addresses, elements, types): fills the three arrays from tensors whose storages hold them; a type is
// torch's number of it, -1 where the tensor is not contiguous.
PyObject* describe(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    if (count != 4 || !PyList_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "describe(tensors: list, addresses, elements, types)");
        return nullptr;
    }
    uint64_t* const at = address<uint64_t>(args[1]);
    int64_t* const elements = address<int64_t>(args[2]);
    int64_t* const types = address<int64_t>(args[3]);
    if (PyErr_Occurred()) return nullptr;
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(args[0]); ++i) {
        PyObject* const o = PyList_GET_ITEM(args[0], i);
        if (!THPVariable_Check(o)) return fail(PyExc_TypeError, "entries", "%s must be tensors");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!held(t)) return fail(PyExc_ValueError, "parameters and states", "%s: a tensor's storage does not hold its elements");
        at[i] = reinterpret_cast<uint64_t>(t.const_data_ptr());
        elements[i] = t.numel();
        types[i] = type_of(t);
    }
    Py_RETURN_NONE;
}

// same(tensors, addresses, elements, types) -> whether every tensor of the list still is what `describe` left in the
// arrays.  An address alone is not enough: a view of a few of its elements has it too.  (A storage that is resized moves.)
PyObject* same(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    if (count != 4 || !PyList_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "same(tensors: list, addresses, elements, types)");
        return nullptr;
    }
    const uint64_t* const at = address<const uint64_t>(args[1]);
    const int64_t* const elements = address<const int64_t>(args[2]);
    const int64_t* const types = address<const int64_t>(args[3]);
    if (PyErr_Occurred()) return nullptr;
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(args[0]); ++i) {
        PyObject* const o = PyList_GET_ITEM(args[0], i);
        if (!THPVariable_Check(o)) Py_RETURN_FALSE;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (reinterpret_cast<uint64_t>(t.const_data_ptr()) != at[i] || t.numel() != elements[i] || type_of(t) != types[i]) Py_RETURN_FALSE;
    }
    Py_RETURN_TRUE;
}

// apart(addresses, elements, n, bytes, lo, hi, m) -> whether none of the n ranges of elements[i] * bytes at
// addresses[i] (0: none) shares a byte with one of the m ranges [lo[k], hi[k]), which are in order and apart.
PyObject* apart(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    if (count != 7) {
        PyErr_SetString(PyExc_TypeError, "apart(addresses, elements, n, bytes, lo, hi, m)");
        return nullptr;
    }
    const uint64_t* const at = address<const uint64_t>(args[0]);
    const int64_t* const elements = address<const int64_t>(args[1]);
    const Py_ssize_t n = PyLong_AsSsize_t(args[2]);
    const uint64_t bytes = PyLong_AsUnsignedLongLong(args[3]);
    const uint64_t* const lo = address<const uint64_t>(args[4]);
    const uint64_t* const hi = address<const uint64_t>(args[5]);
    const Py_ssize_t m = PyLong_AsSsize_t(args[6]);
    if (PyErr_Occurred()) return nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!at[i] || elements[i] <= 0) continue;
        const uint64_t* k = std::upper_bound(hi, hi + m, at[i]);      // the first range that ends behind it
        if (k != hi + m && lo[k - hi] < at[i] + static_cast<uint64_t>(elements[i]) * bytes) Py_RETURN_FALSE;
    }
    Py_RETURN_TRUE;
}

// disjoint(a, b, elements, n, bytes) -> whether the 2 n ranges of elements[i] * bytes at a[i] and b[i] share no byte.
PyObject* disjoint(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    if (count != 5) {
        PyErr_SetString(PyExc_TypeError, "disjoint(a, b, elements, n, bytes)");
        return nullptr;
    }
    const uint64_t* const list[2] = {address<const uint64_t>(args[0]), address<const uint64_t>(args[1])};
    const int64_t* const elements = address<const int64_t>(args[2]);
    const Py_ssize_t n = PyLong_AsSsize_t(args[3]);
    const uint64_t bytes = PyLong_AsUnsignedLongLong(args[4]);
    if (PyErr_Occurred()) return nullptr;
    using Range = std::pair<uint64_t, uint64_t>;
    std::unique_ptr<Range[]> r(new (std::nothrow) Range[static_cast<size_t>(2 * n) + 1]);
    if (!r) return PyErr_NoMemory();
    size_t k = 0;
    for (const uint64_t* at : list)
        for (Py_ssize_t i = 0; i < n; ++i)
            if (elements[i] > 0) r[k++] = {at[i], at[i] + static_cast<uint64_t>(elements[i]) * bytes};
    std::sort(r.get(), r.get() + k);
    for (size_t i = 1; i < k; ++i)
        if (r[i].first < r[i - 1].second) Py_RETURN_FALSE;
    Py_RETURN_TRUE;
}

// written(tensors, addresses, n): counts an in-place change of each tensor of the list but those whose addresses[i % n]
// is 0, so that a graph that has saved one of them raises when it is run backward, as after torch's own in-place
// operations.
PyObject* written(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    if (count != 3 || !PyList_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "written(tensors: list, addresses, n)");
        return nullptr;
    }
    const uint64_t* const at = address<const uint64_t>(args[1]);
    const Py_ssize_t n = PyLong_AsSsize_t(args[2]);
    if (PyErr_Occurred()) return nullptr;
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(args[0]); ++i) {
        PyObject* const o = PyList_GET_ITEM(args[0], i);
        if (!at[i % n] || !THPVariable_Check(o)) continue;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();     // inference tensors have no count
    }
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"read", entry<read>(), METH_FASTCALL, nullptr},
    {"describe", entry<describe>(), METH_FASTCALL, nullptr},
    {"same", entry<same>(), METH_FASTCALL, nullptr},
    {"written", entry<written>(), METH_FASTCALL, nullptr},
    {"disjoint", entry<disjoint>(), METH_FASTCALL, nullptr},
    {"apart", entry<apart>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the headers' torch, whose tensors are laid out as this module reads them.
PyMODINIT_FUNC PyInit__tensor_lists()
{
    PyObject* const m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
