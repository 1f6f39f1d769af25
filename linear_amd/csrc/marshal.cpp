// marshal.cpp -- lists of tensors as the C ABI's tables, for the Python binding's calls over many
// tensors: reading 63 tensors' types, sizes, addresses and devices one attribute at a time takes the
// interpreter longer than the kernels run.  Every function returns None for whatever is not the plain
// case (a gap between rows, a wrong type, size or device, anything that is no tensor); the binding
// then goes through its own checks, which name what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <vector>

namespace {

struct Row {                                          // linear_tensor (include/linear_amd.h)
    int64_t data, rows, cols, ld, type;
};

// The tensors of a list, or of a tuple, without new references.
struct List {
    PyObject** items = nullptr;
    Py_ssize_t count = 0;
    bool take(PyObject* o) {
        if (!PyList_Check(o) && !PyTuple_Check(o)) return false;
        items = PySequence_Fast_ITEMS(o);
        count = PySequence_Fast_GET_SIZE(o);
        for (Py_ssize_t i = 0; i < count; ++i)
            if (!THPVariable_Check(items[i])) return false;
        return true;
    }
    const at::Tensor& operator[](Py_ssize_t i) const { return THPVariable_Unpack(items[i]); }
};

// A contiguous tensor on the GPU `device` (set by the first one).
bool plain(const at::Tensor& t, int& device) {
    if (!t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous()) return false;
    const int d = t.get_device();
    if (device < 0) device = d;
    return d == device;
}

bool row_of(const at::Tensor& t, int& device, Row& r) {
    if (!plain(t, device)) return false;
    switch (t.scalar_type()) {
        case at::kHalf: r.type = 0; break;
        case at::kBFloat16: r.type = 1; break;
        case at::kFloat: r.type = 2; break;
        default: return false;
    }
    r.data = (int64_t)(uintptr_t)t.data_ptr();
    r.rows = 1;
    r.cols = r.ld = t.numel();
    return true;
}

// One value of a moment: its address, where its type and size are those of n values.
bool state_of(const at::Tensor& t, int64_t n, bool eight, int& device, int64_t& p) {
    if (!plain(t, device) || t.scalar_type() != (eight ? at::kByte : at::kFloat)) return false;
    if (t.numel() != (eight ? n + (n + 31) / 32 : n)) return false;
    p = (int64_t)(uintptr_t)t.data_ptr();
    return true;
}

template <typename T>
PyObject* bytes_of(const std::vector<T>& v) {
    return PyBytes_FromStringAndSize((const char*)v.data(), (Py_ssize_t)(v.size() * sizeof(T)));
}

// f(args, nargs), or None where reading a tensor throws.
template <PyObject* F(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    try {
        return F(args, nargs);
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// adamw(params, grads, m, v, copies or None): (params, grads, copies or None, m, v, 8-bit moments, device).
PyObject* adamw(PyObject* const* args, Py_ssize_t nargs) {
    List p, g, m, v, c;
    const bool copies = nargs == 5 && args[4] != Py_None;
    if (nargs != 5 || !p.take(args[0]) || !g.take(args[1]) || !m.take(args[2]) || !v.take(args[3]) ||
        (copies && !c.take(args[4])))
        Py_RETURN_NONE;
    const Py_ssize_t n = p.count;
    if (n == 0 || g.count != n || m.count != n || v.count != n || (copies && c.count != n)) Py_RETURN_NONE;
    std::vector<Row> pr(n), gr(n), cr(copies ? n : 0);
    std::vector<int64_t> mp(n), vp(n);
    const bool eight = m[0].scalar_type() == at::kByte;
    int device = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!row_of(p[i], device, pr[i]) || !row_of(g[i], device, gr[i]) || p[i].sizes() != g[i].sizes()) Py_RETURN_NONE;
        if (!state_of(m[i], pr[i].cols, eight, device, mp[i]) || !state_of(v[i], pr[i].cols, eight, device, vp[i])) Py_RETURN_NONE;
        if (copies && (!row_of(c[i], device, cr[i]) || p[i].sizes() != c[i].sizes())) Py_RETURN_NONE;
    }
    if (!copies) return Py_BuildValue("(NNONNii)", bytes_of(pr), bytes_of(gr), Py_None, bytes_of(mp), bytes_of(vp), (int)eight, device);
    return Py_BuildValue("(NNNNNii)", bytes_of(pr), bytes_of(gr), bytes_of(cr), bytes_of(mp), bytes_of(vp), (int)eight, device);
}

// states(out, states): (out, states, device) of 8-bit moments and the tensors they are read into.
PyObject* states(PyObject* const* args, Py_ssize_t nargs) {
    List o, s;
    if (nargs != 2 || !o.take(args[0]) || !s.take(args[1]) || o.count != s.count || o.count == 0) Py_RETURN_NONE;
    std::vector<Row> rows(o.count);
    std::vector<int64_t> p(o.count);
    int device = -1;
    for (Py_ssize_t i = 0; i < o.count; ++i)
        if (!row_of(o[i], device, rows[i]) || !state_of(s[i], rows[i].cols, true, device, p[i])) Py_RETURN_NONE;
    return Py_BuildValue("(NNi)", bytes_of(rows), bytes_of(p), device);
}

PyMethodDef kMethods[] = {
    {"adamw", (PyCFunction)(void (*)(void))guarded<adamw>, METH_FASTCALL, nullptr},
    {"states", (PyCFunction)(void (*)(void))guarded<states>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
