// marshal.cpp -- tensors as the C ABI's arguments, for the Python binding's calls whose kernels run no
// longer than the interpreter takes to read types, sizes, addresses and devices one attribute at a time
// (an AdamW step's 63 tensors 90 us; a small cross entropy 9 of the call's 16).  Every function returns
// None for whatever is not the plain case (a gap between rows, a wrong type, size or device, nothing
// to compute, anything that is no tensor); the binding then goes through its own checks, which name
// what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/VirtualGuardImpl.h>
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

// The addresses that a call of the cross entropy passes on, and its sizes.
struct Head {
    int device = -1;
    int64_t M = 0, N = 0, K = 0, x = 0, w = 0, b = 0, target = 0;
    at::ScalarType type = at::kHalf;

    // p: the address of n contiguous values of type t; None where that is allowed gives 0.
    bool vector(PyObject* o, at::ScalarType t, int64_t n, bool none, int64_t& p) {
        p = 0;
        if (o == Py_None) return none;
        if (!THPVariable_Check(o)) return false;
        const at::Tensor& v = THPVariable_Unpack(o);
        if (!plain(v, device) || v.scalar_type() != t || v.dim() != 1 || v.size(0) != n) return false;
        p = (int64_t)(uintptr_t)v.data_ptr();
        return true;
    }
    bool take(PyObject* xo, PyObject* wo, PyObject* to, PyObject* bo, bool bf16) {
        if (!THPVariable_Check(xo) || !THPVariable_Check(wo)) return false;
        const at::Tensor &xt = THPVariable_Unpack(xo), &wt = THPVariable_Unpack(wo);
        type = bf16 ? at::kBFloat16 : at::kHalf;
        if (!plain(xt, device) || !plain(wt, device) || xt.scalar_type() != type || wt.scalar_type() != type) return false;
        // (the library launches on the current device)
        if (c10::impl::VirtualGuardImpl(at::kCUDA).getDevice().index() != device) return false;
        if (xt.dim() != 2 || wt.dim() != 2 || xt.size(1) != wt.size(1) || xt.numel() == 0 || wt.numel() == 0) return false;
        M = xt.size(0);
        N = wt.size(0);
        K = xt.size(1);
        x = (int64_t)(uintptr_t)xt.data_ptr();
        w = (int64_t)(uintptr_t)wt.data_ptr();
        return vector(to, at::kLong, M, false, target) && vector(bo, type, N, true, b);
    }
    at::Tensor make(at::IntArrayRef sizes, at::ScalarType t) const {
        return at::empty(sizes, at::TensorOptions().dtype(t).device(at::kCUDA, (c10::DeviceIndex)device));
    }
};

int64_t address(const at::Tensor& t) { return t.defined() ? (int64_t)(uintptr_t)t.data_ptr() : 0; }
PyObject* wrapped(const at::Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

// cross_entropy(x, weight, target, b or None, bfloat16): (device, M, N, K, loss, lse, the C call's
// arguments up to M), with new tensors loss and lse.
PyObject* cross_entropy(PyObject* const* args, Py_ssize_t nargs) {
    Head h;
    if (nargs != 5 || !h.take(args[0], args[1], args[2], args[3], args[4] == Py_True)) Py_RETURN_NONE;
    const at::Tensor loss = h.make({h.M}, at::kFloat), lse = h.make({h.M}, at::kFloat);
    return Py_BuildValue("(iLLLNN(LLLLLLLL))", h.device, (long long)h.M, (long long)h.N, (long long)h.K, wrapped(loss), wrapped(lse),
                         (long long)h.x, (long long)h.K, (long long)h.w, (long long)h.K, (long long)h.b, (long long)h.target,
                         (long long)address(loss), (long long)address(lse));
}

// cross_entropy_backward(dloss, x, weight, target, lse, b or None, dlse or None, dx wanted, dw wanted, db
// wanted, bfloat16, FP32 dw and db): (device, M, N, K, dx, dw, db, the C call's arguments up to db).
PyObject* cross_entropy_backward(PyObject* const* args, Py_ssize_t nargs) {
    Head h;
    int64_t dloss, lse, dlse;
    if (nargs != 12 || !h.take(args[1], args[2], args[3], args[5], args[10] == Py_True)) Py_RETURN_NONE;
    if (!h.vector(args[0], at::kFloat, h.M, false, dloss) || !h.vector(args[4], at::kFloat, h.M, false, lse) ||
        !h.vector(args[6], at::kFloat, h.M, true, dlse))
        Py_RETURN_NONE;
    const at::ScalarType out = args[11] == Py_True ? at::kFloat : h.type;
    at::Tensor dx, dw, db;
    if (args[7] == Py_True) dx = h.make({h.M, h.K}, h.type);
    if (args[8] == Py_True) dw = h.make({h.N, h.K}, out);
    if (args[9] == Py_True) db = h.make({h.N}, out);
    return Py_BuildValue("(iLLLNNN(LLLLLLLLLLLLLL))", h.device, (long long)h.M, (long long)h.N, (long long)h.K, wrapped(dx),
                         wrapped(dw), wrapped(db), (long long)dloss, (long long)dlse, (long long)h.x, (long long)h.K,
                         (long long)h.w, (long long)h.K, (long long)h.b, (long long)h.target, (long long)lse,
                         (long long)address(dx), (long long)h.K, (long long)address(dw), (long long)h.K, (long long)address(db));
}

// scratch(bytes, device): a new uint8 tensor there, and its address.
PyObject* scratch(PyObject* const* args, Py_ssize_t nargs) {
    Head h;
    if (nargs != 2) Py_RETURN_NONE;
    const long long n = PyLong_AsLongLong(args[0]), device = PyLong_AsLongLong(args[1]);
    if (PyErr_Occurred()) return nullptr;
    h.device = (int)device;
    const at::Tensor t = h.make({(int64_t)n}, at::kByte);
    return Py_BuildValue("(NL)", wrapped(t), (long long)address(t));
}

PyMethodDef kMethods[] = {
    {"cross_entropy", (PyCFunction)(void (*)(void))guarded<cross_entropy>, METH_FASTCALL, nullptr},
    {"cross_entropy_backward", (PyCFunction)(void (*)(void))guarded<cross_entropy_backward>, METH_FASTCALL, nullptr},
    {"scratch", (PyCFunction)(void (*)(void))guarded<scratch>, METH_FASTCALL, nullptr},
    {"adamw", (PyCFunction)(void (*)(void))guarded<adamw>, METH_FASTCALL, nullptr},
    {"states", (PyCFunction)(void (*)(void))guarded<states>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
