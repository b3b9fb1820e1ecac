// seq_binding.cpp -- the Python extension module behind sequence.py: checks the
// tensors of a call, allocates its outputs and scratch, fills the entry's
// argument struct and calls it, all in one step, because a generation step's
// kernels take 2.5 to 5 us and checking a dozen tensors from Python takes 8.
//
// An entry is described once (`entry`): the operands in the order of its struct
// in sequence_ops.h, each with a kind and its shape as indices into the call's
// sizes.  The struct is int32 words, then 8-byte fields: an activation is its
// address and two strides, any other operand an address.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <exception>
#include <string>
#include <vector>

namespace {

enum Kind {
    kAct,     // activation of the call's type: address, batch and channel strides
    kAct32,   // the same in float32
    kStates,  // B or C: address, batch stride, stride between states
    kDense,   // contiguous, of the call's type
    kDense32, // contiguous float32
    kIndex,   // contiguous int32
    kCodes,   // contiguous int8
};
enum Use { kNeeded, kOptional, kOut };

struct Operand {
    std::string name;
    int kind, use;
    std::vector<std::pair<int, int>> dims;  // (index of a size, added to it)
};

struct Entry {
    int (*call)(const void *, void *);
    int64_t (*workspace)(int32_t, int32_t, int32_t, int32_t, int32_t);
    int header;                       // sizes in the struct, after the type
    int lead;                         // the operand that has the call's type and device
    std::vector<int> workspace_sizes; // indices of the workspace function's arguments (-1: the type)
    std::vector<Operand> operands;
};

constexpr char kCapsule[] = "conv2d_backward_amd.entry";
constexpr int kMaxSizes = 16, kMaxDims = 4;

bool refuse(const char *format, const char *name, const char *more = "") {
    PyErr_Format(PyExc_ValueError, format, name, more);
    return false;
}

std::string text_of(const int64_t *shape, size_t n) {
    std::string s = "(";
    for (size_t i = 0; i < n; ++i) s += std::to_string(shape[i]) + (i + 1 < n || n == 1 ? ", " : "");
    return s + ")";
}

at::ScalarType type_of(int kind, at::ScalarType type) {
    if (kind == kAct32 || kind == kDense32) return at::kFloat;
    return kind == kIndex ? at::kInt : kind == kCodes ? at::kChar : type;
}

// Appends an operand's fields; false with a Python error set where it does not fit.
bool take(const Operand &o, const at::Tensor &t, const int64_t *shape, size_t n,
          at::ScalarType type, c10::Device device, std::vector<int64_t> &fields) {
    if (t.device() != device)
        return refuse("%s must be on %s like the other tensors", o.name.c_str(),
                      device.str().c_str());
    if (t.scalar_type() != type)
        return refuse("%s must be %s", o.name.c_str(), c10::toString(type));
    // B and C of one group may come without its axis.
    const bool ungrouped = o.kind == kStates && t.dim() == (int64_t)n - 1 && shape[1] == 1;
    bool fits = ungrouped || t.dim() == (int64_t)n;
    for (size_t i = 0, k = 0; fits && i < n; ++i) {
        if (ungrouped && i == 1) continue;
        fits = t.size(k++) == shape[i];
    }
    if (!fits) {
        const std::string more = text_of(shape, n) + ", is " + text_of(t.sizes().data(), t.dim());
        return refuse("%s must be %s", o.name.c_str(), more.c_str());
    }
    fields.push_back(reinterpret_cast<int64_t>(t.data_ptr()));
    const int64_t *stride = t.strides().data();
    switch (o.kind) {
        case kAct:
        case kAct32:
            if (n == 3 && shape[2] > 1 && stride[2] != 1)
                return refuse("%s must have contiguous positions%s", o.name.c_str());
            fields.push_back(stride[0]);
            fields.push_back(stride[1]);
            return true;
        case kStates: {
            const int at = ungrouped ? 1 : 2;
            if (n == 4 && shape[3] > 1 && stride[at + 1] != 1)
                return refuse("%s must have contiguous positions%s", o.name.c_str());
            const int64_t step = shape[2] > 1 || ungrouped ? stride[at] : stride[1];
            if (shape[1] > 1 && shape[2] > 1 && stride[1] != shape[2] * step)
                return refuse("the groups of %s must follow each other like its states%s",
                              o.name.c_str());
            fields.push_back(stride[0]);
            fields.push_back(step);
            return true;
        }
        default:
            if (!t.is_contiguous()) return refuse("%s must be contiguous%s", o.name.c_str());
            return true;
    }
}

// Sizes that the caller leaves to the operands: the first needed one that has each.
bool bind(const Entry &e, PyObject *given, int64_t *size, bool *known) {
    for (size_t i = 0; i < e.operands.size(); ++i) {
        const Operand &o = e.operands[i];
        bool all = true;
        for (const auto &d : o.dims) all = all && known[d.first];
        if (all || o.use != kNeeded) continue;
        PyObject *v = PyTuple_GET_ITEM(given, i);
        if (!THPVariable_Check(v)) return refuse("%s must be a tensor%s", o.name.c_str());
        const at::Tensor &t = THPVariable_Unpack(v);
        const int64_t n = o.dims.size();
        const bool ungrouped = o.kind == kStates && t.dim() == n - 1;
        if (!ungrouped && t.dim() != n) {
            const std::string more = std::to_string(n) + " dimensions, has " + std::to_string(t.dim());
            return refuse("%s must have %s", o.name.c_str(), more.c_str());
        }
        for (int64_t k = 0, at = 0; k < n; ++k) {
            const auto &d = o.dims[k];
            const int64_t here = ungrouped && k == 1 ? 1 : t.size(at++) - d.second;
            if (known[d.first]) continue;
            size[d.first] = here;
            known[d.first] = true;
        }
    }
    return true;
}

// call(entry, stream, sizes, operands[, code]) -> status, or the outputs in order.  A size
// that is None comes from the operands.  code: the type of the call where the leading
// operand does not have it.
// An operand is a tensor, or None: an optional one is missing, an output is
// allocated; False: an output is not wanted.
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t count) {
    if (count != 4 && count != 5) {
        PyErr_SetString(PyExc_TypeError, "call takes an entry, a stream, sizes and operands");
        return nullptr;
    }
    auto *e = static_cast<Entry *>(PyCapsule_GetPointer(args[0], kCapsule));
    if (!e) return nullptr;
    void *stream = PyLong_AsVoidPtr(args[1]);
    if (PyErr_Occurred()) return nullptr;
    PyObject *sizes = args[2], *given = args[3];
    const Py_ssize_t n_sizes = PyTuple_GET_SIZE(sizes);
    if (n_sizes > kMaxSizes || PyTuple_GET_SIZE(given) != (Py_ssize_t)e->operands.size()) {
        PyErr_SetString(PyExc_TypeError, "wrong number of sizes or operands");
        return nullptr;
    }
    try {
        PyObject *first = PyTuple_GET_ITEM(given, e->lead);
        const char *lead_name = e->operands[e->lead].name.c_str();
        if (!THPVariable_Check(first) || !THPVariable_Unpack(first).is_cuda()) {
            refuse("%s must be a tensor on a GPU device%s", lead_name);
            return nullptr;
        }
        const at::Tensor &lead = THPVariable_Unpack(first);
        const c10::Device device = lead.device();
        at::ScalarType type = lead.scalar_type();
        if (count == 5) {
            constexpr at::ScalarType kTypes[] = {at::kFloat, at::kBFloat16, at::kHalf};
            const long given_code = PyLong_AsLong(args[4]);
            if (PyErr_Occurred()) return nullptr;
            type = given_code >= 0 && given_code < 3 ? kTypes[given_code] : at::kByte;
        }
        const int code = type == at::kFloat ? 0 : type == at::kBFloat16 ? 1 : type == at::kHalf ? 2 : -1;
        if (code < 0) {
            refuse("%s must be float32, bfloat16 or float16%s", lead_name);
            return nullptr;
        }
        // The header: the type, then the first sizes (a float goes as it is stored).
        int64_t size[kMaxSizes];
        int32_t word[kMaxSizes];
        bool known[kMaxSizes], whole = true;
        for (Py_ssize_t i = 0; i < n_sizes; ++i) {
            PyObject *v = PyTuple_GET_ITEM(sizes, i);
            size[i] = word[i] = 0;
            known[i] = v != Py_None;
            whole = whole && known[i];
            if (PyFloat_Check(v)) {
                const float f = (float)PyFloat_AS_DOUBLE(v);
                std::memcpy(&word[i], &f, 4);
            } else if (known[i]) {
                size[i] = PyLong_AsLongLong(v);
                if (PyErr_Occurred()) return nullptr;
            }
        }
        if (!whole && !bind(*e, given, size, known)) return nullptr;
        std::vector<int32_t> words{code};
        words.reserve(16);
        for (Py_ssize_t i = 0; i < n_sizes; ++i) {
            if (size[i] != (int32_t)size[i]) {
                PyErr_SetString(PyExc_ValueError, "a size is beyond 32 bits");
                return nullptr;
            }
            if (size[i]) word[i] = (int32_t)size[i];
            if (i < e->header) words.push_back(word[i]);
        }
        if (words.size() % 2) words.push_back(0);
        std::vector<int64_t> fields(words.size() / 2);
        std::memcpy(fields.data(), words.data(), words.size() * 4);
        fields.reserve(64);
        std::vector<at::Tensor> made;  // outputs, an undefined one for each not wanted
        std::vector<PyObject *> passed;
        for (size_t i = 0; i < e->operands.size(); ++i) {
            const Operand &o = e->operands[i];
            PyObject *v = PyTuple_GET_ITEM(given, i);
            const size_t n = o.dims.size();
            int64_t shape[kMaxDims];
            for (size_t k = 0; k < n; ++k) shape[k] = size[o.dims[k].first] + o.dims[k].second;
            const at::ScalarType want = type_of(o.kind, type);
            const bool missing = v == Py_None ? o.use == kOptional : v == Py_False && o.use == kOut;
            if (missing) {
                fields.push_back(0);
                if (o.kind <= kStates) fields.insert(fields.end(), 2, 0);
                if (o.use == kOut) {
                    made.emplace_back();
                    passed.push_back(nullptr);
                }
                continue;
            }
            if (o.use == kOut && v == Py_None) {
                for (size_t k = 0; k < n; ++k)
                    if (shape[k] < 0) shape[k] = 0;  // sizes that the call refuses
                made.push_back(at::empty(at::IntArrayRef(shape, n), lead.options().dtype(want)));
                passed.push_back(nullptr);
                if (!take(o, made.back(), shape, n, want, device, fields)) return nullptr;
                continue;
            }
            if (!THPVariable_Check(v)) {
                refuse("%s must be a tensor%s", o.name.c_str());
                return nullptr;
            }
            const at::Tensor &t = THPVariable_Unpack(v);
            if (!take(o, t, shape, n, want, device, fields)) return nullptr;
            if (o.use == kOut) {
                made.emplace_back();
                passed.push_back(v);
            }
        }
        at::Tensor scratch;
        if (e->workspace) {
            int32_t w[5] = {0, 0, 0, 0, 0};
            for (size_t k = 0; k < e->workspace_sizes.size(); ++k)
                w[k] = e->workspace_sizes[k] < 0 ? code : (int32_t)size[e->workspace_sizes[k]];
            const int64_t bytes = e->workspace(w[0], w[1], w[2], w[3], w[4]);
            // (-1: sizes that the call itself refuses)
            if (bytes > 0) scratch = at::empty({bytes}, lead.options().dtype(at::kByte));
            fields.push_back(bytes > 0 ? reinterpret_cast<int64_t>(scratch.data_ptr()) : 0);
            fields.push_back(bytes > 0 ? bytes : 0);
        }
        const int status = e->call(fields.data(), stream);
        if (status) return PyLong_FromLong(status);
        PyObject *out = PyTuple_New(made.size());
        if (!out) return nullptr;
        for (size_t i = 0; i < made.size(); ++i) {
            PyObject *v = passed[i];
            if (v) {
                Py_INCREF(v);
            } else if (made[i].defined()) {
                v = THPVariable_Wrap(made[i]);
            } else {
                v = Py_None;
                Py_INCREF(v);
            }
            if (!v) {
                Py_DECREF(out);
                return nullptr;
            }
            PyTuple_SET_ITEM(out, i, v);
        }
        return out;
    } catch (const c10::OutOfMemoryError &err) {
        PyErr_SetString(PyExc_MemoryError, err.what_without_backtrace());
    } catch (const std::exception &err) {
        PyErr_SetString(PyExc_RuntimeError, err.what());
    }
    return nullptr;
}

// entry(address, header sizes, lead, workspace address, workspace sizes, operands),
// where an operand is (name, kind, use, ((index, added), ..)).
PyObject *entry(PyObject *, PyObject *args) {
    unsigned long long address, workspace;
    int header, lead;
    PyObject *sizes, *operands;
    if (!PyArg_ParseTuple(args, "KiiKO!O!", &address, &header, &lead, &workspace, &PyTuple_Type, &sizes,
                          &PyTuple_Type, &operands))
        return nullptr;
    auto *e = new Entry;
    e->call = reinterpret_cast<int (*)(const void *, void *)>(address);
    e->workspace =
        reinterpret_cast<int64_t (*)(int32_t, int32_t, int32_t, int32_t, int32_t)>(workspace);
    e->header = header;
    e->lead = lead;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(sizes); ++i)
        e->workspace_sizes.push_back((int)PyLong_AsLong(PyTuple_GET_ITEM(sizes, i)));
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(operands) && !PyErr_Occurred(); ++i) {
        const char *name;
        PyObject *dims;
        Operand o;
        if (!PyArg_ParseTuple(PyTuple_GET_ITEM(operands, i), "siiO!", &name, &o.kind, &o.use,
                              &PyTuple_Type, &dims))
            break;
        o.name = name;
        for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(dims); ++k) {
            int index, added;
            if (!PyArg_ParseTuple(PyTuple_GET_ITEM(dims, k), "ii", &index, &added)) break;
            o.dims.emplace_back(index, added);
        }
        e->operands.push_back(o);
    }
    PyObject *made = PyErr_Occurred() ? nullptr : PyCapsule_New(e, kCapsule, nullptr);
    if (!made) delete e;
    return made;  // (entries live as long as the process)
}

PyMethodDef methods[] = {
    {"entry", entry, METH_VARARGS, "Describe an entry point."},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "Check, allocate and call."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sequence", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sequence() { return PyModule_Create(&module); }
