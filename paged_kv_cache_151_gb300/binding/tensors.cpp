// tensors.cpp -- the checks of a call's tensors, for the Python binding.
//
// A call over a dozen tensors asks each of them for its device, type, shape, strides and
// address; from Python that takes longer than a small kernel runs (write of 256 rows:
// 8.3 us a call, of which the C call takes 3.6).  A Spec states once what a
// function's tensors have to be and checks them all in one call:
//
//   Spec("out:T[R,V]~ logits:T[R,V]~ query_start:i32[B+1] tokens:i32[R]?")
//
// Each tensor: name, ":", type, "[", sizes, "]", flags.
//   type   i32 i64 u8 f32; T: float32, bfloat16 or float16, the same for all T;
//          H: bfloat16 or float16, the same for all H; O: T's type or float32
//   sizes  numbers, or one-letter names that stand for the same size wherever they
//          are, a following + 1 adding one
//   flags  "~": rows (along the first size) any distance apart, else contiguous;
//          "?": may be None
// Calling it with the current device and the tensors gives a tuple of numbers: each
// tensor's address (0: None), the sizes in the order of their first letters (0 where
// only missing tensors have them), the row distances of the "~" tensors in elements (a
// single row's: what it holds, as it is never used), and the codes of T or H and of O.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <string>
#include <vector>

namespace {

struct Size {
    int letter;                                    // index of its letter, -1: a number
    int64_t add;                                   // the number, or what is added
};

struct Arg {
    std::string name, text;                        // text: what is wanted, for messages
    char type[4];
    std::vector<Size> sizes;
    bool rows, optional;
};

struct Spec {
    PyObject_HEAD
    std::vector<Arg> *args;
    std::string *letters;
    int n_rows;
    bool any_out;                                  // has an O
};

int float_code(at::ScalarType t) {                 // PA_F32, PA_BF16, PA_F16
    return t == at::kFloat ? 0 : t == at::kBFloat16 ? 1 : t == at::kHalf ? 2 : -1;
}

PyObject *wrong(const Arg &a) {
    PyErr_Format(PyExc_ValueError, "%s must be %s", a.name.c_str(), a.text.c_str());
    return nullptr;
}

PyObject *check(PyObject *self_, PyObject *args, PyObject *kwargs) {
    auto *self = reinterpret_cast<Spec *>(self_);
    const auto &specs = *self->args;
    const Py_ssize_t n = (Py_ssize_t)specs.size();
    if (kwargs || PyTuple_GET_SIZE(args) != n + 1) {
        PyErr_SetString(PyExc_TypeError, "a device and one value per tensor are wanted");
        return nullptr;
    }
    const long device = PyLong_AsLong(PyTuple_GET_ITEM(args, 0));
    if (device == -1 && PyErr_Occurred()) return nullptr;
    constexpr int MOST = 64;
    int64_t address[MOST], size[MOST], rows[MOST];
    const int letters = (int)self->letters->size();
    for (int i = 0; i < letters; ++i) size[i] = -1;
    int code = -1, out_code = -1, n_rows = 0;
    for (Py_ssize_t i = 0; i < n; ++i) {
        const Arg &a = specs[i];
        PyObject *o = PyTuple_GET_ITEM(args, i + 1);
        if (o == Py_None && a.optional) {
            address[i] = 0;
            if (a.rows) rows[n_rows++] = 0;
            continue;
        }
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", a.name.c_str());
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) {
            PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", a.name.c_str());
            return nullptr;
        }
        if (t.get_device() != device) {
            PyErr_Format(PyExc_ValueError, "%s is not on the current device", a.name.c_str());
            return nullptr;
        }
        const at::ScalarType type = t.scalar_type();
        switch (a.type[0]) {
            case 'T': case 'H': {
                const int c = float_code(type);
                if (c < (a.type[0] == 'H' ? 1 : 0) || (code >= 0 && c != code)) return wrong(a);
                code = c;
                break;
            }
            case 'O': {
                out_code = float_code(type);       // against T's once all are seen
                if (out_code < 0) return wrong(a);
                break;
            }
            case 'f': if (type != at::kFloat) return wrong(a); break;
            case 'u': if (type != at::kByte) return wrong(a); break;
            default: if (type != (a.type[1] == '3' ? at::kInt : at::kLong)) return wrong(a);
        }
        const auto shape = t.sizes();
        if (shape.size() != a.sizes.size()) return wrong(a);
        for (size_t d = 0; d < shape.size(); ++d) {
            const Size &s = a.sizes[d];
            if (s.letter < 0) {
                if (shape[d] != s.add) return wrong(a);
            } else if (size[s.letter] < 0) {
                size[s.letter] = shape[d] - s.add;
                if (size[s.letter] < 0) return wrong(a);
            } else if (shape[d] != size[s.letter] + s.add) {
                return wrong(a);
            }
        }
        if (!a.rows) {
            if (!t.is_contiguous()) return wrong(a);
        } else {
            const auto stride = t.strides();
            int64_t inside = 1;                    // elements of a row
            for (size_t d = shape.size(); d-- > 1;) {
                if (shape[d] > 1 && stride[d] != inside && t.numel() > 0) return wrong(a);
                inside *= shape[d];
            }
            rows[n_rows++] = shape[0] > 1 ? stride[0] : inside;
        }
        address[i] = reinterpret_cast<int64_t>(t.data_ptr());
    }
    if (self->any_out && out_code > 0 && out_code != code) {
        for (const Arg &a : specs)
            if (a.type[0] == 'O') return wrong(a);
    }
    const Py_ssize_t total = n + letters + n_rows + (code >= 0) + (self->any_out ? 1 : 0);
    PyObject *r = PyTuple_New(total);
    if (!r) return nullptr;
    Py_ssize_t at = 0;
    auto put = [&](int64_t v) {
        PyObject *x = PyLong_FromLongLong(v);
        if (x) PyTuple_SET_ITEM(r, at++, x);
        return x != nullptr;
    };
    bool ok = true;
    for (Py_ssize_t i = 0; i < n; ++i) ok = ok && put(address[i]);
    for (int i = 0; i < letters; ++i) ok = ok && put(size[i] < 0 ? 0 : size[i]);
    for (int i = 0; i < n_rows; ++i) ok = ok && put(rows[i]);
    if (code >= 0) ok = ok && put(code);
    if (self->any_out) ok = ok && put(out_code);
    if (!ok) {
        Py_DECREF(r);
        return nullptr;
    }
    return r;
}

// (a sparse tensor has no strides to ask for, one without storage no address)
PyObject *spec_call(PyObject *self, PyObject *args, PyObject *kwargs) {
    try {
        return check(self, args, kwargs);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
}

PyObject *make(PyTypeObject *type, PyObject *args, PyObject *kwargs) {
    const char *text;
    if (kwargs || !PyArg_ParseTuple(args, "s", &text)) return nullptr;
    auto *self = reinterpret_cast<Spec *>(type->tp_alloc(type, 0));
    if (!self) return nullptr;
    self->args = new std::vector<Arg>;
    self->letters = new std::string;
    self->n_rows = 0;
    self->any_out = false;
    const char *p = text;
    bool bad = false;
    while (*p && !bad) {
        while (*p == ' ') ++p;
        if (!*p) break;
        Arg a;
        while (*p && *p != ':') a.name += *p++;
        if (*p) ++p;
        std::string t, dims;
        while (*p && *p != '[') t += *p++;
        if (*p) ++p;
        while (*p && *p != ']') dims += *p++;
        bad = *p != ']' || t.empty() || t.size() > 3;
        if (bad) break;
        ++p;
        a.rows = a.optional = false;
        for (; *p && *p != ' '; ++p) {
            if (*p == '~') a.rows = true;
            else if (*p == '?') a.optional = true;
            else bad = true;
        }
        std::memset(a.type, 0, sizeof a.type);
        std::memcpy(a.type, t.data(), t.size());
        for (size_t i = 0; i < dims.size();) {
            Size s{-1, 0};
            if (dims[i] >= '0' && dims[i] <= '9') {
                while (i < dims.size() && dims[i] >= '0' && dims[i] <= '9') s.add = 10 * s.add + (dims[i++] - '0');
            } else {
                const size_t at = self->letters->find(dims[i]);
                s.letter = (int)(at == std::string::npos ? self->letters->size() : at);
                if (at == std::string::npos) *self->letters += dims[i];
                ++i;
                if (dims.compare(i, 2, "+1") == 0) {
                    s.add = 1;
                    i += 2;
                }
            }
            a.sizes.push_back(s);
            if (i < dims.size()) bad = bad || dims[i++] != ',';
        }
        a.text = std::string(a.rows ? "a tensor with contiguous rows, " : "a contiguous tensor, ") +
                 (t == "T" ? "float32, bfloat16 or float16 like the others"
                  : t == "H" ? "bfloat16 or float16 like the others"
                  : t == "O" ? "float32 or like the input"
                  : t == "i32" ? "int32" : t == "i64" ? "int64" : t == "u8" ? "uint8" : "float32") +
                 ", [" + dims + "]";
        self->n_rows += a.rows;
        self->any_out = self->any_out || t == "O";
        self->args->push_back(a);
    }
    if (bad || self->args->size() > 60 || self->letters->size() > 60) {
        Py_DECREF(reinterpret_cast<PyObject *>(self));
        PyErr_SetString(PyExc_ValueError, "not a description of tensors");
        return nullptr;
    }
    return reinterpret_cast<PyObject *>(self);
}

PyObject *spec_new(PyTypeObject *type, PyObject *args, PyObject *kwargs) {
    try {
        return make(type, args, kwargs);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_MemoryError, e.what());
        return nullptr;
    }
}

void spec_dealloc(PyObject *self_) {
    auto *self = reinterpret_cast<Spec *>(self_);
    delete self->args;
    delete self->letters;
    Py_TYPE(self_)->tp_free(self_);
}

PyTypeObject SpecType = {PyVarObject_HEAD_INIT(nullptr, 0)};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", "Checks of a call's tensors.", -1, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() {
    SpecType.tp_name = "_tensors.Spec";
    SpecType.tp_basicsize = sizeof(Spec);
    SpecType.tp_flags = Py_TPFLAGS_DEFAULT;
    SpecType.tp_new = spec_new;
    SpecType.tp_call = spec_call;
    SpecType.tp_dealloc = spec_dealloc;
    if (PyType_Ready(&SpecType) < 0) return nullptr;
    PyObject *m = PyModule_Create(&module);
    if (!m) return nullptr;
    Py_INCREF(&SpecType);
    if (PyModule_AddObject(m, "Spec", reinterpret_cast<PyObject *>(&SpecType)) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
