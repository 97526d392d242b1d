// The Python side of the calls around the cache: arguments as torch tensors, device addresses or None, turned into pointers
// and strides and passed on to the C ABI.  (Small calls are over on the GPU before ctypes and checks in Python are done
// with them: with those the host took 6.6 us for the bookkeeping of 64 conversations, 7.6 to verify one sequence's drafts and
// 9.7 to append a token each of eight, so 4.5, 4.8 and 5.9; a launch is 2.3 of that.)
// What cannot be a buffer of the library raises, as in the package's Python; a status that is not USP_OK goes to the package's
// check().
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include <cuda_runtime_api.h>

#include "../../include/usp.h"

namespace {

// From the package: the stream's handle of a `stream` argument, what raises a status, torch's current stream of a device (or None).
PyObject *stream_of, *check, *raw_stream;
PyObject *tensor_type, *s_is_cuda, *s_is_contiguous, *s_data_ptr, *s_numel, *s_nbytes, *s_shape, *s_stride, *s_dtype;

// The arguments of a call, taken from the left.  After the first that is wrong the Python error is set and the rest is 0.
struct Args {
    PyObject* const* at;
    Py_ssize_t left;
    bool bad = false;
    bool device_seen = false;  // (a device tensor: CUDA is initialised)

    Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : at(a), left(n) {
        if (n != want) {
            PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
            bad = true;
        }
    }
    PyObject* next() {
        if (bad || left == 0) return nullptr;
        --left;
        return *at++;
    }
    void fail(PyObject* kind, const char* what) {
        if (!PyErr_Occurred()) PyErr_SetString(kind, what);
        bad = true;
    }
    bool is_tensor(PyObject* x) {
        if ((PyObject*)Py_TYPE(x) == tensor_type) return true;
        const int is = PyObject_IsInstance(x, tensor_type);
        if (is < 0) bad = true;
        return is > 0;
    }
    // A number that an attribute or a method without arguments of x gives.
    long long asked(PyObject* x, PyObject* name, bool method) {
        PyObject* y = method ? PyObject_CallMethodNoArgs(x, name) : PyObject_GetAttr(x, name);
        long long v = 0;
        if (y) {
            v = PyLong_AsLongLong(y);
            Py_DECREF(y);
        }
        if (PyErr_Occurred()) bad = true;
        return v;
    }
    uint64_t address(PyObject* x) {
        PyObject* y = PyObject_CallMethodNoArgs(x, s_data_ptr);
        uint64_t v = 0;
        if (y) {
            v = PyLong_AsUnsignedLongLongMask(y);
            Py_DECREF(y);
        }
        if (PyErr_Occurred()) bad = true;
        return v;
    }
    bool on_device(PyObject* x) {
        const bool is = truth(x, s_is_cuda, false);
        device_seen |= is;
        return is;
    }
    bool truth(PyObject* x, PyObject* name, bool method) {
        PyObject* y = method ? PyObject_CallMethodNoArgs(x, name) : PyObject_GetAttr(x, name);
        const int v = y ? PyObject_IsTrue(y) : -1;
        Py_XDECREF(y);
        if (v < 0) bad = true;
        return v > 0;
    }

    long long number() {
        PyObject* x = next();
        if (!x) return 0;
        const long long v = PyLong_AsLongLong(x);
        if (v == -1 && PyErr_Occurred()) bad = true;
        return v;
    }
    // (numbers that the C side takes as int)
    int integer() {
        const long long v = number();
        if (!bad && (v < INT32_MIN || v > INT32_MAX)) fail(PyExc_OverflowError, "number out of range");
        return bad ? 0 : (int)v;
    }
    void* stream() {  // None: torch's current one
        PyObject* x = next();
        if (!x) return nullptr;
        int device = 0;
        PyObject* y = nullptr;
        if (x == Py_None && device_seen && raw_stream != Py_None && cudaGetDevice(&device) == cudaSuccess) {
            PyObject* d = PyLong_FromLong(device);
            y = d ? PyObject_CallOneArg(raw_stream, d) : nullptr;
            Py_XDECREF(d);
        } else {
            y = PyObject_CallOneArg(stream_of, x);
        }
        const uint64_t v = y ? PyLong_AsUnsignedLongLongMask(y) : 0;
        Py_XDECREF(y);
        if (PyErr_Occurred()) bad = true;
        return (void*)(uintptr_t)v;
    }
    void* raw() {  // a host address
        PyObject* x = next();
        if (!x) return nullptr;
        const uint64_t v = PyLong_AsUnsignedLongLongMask(x);
        if (PyErr_Occurred()) bad = true;
        return (void*)(uintptr_t)v;
    }
    // A device address, or None, in x: true.
    bool plain(PyObject* x, uint64_t* v) {
        if (x == Py_None) {
            *v = 0;
            return true;
        }
        if (!PyLong_Check(x)) return false;
        *v = PyLong_AsUnsignedLongLongMask(x);
        if (PyErr_Occurred()) bad = true;
        return true;
    }
    void not_a_buffer(PyObject* x) {
        if (!PyErr_Occurred())
            PyErr_Format(PyExc_TypeError, "expected a torch tensor, a device pointer or None, got %s", Py_TYPE(x)->tp_name);
        bad = true;
    }
    // A contiguous device tensor.
    template <typename T>
    T* device() {
        PyObject* x = next();
        uint64_t v = 0;
        if (!x || plain(x, &v)) return (T*)(uintptr_t)v;
        if (!is_tensor(x)) {
            not_a_buffer(x);
            return nullptr;
        }
        if (!on_device(x) && !bad && asked(x, s_numel, true) > 0) fail(PyExc_ValueError, "libusp takes device tensors");
        if (!bad && !truth(x, s_is_contiguous, true) && !bad) fail(PyExc_ValueError, "libusp takes contiguous tensors");
        return bad ? nullptr : (T*)(uintptr_t)address(x);
    }
    // A workspace and its size, which the argument after it gives, None: the tensor's.
    void* workspace(size_t* bytes) {
        PyObject *x = bad || left < 2 ? nullptr : at[0], *n = x ? at[1] : nullptr;
        void* p = device<void>();
        if (!next() || bad) return nullptr;
        *bytes = 0;
        if (n != Py_None) {
            *bytes = PyLong_AsSize_t(n);
            if (PyErr_Occurred()) bad = true;
        } else if (x != Py_None && !PyLong_Check(x)) {
            *bytes = (size_t)asked(x, s_nbytes, false);
        }
        return p;
    }
    // Shape and strides of x; the number of its dimensions, 0 if there are more than five.
    Py_ssize_t layout(PyObject* x, long long (&shape)[5], long long (&stride)[5]) {
        PyObject *a = PyObject_GetAttr(x, s_shape), *b = a ? PyObject_CallMethodNoArgs(x, s_stride) : nullptr;
        Py_ssize_t dims = 0;
        if (a && b && PyTuple_Check(a) && PyTuple_Check(b) && PyTuple_GET_SIZE(a) == PyTuple_GET_SIZE(b) && PyTuple_GET_SIZE(a) <= 5) {
            dims = PyTuple_GET_SIZE(a);
            for (Py_ssize_t i = 0; i < dims; ++i) {
                shape[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(a, i));
                stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(b, i));
            }
        }
        Py_XDECREF(a);
        Py_XDECREF(b);
        if (PyErr_Occurred()) bad = true;
        return bad ? 0 : dims;
    }
    // Rows of `heads` times d contiguous elements, one to a token: [tokens][heads][d], or (five) [P][B][N/P][heads][d] with the
    // tokens evenly apart.
    void* rows(int64_t* step, int heads, int d, bool five) {
        PyObject* x = next();
        uint64_t v = 0;
        *step = (int64_t)heads * d;
        if (!x || plain(x, &v)) return (void*)(uintptr_t)v;
        if (!is_tensor(x)) {
            not_a_buffer(x);
            return nullptr;
        }
        long long shape[5], stride[5], tokens;
        const Py_ssize_t dims = layout(x, shape, stride);
        if (dims == 3) {
            tokens = shape[0];
            if (tokens > 1) *step = stride[0];
        } else if (five && dims == 5) {
            const long long P = shape[0], B = shape[1], n = shape[2];
            tokens = P * B * n;
            if (tokens > 0) {
                // the one distance between tokens: of the innermost dimension that has more than one of them
                *step = n > 1 ? stride[2] : B > 1 ? stride[1] : P > 1 ? stride[0] : *step;
                if ((B > 1 && stride[1] != n * *step) || (P > 1 && stride[0] != B * n * *step))
                    fail(PyExc_ValueError, "tokens must be evenly apart");
            }
            shape[1] = shape[3], shape[2] = shape[4], stride[1] = stride[3], stride[2] = stride[4];
        } else {
            if (!bad) PyErr_Format(PyExc_ValueError, "expected [tokens][%d][%d], got another number of dimensions", heads, d);
            bad = true;
            return nullptr;
        }
        if (!bad && (shape[1] != heads || shape[2] != d)) {
            PyErr_Format(PyExc_ValueError, "expected rows of [%d][%d], got [%lld][%lld]", heads, d, shape[1], shape[2]);
            bad = true;
        }
        if (!bad && tokens > 0 && !on_device(x)) fail(PyExc_ValueError, "libusp takes device tensors");
        if (!bad && tokens > 0 && (stride[2] != 1 || (heads > 1 && stride[1] != d)))
            fail(PyExc_ValueError, "the heads of a token must be contiguous");
        return bad ? nullptr : (void*)(uintptr_t)address(x);
    }
    // Rows of `vocab` contiguous probabilities of type `dtype` (a torch.dtype).
    void* probabilities(int64_t* step, int vocab, PyObject* dtype) {
        PyObject* x = next();
        uint64_t v = 0;
        *step = vocab;
        if (!x || plain(x, &v)) return (void*)(uintptr_t)v;
        if (!is_tensor(x)) {
            not_a_buffer(x);
            return nullptr;
        }
        long long shape[5], stride[5];
        if (layout(x, shape, stride) != 2 || shape[1] != vocab) {
            if (!bad) PyErr_Format(PyExc_ValueError, "expected rows of %d elements", vocab);
            bad = true;
            return nullptr;
        }
        PyObject* type = PyObject_GetAttr(x, s_dtype);
        if (!type) bad = true;
        if (type && type != dtype) {
            PyErr_Format(PyExc_ValueError, "expected %R, got %R", dtype, type);
            bad = true;
        }
        Py_XDECREF(type);
        if (shape[0] > 1) *step = stride[0];
        if (!bad && shape[0] > 0 && !on_device(x)) fail(PyExc_ValueError, "libusp takes device tensors");
        if (!bad && shape[0] > 0 && vocab > 1 && stride[1] != 1) fail(PyExc_ValueError, "the probabilities of a row must be contiguous");
        return bad ? nullptr : (void*)(uintptr_t)address(x);
    }
};

// The call itself, without the interpreter's lock (a launch waits where the GPU's queue is full).
template <typename F>
PyObject* made(const char* name, Args& a, F&& call) {
    if (a.bad) return nullptr;
    usp_status s;
    Py_BEGIN_ALLOW_THREADS;
    s = call();
    Py_END_ALLOW_THREADS;
    if (s == USP_OK) Py_RETURN_NONE;
    return PyObject_CallFunction(check, "si", name, (int)s);
}

PyObject* rotary_embed(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 10);
    const auto* p = (const usp_problem*)a.raw();
    const auto* r = (const usp_rotary*)a.raw();
    const int Hq = p ? p->Hq : 0, Hkv = p ? p->Hkv : 0, d = p ? p->d : 0;
    int64_t qs, ks, qos, kos;
    const void *q = a.rows(&qs, Hq, d, true), *k = a.rows(&ks, Hkv, d, true);
    const auto* pos = a.device<const int32_t>();
    const auto* f = a.device<const float>();
    void *qo = a.rows(&qos, Hq, d, true), *ko = a.rows(&kos, Hkv, d, true);
    const int inverse = a.integer();
    void* s = a.stream();
    return made("usp_rotary_embed", a, [&] { return usp_rotary_embed(p, r, inverse, q, qs, k, ks, pos, f, qo, qos, ko, kos, s); });
}

PyObject* kv_append_axes(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 16);
    const auto* c = (const usp_cache*)a.raw();
    const int Hq = c ? c->Hq : 0, Hkv = c ? c->Hkv : 0, d = c ? c->d : 0, tokens = a.integer();
    int64_t qs, ks, vs;
    const void *q = a.rows(&qs, Hq, d, false), *k = a.rows(&ks, Hkv, d, false), *v = a.rows(&vs, Hkv, d, false);
    const int32_t *seq = a.device<const int32_t>(), *pos = a.device<const int32_t>(), *rot_pos = a.device<const int32_t>();
    const auto* f = a.device<const float>();
    const auto* r = (const usp_rotary*)a.raw();
    void *qo = a.device<void>(), *ko = a.device<void>(), *kp = a.device<void>(), *vp = a.device<void>();
    const auto* table = a.device<const int32_t>();
    void* s = a.stream();
    return made("usp_kv_append_axes", a, [&] {
        return usp_kv_append_axes(c, tokens, q, qs, k, ks, v, vs, seq, pos, rot_pos, f, r, qo, ko, kp, vp, table, s);
    });
}

PyObject* pages_update(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 11);
    const auto* c = (const usp_cache*)a.raw();
    const int32_t *parent = a.device<const int32_t>(), *keep = a.device<const int32_t>(), *grow = a.device<const int32_t>();
    int32_t *lens = a.device<int32_t>(), *table = a.device<int32_t>(), *ref = a.device<int32_t>(), *copies = a.device<int32_t>();
    size_t bytes = 0;
    void* ws = a.workspace(&bytes);
    void* s = a.stream();
    return made("usp_pages_update", a, [&] { return usp_pages_update(c, parent, keep, grow, lens, table, ref, copies, ws, bytes, s); });
}

PyObject* pages_compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 8);
    const auto* c = (const usp_cache*)a.raw();
    const int32_t *table = a.device<const int32_t>(), *ref = a.device<const int32_t>();
    int32_t *table_out = a.device<int32_t>(), *ref_out = a.device<int32_t>(), *new_id = a.device<int32_t>(), *copies = a.device<int32_t>();
    void* s = a.stream();
    return made("usp_pages_compact", a, [&] { return usp_pages_compact(c, table, ref, table_out, ref_out, new_id, copies, s); });
}

PyObject* pages_copy(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 8);
    const auto* c = (const usp_cache*)a.raw();
    const int most = a.integer();
    const auto* copies = a.device<const int32_t>();
    void *kp = a.device<void>(), *vp = a.device<void>();
    const int layers = a.integer();
    const int64_t stride = a.number();
    void* s = a.stream();
    return made("usp_pages_copy", a, [&] { return usp_pages_copy(c, most, copies, layers, stride, kp, vp, s); });
}

PyObject* verify_drafts(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 15);
    const int seqs = a.integer(), tokens = a.integer(), vocab = a.integer(), type = a.integer();
    PyObject* dtype = a.next();
    int64_t ts, ds;
    const void *target = a.probabilities(&ts, vocab, dtype), *draft = a.probabilities(&ds, vocab, dtype);
    const auto* ids = a.device<const int32_t>();
    const auto* u = a.device<const float>();
    const int32_t *start = a.device<const int32_t>(), *lens = a.device<const int32_t>();
    int32_t *accepted = a.device<int32_t>(), *next = a.device<int32_t>(), *keep = a.device<int32_t>();
    void* s = a.stream();
    return made("usp_verify_drafts", a, [&] {
        return usp_verify_drafts(seqs, tokens, vocab, type, target, ts, draft, ds, ids, u, start, lens, accepted, next, keep, s);
    });
}

// configure(stream_of, check, raw_stream), by the package before any call.
PyObject* configure(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 3);
    PyObject** const to[] = {&stream_of, &check, &raw_stream};
    for (PyObject** x : to) {
        PyObject* y = a.next();
        if (!y) return nullptr;
        Py_INCREF(y);
        Py_XDECREF(*x);
        *x = y;
    }
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)(void))F, METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<rotary_embed>("rotary_embed"),   method<kv_append_axes>("kv_append_axes"),
                         method<pages_update>("pages_update"),   method<pages_compact>("pages_compact"),
                         method<pages_copy>("pages_copy"),       method<verify_drafts>("verify_drafts"),
                         method<configure>("configure"),         {nullptr, nullptr, 0, nullptr}};
PyModuleDef definition = {PyModuleDef_HEAD_INIT, "uspbinding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_uspbinding(void) {
    PyObject* torch = PyImport_ImportModule("torch");
    if (!torch) return nullptr;
    tensor_type = PyObject_GetAttrString(torch, "Tensor");
    Py_DECREF(torch);
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_numel = PyUnicode_InternFromString("numel");
    s_nbytes = PyUnicode_InternFromString("nbytes");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype");
    if (!tensor_type || !s_dtype) return nullptr;
    return PyModule_Create(&definition);
}
