// The Python side of the calls around the cache: arguments as torch tensors, device addresses or None, turned into pointers
// and strides and passed on to the C ABI.  (Small calls are over on the GPU before ctypes and checks in Python are done
// with them: with those the host took 6.6 us for the bookkeeping of 64 conversations, 7.6 to verify one sequence's drafts and
// 9.7 to append a token each of eight, so 4.4, 4.7 and 5.4; a launch is 2.3 of that.)
// What cannot be the buffer of the library that the call says (its place, its type, how much it holds, how it lies) raises, as in
// the package's Python; a status that is not USP_OK goes to the package's check().
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <cstring>
#include <initializer_list>

#include <cuda_runtime_api.h>

#include "../../include/usp.h"

namespace {

// From the package: the stream's handle of a `stream` argument, what raises a status, torch's current stream of a device (or None),
// the address of an object's struct, and the classes of objects that have one.
PyObject *stream_of, *check, *raw_stream, *struct_of, *problem_type, *cache_type, *rotary_type;
PyObject *t_int32, *t_float32, *t_bfloat16;  // torch's
PyObject *tensor_type, *s_made;

// An attribute of tensors, or a method that is called without arguments.  Of a torch.Tensor itself what its class has under the
// name is called as it is (looked up anew it takes 15 ns more, and a call asks up to fifty times); of a subclass's objects, or
// where the class has something else there, it is looked up.
struct Asked {
    const char* text;
    PyObject *name = nullptr, *none = nullptr;
    PyGetSetDef* attribute = nullptr;
    PyMethodDef* method = nullptr;
    bool is_method = false;

    bool find() {
        name = PyUnicode_InternFromString(text);
        none = PyTuple_New(0);
        PyObject* x = name && none ? PyObject_GetAttr(tensor_type, name) : nullptr;
        if (!x) return false;
        if (Py_TYPE(x) == &PyGetSetDescr_Type) attribute = ((PyGetSetDescrObject*)x)->d_getset;
        if (Py_TYPE(x) == &PyMethodDescr_Type) method = ((PyMethodDescrObject*)x)->d_method;
        is_method = PyCallable_Check(x);
        return true;  // (x, and what it names, stay)
    }
    PyObject* of(PyObject* x) const {
        if ((PyObject*)Py_TYPE(x) == tensor_type) {
            if (attribute) return attribute->get(x, attribute->closure);
            if (method && method->ml_flags == METH_NOARGS) return method->ml_meth(x, nullptr);
            if (method && method->ml_flags == METH_VARARGS) return method->ml_meth(x, none);
            if (method && method->ml_flags == (METH_VARARGS | METH_KEYWORDS))
                return ((PyCFunctionWithKeywords)(void (*)(void))method->ml_meth)(x, none, nullptr);
        }
        return is_method ? PyObject_CallMethodNoArgs(x, name) : PyObject_GetAttr(x, name);
    }
};
Asked is_cuda{"is_cuda"}, is_contiguous{"is_contiguous"}, data_ptr{"data_ptr"}, nbytes{"nbytes"}, shape_of{"shape"},
    stride_of{"stride"}, dtype_of{"dtype"};

// How many elements of a type (of torch's, or null: any) and of how many bytes a tensor has to have.
struct Want {
    PyObject* type;
    int64_t n;
    int size = 4;
};
// The product of sizes, as far as it goes; 0 where one is not positive (the C side says what is wrong with it).
template <typename... N>
int64_t times(N... sizes) {
    int64_t n = 1;
    for (const int64_t x : {(int64_t)sizes...}) {
        if (x <= 0) return 0;
        if (__builtin_mul_overflow(n, x, &n)) n = INT64_MAX;
    }
    return n;
}
Want ints(int64_t n) { return {t_int32, n}; }
Want floats(int64_t n) { return {t_float32, n}; }
int size_of(int dtype) { return dtype == USP_BF16 ? 2 : 4; }
PyObject* type_of(int dtype) { return dtype == USP_F32 ? t_float32 : dtype == USP_BF16 ? t_bfloat16 : nullptr; }
int64_t pool(const usp_cache* c) { return c ? times(c->n_pages, c->Hkv, c->page_size, c->d) : 0; }
int64_t table(const usp_cache* c) { return c ? times(c->n_seqs, c->max_pages) : 0; }

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
    // A number that x says.
    long long asked(PyObject* x, const Asked& what) {
        PyObject* y = what.of(x);
        long long v = 0;
        if (y) {
            v = PyLong_AsLongLong(y);
            Py_DECREF(y);
        }
        if (PyErr_Occurred()) bad = true;
        return v;
    }
    uint64_t address(PyObject* x) {
        PyObject* y = data_ptr.of(x);
        uint64_t v = 0;
        if (y) {
            v = PyLong_AsUnsignedLongLongMask(y);
            Py_DECREF(y);
        }
        if (PyErr_Occurred()) bad = true;
        return v;
    }
    bool on_device(PyObject* x) {
        const bool is = truth(x, is_cuda);
        device_seen |= is;
        return is;
    }
    bool truth(PyObject* x, const Asked& what) {
        PyObject* y = what.of(x);
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
    // The struct of an object of class `kind`, which keeps it with its address as `_made`, or of what the package takes for one.
    template <typename T>
    const T* made_of(PyObject* kind) {
        PyObject* x = next();
        if (!x) return nullptr;
        PyObject *kept = (PyObject*)Py_TYPE(x) == kind ? PyObject_GetAttr(x, s_made) : nullptr, *y = nullptr;
        if (kept && PyTuple_Check(kept) && PyTuple_GET_SIZE(kept) == 2) {
            y = Py_NewRef(PyTuple_GET_ITEM(kept, 1));
        } else {
            if (PyErr_ExceptionMatches(PyExc_AttributeError)) PyErr_Clear();  // (not made yet)
            PyObject* const both[] = {x, kind};
            if (!PyErr_Occurred()) y = PyObject_Vectorcall(struct_of, both, 2, nullptr);
        }
        Py_XDECREF(kept);
        const uint64_t v = y ? PyLong_AsUnsignedLongLongMask(y) : 0;
        Py_XDECREF(y);
        if (PyErr_Occurred()) bad = true;
        return bad ? nullptr : (const T*)(uintptr_t)v;
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
    void typed(PyObject* x, PyObject* type) {
        if (bad || !type) return;
        PyObject* is = dtype_of.of(x);
        if (is && is != type) PyErr_Format(PyExc_ValueError, "expected %R, got %R", type, is);
        bad |= is != type;
        Py_XDECREF(is);
    }
    // A contiguous device tensor.  (One without elements is no more than a null pointer.)
    template <typename T>
    T* device(const Want& want) {
        PyObject* x = next();
        uint64_t v = 0;
        if (!x || plain(x, &v)) return (T*)(uintptr_t)v;
        if (!is_tensor(x)) {
            not_a_buffer(x);
            return nullptr;
        }
        const long long bytes = asked(x, nbytes);
        if (bytes > 0) {
            typed(x, want.type);
            if (!bad && bytes / want.size < want.n) {
                PyErr_Format(PyExc_ValueError, "expected %lld elements of %d bytes at least, got %lld bytes", (long long)want.n, want.size, bytes);
                bad = true;
            }
        }
        if (!bad && !on_device(x) && bytes > 0) fail(PyExc_ValueError, "libusp takes device tensors");
        if (!bad && !truth(x, is_contiguous) && !bad) fail(PyExc_ValueError, "libusp takes contiguous tensors");
        return bad ? nullptr : (T*)(uintptr_t)address(x);
    }
    // A workspace and its size, which the argument after it gives, None: the tensor's.
    void* workspace(size_t* bytes) {
        PyObject *x = bad || left < 2 ? nullptr : at[0], *n = x ? at[1] : nullptr;
        *bytes = 0;
        if (x && n != Py_None) {
            *bytes = PyLong_AsSize_t(n);
            if (PyErr_Occurred()) bad = true;
        }
        if (x && !bad && x != Py_None && !PyLong_Check(x) && is_tensor(x)) {
            const size_t whole = (size_t)asked(x, nbytes);
            if (n == Py_None) *bytes = whole;
            if (!bad && *bytes > whole) fail(PyExc_ValueError, "a workspace of more bytes than the tensor has");
        }
        void* p = device<void>({nullptr, 0});
        return next() && !bad ? p : nullptr;
    }
    // Shape and strides of x; the number of its dimensions, 0 if there are more than five.
    Py_ssize_t layout(PyObject* x, long long (&shape)[5], long long (&stride)[5]) {
        PyObject *a = shape_of.of(x), *b = a ? stride_of.of(x) : nullptr;
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
    // Rows of `heads` times d contiguous elements, one to each of want.n tokens at least: [tokens][heads][d], or (five)
    // [P][B][N/P][heads][d] with the tokens evenly apart.
    void* rows(int64_t* step, int heads, int d, bool five, const Want& want) {
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
        if (!bad && tokens < want.n) {
            PyErr_Format(PyExc_ValueError, "expected rows of %lld tokens at least, got %lld", (long long)want.n, tokens);
            bad = true;
        }
        if (tokens > 0) typed(x, want.type);
        if (!bad && tokens > 0 && !on_device(x)) fail(PyExc_ValueError, "libusp takes device tensors");
        if (!bad && tokens > 0 && (stride[2] != 1 || (heads > 1 && stride[1] != d)))
            fail(PyExc_ValueError, "the heads of a token must be contiguous");
        return bad ? nullptr : (void*)(uintptr_t)address(x);
    }
    // The type of probabilities, "f32", "bf16" or None: that of the tensor `of`.
    int probability_type(PyObject* of) {
        PyObject* x = next();
        if (!x) return USP_F32;
        if (x == Py_None && of != Py_None && is_tensor(of)) {
            PyObject* type = dtype_of.of(of);
            if (type && type != t_float32 && type != t_bfloat16) PyErr_Format(PyExc_ValueError, "expected float32 or bfloat16, got %R", type);
            bad |= PyErr_Occurred() != nullptr;
            Py_XDECREF(type);
            return type == t_bfloat16 ? USP_BF16 : USP_F32;
        }
        if (x == Py_None) {  // (nothing, or what is no buffer and refused as such)
            if (of != Py_None && PyLong_Check(of)) fail(PyExc_ValueError, "dtype: 'f32' or 'bf16' is needed with a device pointer");
            return USP_F32;
        }
        const char* name = PyUnicode_Check(x) ? PyUnicode_AsUTF8(x) : nullptr;
        const bool f32 = name && !strcmp(name, "f32"), bf16 = name && !strcmp(name, "bf16");
        if (!f32 && !bf16) {
            if (!PyErr_Occurred()) PyErr_Format(PyExc_KeyError, "%R", x);
            bad = true;
        }
        return bf16 ? USP_BF16 : USP_F32;
    }
    // want.n rows, at least, of `vocab` contiguous probabilities.
    void* probabilities(int64_t* step, int vocab, const Want& want) {
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
        typed(x, want.type);
        if (!bad && shape[0] < want.n) {
            PyErr_Format(PyExc_ValueError, "expected %lld rows at least, got %lld", (long long)want.n, shape[0]);
            bad = true;
        }
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
    const auto* p = a.made_of<usp_problem>(problem_type);
    const auto* r = a.made_of<usp_rotary>(rotary_type);
    const int Hq = p ? p->Hq : 0, Hkv = p ? p->Hkv : 0, d = p ? p->d : 0;
    const Want tokens{p ? type_of(p->dtype) : nullptr, p ? times(p->B, p->N) : 0};
    int64_t qs, ks, qos, kos;
    const void *q = a.rows(&qs, Hq, d, true, tokens), *k = a.rows(&ks, Hkv, d, true, tokens);
    const auto* pos = a.device<const int32_t>(ints(r && r->rot > 0 ? times(r->n_axes, tokens.n) : 0));
    const auto* f = a.device<const float>(floats(r && tokens.n > 0 ? r->rot / 2 : 0));
    void *qo = a.rows(&qos, Hq, d, true, tokens), *ko = a.rows(&kos, Hkv, d, true, tokens);
    const int inverse = a.integer();
    void* s = a.stream();
    return made("usp_rotary_embed", a, [&] { return usp_rotary_embed(p, r, inverse, q, qs, k, ks, pos, f, qo, qos, ko, kos, s); });
}

PyObject* kv_append_axes(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 16);
    const auto* c = a.made_of<usp_cache>(cache_type);
    const auto* r = a.made_of<usp_rotary>(rotary_type);
    const int Hq = c ? c->Hq : 0, Hkv = c ? c->Hkv : 0, d = c ? c->d : 0, tokens = a.integer();
    PyObject* type = c ? type_of(c->dtype) : nullptr;
    const int size = c ? size_of(c->dtype) : 4;
    const Want each{type, tokens, size}, all{type, pool(c), size};
    int64_t qs, ks, vs;
    const void *q = a.rows(&qs, Hq, d, false, each), *k = a.rows(&ks, Hkv, d, false, each), *v = a.rows(&vs, Hkv, d, false, each);
    const int32_t *seq = a.device<const int32_t>(ints(tokens)), *pos = a.device<const int32_t>(ints(tokens));
    const auto* rot_pos = a.device<const int32_t>(ints(r && r->rot > 0 ? times(r->n_axes, tokens) : 0));
    const auto* f = a.device<const float>(floats(r && tokens > 0 ? r->rot / 2 : 0));
    void *qo = a.device<void>({type, times(tokens, Hq, d), size}), *ko = a.device<void>({type, times(tokens, Hkv, d), size});
    void *kp = a.device<void>(all), *vp = a.device<void>(all);
    const auto* ids = a.device<const int32_t>(ints(table(c)));
    void* s = a.stream();
    return made("usp_kv_append_axes", a, [&] {
        return usp_kv_append_axes(c, tokens, q, qs, k, ks, v, vs, seq, pos, rot_pos, f, r, qo, ko, kp, vp, ids, s);
    });
}

PyObject* pages_update(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 11);
    const auto* c = a.made_of<usp_cache>(cache_type);
    const Want slots = ints(c ? c->n_seqs : 0);
    const int32_t *parent = a.device<const int32_t>(slots), *keep = a.device<const int32_t>(slots), *grow = a.device<const int32_t>(slots);
    int32_t *lens = a.device<int32_t>(slots), *ids = a.device<int32_t>(ints(table(c))), *ref = a.device<int32_t>(ints(c ? c->n_pages : 0));
    int32_t* copies = a.device<int32_t>(ints(times(4, 1 + slots.n)));
    size_t bytes = 0;
    void* ws = a.workspace(&bytes);
    void* s = a.stream();
    return made("usp_pages_update", a, [&] { return usp_pages_update(c, parent, keep, grow, lens, ids, ref, copies, ws, bytes, s); });
}

PyObject* pages_compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 8);
    const auto* c = a.made_of<usp_cache>(cache_type);
    const Want entries = ints(table(c)), pages = ints(c ? c->n_pages : 0);
    const int32_t *ids = a.device<const int32_t>(entries), *ref = a.device<const int32_t>(pages);
    int32_t *ids_out = a.device<int32_t>(entries), *ref_out = a.device<int32_t>(pages), *new_id = a.device<int32_t>(pages);
    int32_t* copies = a.device<int32_t>(ints(times(4, 1 + pages.n / 2)));
    void* s = a.stream();
    return made("usp_pages_compact", a, [&] { return usp_pages_compact(c, ids, ref, ids_out, ref_out, new_id, copies, s); });
}

PyObject* pages_copy(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 8);
    const auto* c = a.made_of<usp_cache>(cache_type);
    const int layers = a.integer();
    const int64_t stride = a.number();
    const int most = a.integer();
    const auto* copies = a.device<const int32_t>(ints(most > 0 ? 4 : 0));  // (row 0 says how many rows are read)
    const int64_t one = pool(c), before = layers > 1 ? times(layers - 1, stride) : 0;
    // (pages are moved as bytes, whatever type the tensor says)
    const Want all{nullptr, layers < 1 || most < 1 ? 0 : before > INT64_MAX - one ? INT64_MAX : before + one, c ? size_of(c->dtype) : 4};
    void *kp = a.device<void>(all), *vp = a.device<void>(all);
    void* s = a.stream();
    return made("usp_pages_copy", a, [&] { return usp_pages_copy(c, most, copies, layers, stride, kp, vp, s); });
}

PyObject* verify_drafts(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 14);
    const int seqs = a.integer(), tokens = a.integer(), vocab = a.integer(), type = a.probability_type(n == 14 ? args[4] : Py_None);
    const Want each{type_of(type), tokens};
    int64_t ts, ds;
    const void *target = a.probabilities(&ts, vocab, each), *draft = a.probabilities(&ds, vocab, each);
    const auto* ids = a.device<const int32_t>(ints(tokens));
    const auto* u = a.device<const float>(floats(tokens));
    const Want slots = ints(seqs);
    const auto* start = a.device<const int32_t>(ints(seqs > 0 ? (int64_t)seqs + 1 : 0));
    const auto* lens = a.device<const int32_t>(slots);
    int32_t *accepted = a.device<int32_t>(slots), *next = a.device<int32_t>(slots), *keep = a.device<int32_t>(slots);
    void* s = a.stream();
    return made("usp_verify_drafts", a, [&] {
        return usp_verify_drafts(seqs, tokens, vocab, type, target, ts, draft, ds, ids, u, start, lens, accepted, next, keep, s);
    });
}

// configure(stream_of, check, raw_stream, struct_of, problem_type, cache_type, rotary_type), by the package before any call.
PyObject* configure(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a(args, n, 7);
    PyObject** const to[] = {&stream_of, &check, &raw_stream, &struct_of, &problem_type, &cache_type, &rotary_type};
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
    t_int32 = PyObject_GetAttrString(torch, "int32");
    t_float32 = PyObject_GetAttrString(torch, "float32");
    t_bfloat16 = PyObject_GetAttrString(torch, "bfloat16");
    Py_DECREF(torch);
    s_made = PyUnicode_InternFromString("_made");
    if (!tensor_type || !t_int32 || !t_float32 || !t_bfloat16 || !s_made) return nullptr;
    for (Asked* x : {&is_cuda, &is_contiguous, &data_ptr, &nbytes, &shape_of, &stride_of, &dtype_of})
        if (!x->find()) return nullptr;
    return PyModule_Create(&definition);
}
