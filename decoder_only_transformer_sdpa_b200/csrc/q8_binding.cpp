// q8_binding.cpp -- the module `_q8`: the 8-bit cache's calls on torch tensors.
//
// Checks what a call gets, makes the outputs that it was not lent and hands
// addresses, strides and the device's current stream to the entry points of
// libattn.so.  What bounds it is the host's time: a decode of one token is 4.5 us
// of GPU time, and issuing it takes 5.6 us from here, 2.4 us of that the launch
// and 2.8 us the two outputs (2.5 straight from the allocator, unseen by dispatch
// modes); the same steps from Python (each tensor's attributes one by one, then
// ctypes) took 11.6 us, and the GPU waited for them.
//
// The functions of libattn.so come as addresses (`bind`), so that the build of
// it that the package has loaded is the one that runs.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/attn.h"

namespace {

struct Api {
    decltype(&attn_q8_append) append;
    decltype(&attn_q8_read) read;
    decltype(&attn_q8_decode_workspace_bytes) decode_workspace_bytes;
    decltype(&attn_q8_decode) decode;
    decltype(&attn_q8_select) select;
    decltype(&attn_q8_evict_workspace_bytes) evict_workspace_bytes;
    decltype(&attn_q8_evict) evict;
};
Api api;
PyObject *error_class;  // AttnError(status, where)

constexpr long kMaxBlocks = 32768;

// A cache's structure and device.  The Python object that owns this one keeps the tensors.
struct Cache {
    attn_q8_cache c;
    int index;
};
constexpr const char *kCapsule = "attn_q8_cache";

const Cache &cache_of(PyObject *capsule) {
    auto *c = static_cast<Cache *>(PyCapsule_GetPointer(capsule, kCapsule));
    if (!c) throw python_error();
    return *c;
}

[[noreturn]] void fail_status(int status, const char *where) {
    PyObject *e = PyObject_CallFunction(error_class, "is", status, where);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    throw python_error();
}
template <typename... Args>
[[noreturn]] void fail(PyObject *type, const char *format, Args... args) {
    PyErr_Format(type, format, args...);
    throw python_error();
}

// A shape as Python prints it.
struct Shape {
    PyObject *tuple;
    explicit Shape(at::IntArrayRef s) : tuple(PyTuple_New((Py_ssize_t)s.size())) {
        for (size_t i = 0; tuple && i < s.size(); ++i) PyTuple_SET_ITEM(tuple, (Py_ssize_t)i, PyLong_FromLongLong(s[i]));
        if (!tuple) throw python_error();
    }
    ~Shape() { Py_DECREF(tuple); }
};

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

void check(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, int index) {
    if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, "%s must be %R, got %R", name, (PyObject *)torch::getTHPDtype(type),
             (PyObject *)torch::getTHPDtype(t.scalar_type()));
    if (t.sizes() != shape) {
        const Shape want(shape), got(t.sizes());
        fail(PyExc_ValueError, "%s must have shape %R, got %R", name, want.tuple, got.tuple);
    }
    if (t.get_device() != index) fail(PyExc_ValueError, "%s must be on cuda:%d, got cuda:%d", name, index, (int)t.get_device());
}

// A contiguous tensor of this type and shape.
template <typename T>
T *whole(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int index) {
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, shape, index);
    if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
    return static_cast<T *>(t.data_ptr());
}

// A new contiguous tensor, by torch's dispatcher, so that what watches a program's tensors sees it.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int index) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)index));
}

// The same, made where it is not lent; `kept` holds a reference to it.
template <typename T>
T *output(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int index, THPObjectPtr &kept) {
    if (o != Py_None) {
        T *p = whole<T>(o, name, type, shape, index);
        Py_INCREF(o);
        kept = o;
        return p;
    }
    at::Tensor t = fresh(shape, type, index);
    T *p = static_cast<T *>(t.data_ptr());
    kept = THPVariable_Wrap(std::move(t));
    if (!kept) throw python_error();
    return p;
}

// A bf16 [B, H, T, D] view with unit stride along D.
void *view(const at::Tensor &t, const char *name, at::IntArrayRef shape, int index, attn_strides &strides) {
    check(t, name, at::kBFloat16, shape, index);
    if (t.stride(3) != 1) fail(PyExc_ValueError, "%s must have unit stride along D", name);
    strides = attn_strides{t.stride(0), t.stride(1), t.stride(2)};
    return t.data_ptr();
}

const at::Tensor &four(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 4) fail(PyExc_ValueError, "expected [B, H, T, D]");
    return t;
}

// A whole number between low and high; anything else is a bad shape.
int number(PyObject *o, long low, long high, const char *where) {
    int over = 0;
    const long x = PyLong_AsLongAndOverflow(o, &over);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    if (over || x < low || x > high) fail_status(ATTN_ERR_SHAPE, where);
    return (int)x;
}

// Device memory of the call's own; it goes back to the stream's pool when the call is enqueued.
struct Workspace {
    at::Tensor own;
    void *at = nullptr;
    size_t bytes = 0;
    void lent(PyObject *o, int index) {
        const at::Tensor &t = tensor(o, "workspace");
        if (!t.is_contiguous() || t.get_device() != index)
            fail(PyExc_ValueError, "workspace must be a contiguous tensor on cuda:%d", index);
        at = t.data_ptr();
        bytes = t.nbytes();
    }
    void make(size_t n, int index) {
        if (n == 0) return;
        own = fresh((int64_t)n, at::kByte, index);
        at = own.data_ptr();
        bytes = n;
    }
};

// Runs f(stream) on the current stream of device `index`, without the interpreter's lock.
template <typename F>
void call(int index, const char *where, F f) {
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != index) guard.set_index((c10::DeviceIndex)index);
    cudaStream_t stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f(stream);
    Py_END_ALLOW_THREADS
    if (status != ATTN_OK) fail_status(status, where);
}

void expect(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) fail(PyExc_TypeError, "expected %d arguments, got %d", (int)want, (int)got);
}

PyObject *pair(THPObjectPtr &a, THPObjectPtr &b) { return PyTuple_Pack(2, a.get(), b.get()); }

// append(cache, k, v, lens, new_lens)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    expect(n_args, 5);
    const Cache &c = cache_of(args[0]);
    const at::Tensor &k = four(args[1], "k"), &v = tensor(args[2], "v");
    const int64_t batch[] = {c.c.B}, n = k.size(2), shape[] = {c.c.B, c.c.H, n, c.c.D};
    attn_strides strides[2];
    const void *kp = view(k, "k", shape, c.index, strides[0]), *vp = view(v, "v", shape, c.index, strides[1]);
    const auto *lens = whole<int32_t>(args[3], "lens", at::kInt, batch, c.index);
    const auto *new_lens = args[4] == Py_None ? nullptr : whole<int32_t>(args[4], "new_lens", at::kInt, batch, c.index);
    if (n > INT32_MAX) fail_status(ATTN_ERR_SHAPE, "attn_q8_append");
    const bool plain = k.is_contiguous() && v.is_contiguous();
    call(c.index, "attn_q8_append", [&](cudaStream_t stream) {
        return api.append(&c.c, kp, vp, (int)n, lens, new_lens, plain ? nullptr : strides, stream);
    });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// read(cache, lens, n, starts, k, v) -> (k, v)
PyObject *read(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    expect(n_args, 6);
    const Cache &c = cache_of(args[0]);
    const int n = number(args[2], 1, ATTN_Q8_BLOCK * (kMaxBlocks + 1), "attn_q8_read");
    const int64_t batch[] = {c.c.B}, shape[] = {c.c.B, c.c.H, n, c.c.D};
    const auto *lens = whole<int32_t>(args[1], "lens", at::kInt, batch, c.index);
    const auto *starts = args[3] == Py_None ? nullptr : whole<int32_t>(args[3], "starts", at::kInt, batch, c.index);
    THPObjectPtr k, v;
    void *kp = output<void>(args[4], "k", at::kBFloat16, shape, c.index, k);
    void *vp = output<void>(args[5], "v", at::kBFloat16, shape, c.index, v);
    call(c.index, "attn_q8_read",
         [&](cudaStream_t stream) { return api.read(&c.c, lens, starts, n, kp, vp, stream); });
    return pair(k, v);
    END_HANDLE_TH_ERRORS
}

// decode(cache, q, lens, o, lse, scale, blocks, weight, workspace) -> (o, lse)
PyObject *decode(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    expect(n_args, 9);
    const Cache &c = cache_of(args[0]);
    const at::Tensor &q = four(args[1], "q");
    const int64_t batch[] = {c.c.B}, H = q.size(1), Tq = q.size(2), shape[] = {c.c.B, H, Tq, c.c.D};
    attn_strides strides[2];
    const void *qp = view(q, "q", shape, c.index, strides[0]);
    const auto *lens = whole<int32_t>(args[2], "lens", at::kInt, batch, c.index);
    if (H > INT32_MAX || Tq > ATTN_DECODE_MAX_QUERIES) fail_status(ATTN_ERR_SHAPE, "attn_q8_decode");
    bool plain = q.is_contiguous();
    THPObjectPtr o, lse;
    void *op;
    if (args[3] == Py_None) {
        op = output<void>(args[3], "o", at::kBFloat16, shape, c.index, o);
        strides[1] = attn_strides{H * Tq * c.c.D, Tq * c.c.D, c.c.D};
    } else {
        const at::Tensor &t = tensor(args[3], "o");
        op = view(t, "o", shape, c.index, strides[1]);
        plain = plain && t.is_contiguous();
        Py_INCREF(args[3]);
        o = args[3];
    }
    auto *lp = output<float>(args[4], "lse", at::kFloat, at::IntArrayRef(shape, 3), c.index, lse);
    double scale = 1.0 / std::sqrt((double)c.c.D);
    if (args[5] != Py_None) {
        scale = PyFloat_AsDouble(args[5]);
        if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    }
    attn_q8_decode_options opts{nullptr, 0, number(args[7], ATTN_Q8_WEIGHT_NONE, ATTN_Q8_WEIGHT_ADD, "attn_q8_decode")};
    if (args[6] != Py_None) {
        if (!THPVariable_Check(args[6]) || tensor(args[6], "blocks").dim() != 4 || tensor(args[6], "blocks").size(3) < 1)
            fail(PyExc_ValueError, "blocks must be a [B, H, Tq, n] tensor");
        const int64_t n = tensor(args[6], "blocks").size(3), lists[] = {c.c.B, c.c.H, Tq, n};
        opts.blocks = whole<int32_t>(args[6], "blocks", at::kInt, lists, c.index);
        if (n > kMaxBlocks) fail_status(ATTN_ERR_OPTION, "attn_q8_decode");
        opts.blocks_n = (int32_t)n;
    }
    Workspace ws;
    if (args[8] != Py_None)
        ws.lent(args[8], c.index);
    else
        ws.make(api.decode_workspace_bytes(&c.c, (int)H, (int)Tq, &opts), c.index);
    call(c.index, "attn_q8_decode", [&](cudaStream_t stream) {
        return api.decode(&c.c, qp, op, lp, lens, (int)H, (int)Tq, (float)scale, plain ? nullptr : strides, &opts, ws.at,
                          ws.bytes, stream);
    });
    return pair(o, lse);
    END_HANDLE_TH_ERRORS
}

// select(cache, q, lens, n, blocks) -> blocks
PyObject *select(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    expect(n_args, 5);
    const Cache &c = cache_of(args[0]);
    const at::Tensor &q = four(args[1], "q");
    const int n = number(args[3], 1, kMaxBlocks, "attn_q8_select");
    const int64_t batch[] = {c.c.B}, H = q.size(1), Tq = q.size(2), shape[] = {c.c.B, H, Tq, c.c.D};
    attn_strides strides;
    const void *qp = view(q, "q", shape, c.index, strides);
    const auto *lens = whole<int32_t>(args[2], "lens", at::kInt, batch, c.index);
    if (H > INT32_MAX || Tq > ATTN_DECODE_MAX_QUERIES) fail_status(ATTN_ERR_SHAPE, "attn_q8_select");
    const int64_t lists[] = {c.c.B, c.c.H, Tq, n};
    THPObjectPtr blocks;
    auto *bp = output<int32_t>(args[4], "blocks", at::kInt, lists, c.index, blocks);
    const bool plain = q.is_contiguous();
    call(c.index, "attn_q8_select", [&](cudaStream_t stream) {
        return api.select(&c.c, qp, lens, bp, n, (int)H, (int)Tq, plain ? nullptr : &strides, stream);
    });
    return blocks.release();
    END_HANDLE_TH_ERRORS
}

// evict(cache, out, lens, keep, sink, recent, lens_out, kept, workspace) -> (lens_out, kept)
PyObject *evict(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    expect(n_args, 9);
    const char *where = "attn_q8_evict";
    const Cache &c = cache_of(args[0]), &d = cache_of(args[1]);
    if (d.index != c.index) fail(PyExc_ValueError, "out must be on cuda:%d, got cuda:%d", c.index, d.index);
    const int keep = number(args[3], 1, kMaxBlocks, where), sink = number(args[4], 0, kMaxBlocks, where),
              recent = number(args[5], 0, kMaxBlocks, where);
    const int64_t batch[] = {c.c.B}, shape[] = {c.c.B, c.c.H, keep};
    const auto *lens = whole<int32_t>(args[2], "lens", at::kInt, batch, c.index);
    THPObjectPtr lens_out, kept;
    auto *op = output<int32_t>(args[6], "lens_out", at::kInt, batch, c.index, lens_out);
    auto *kp = output<int32_t>(args[7], "kept", at::kInt, shape, c.index, kept);
    Workspace ws;
    if (args[8] != Py_None)
        ws.lent(args[8], c.index);
    else if (op == lens)  // the only case that needs one
        ws.make(api.evict_workspace_bytes(&c.c), c.index);
    call(c.index, where, [&](cudaStream_t stream) {
        return api.evict(&c.c, &d.c, lens, op, kp, keep, sink, recent, ws.at, ws.bytes, stream);
    });
    return pair(lens_out, kept);
    END_HANDLE_TH_ERRORS
}

// cache(address of an attn_q8_cache, device index): a capsule with a copy of it.
PyObject *cache(PyObject *, PyObject *args) {
    unsigned long long at;
    int index;
    if (!PyArg_ParseTuple(args, "Ki", &at, &index)) return nullptr;
    auto *c = new (std::nothrow) Cache{*reinterpret_cast<const attn_q8_cache *>((uintptr_t)at), index};
    if (!c) return PyErr_NoMemory();
    PyObject *capsule = PyCapsule_New(
        c, kCapsule, [](PyObject *o) { delete static_cast<Cache *>(PyCapsule_GetPointer(o, kCapsule)); });
    if (!capsule) delete c;
    return capsule;
}

// bind(AttnError, addresses of libattn.so's functions in Api's order)
PyObject *bind(PyObject *, PyObject *args) {
    PyObject *error;
    unsigned long long f[7];
    if (!PyArg_ParseTuple(args, "OKKKKKKK", &error, f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6)) return nullptr;
    static_assert(sizeof(Api) == sizeof(f), "one address a function");
    std::memcpy(&api, f, sizeof(api));
    Py_INCREF(error);
    Py_XDECREF(error_class);
    error_class = error;
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

}  // namespace

PyMODINIT_FUNC PyInit__q8() {
    static PyMethodDef methods[] = {{"append", fast<append>(), METH_FASTCALL, nullptr},
                                    {"read", fast<read>(), METH_FASTCALL, nullptr},
                                    {"decode", fast<decode>(), METH_FASTCALL, nullptr},
                                    {"select", fast<select>(), METH_FASTCALL, nullptr},
                                    {"evict", fast<evict>(), METH_FASTCALL, nullptr},
                                    {"cache", cache, METH_VARARGS, nullptr},
                                    {"bind", bind, METH_VARARGS, nullptr},
                                    {nullptr, nullptr, 0, nullptr}};
    static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q8", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
    PyObject *m = PyModule_Create(&module);
    // build.py looks for these words in the file, the package compares them with the torch and the Python it runs in
    static const char words[] = "built for " ATTN_BUILT_FOR;
    if (m && PyModule_AddStringConstant(m, "built_for", words + sizeof("built for ") - 1) < 0) Py_CLEAR(m);
    return m;
}
