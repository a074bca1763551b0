// Python calls of the paged key/value cache operators (module _bind): the checks of
// their tensors and the call of the C ABI.  A decode step makes these calls with a
// few microseconds of device work each; made from Python through ctypes their host
// side took longer than that (10 us a call, here 4).
//
// The module is given the library's functions by address (init), so it links against
// torch only.  Descriptors (csa2_kv_cache, csa2_rotary) are the package's ctypes
// structures, read through the buffer protocol.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <string>

#include "csa2.h"

namespace {

decltype(&csa2_rotate) f_rotate;
decltype(&csa2_kv_append) f_append;
decltype(&csa2_kv_attn) f_attn;
PyObject* s_index;        // "_index": the CUDA device of a descriptor's tensors
PyObject* s_cuda_stream;  // "cuda_stream"

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const std::string& why) {
    PyErr_SetString(PyExc_ValueError, why.c_str());
    throw Refused{};
}

template <class Shape>
std::string text(const Shape& shape) {
    std::ostringstream s;
    s << "(";
    for (auto n : shape) s << n << ", ";
    s << ")";
    return s.str();
}
std::string text(const at::Tensor& t) {
    std::ostringstream s;
    s << t.scalar_type() << " " << text(t.sizes()) << " on " << t.device();
    return s.str();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
        throw Refused{};
    }
    return THPVariable_Unpack(o);
}

int index_of(const at::Tensor& t) { return t.is_cuda() ? (int)t.get_device() : -1; }

void on_device(const at::Tensor& t, const char* what, int index) {
    if (index < 0 || index_of(t) != index)
        refuse(std::string(what) + " is " + text(t) + ", not on the call's CUDA device");
}

// The address of a contiguous tensor of this type and shape.
void* plain(PyObject* o, const char* what, at::ScalarType type, std::initializer_list<int64_t> shape, int index) {
    const at::Tensor& t = tensor(o, what);
    on_device(t, what, index);
    if (t.scalar_type() != type || !t.sizes().equals(at::IntArrayRef(shape)) || !t.is_contiguous()) {
        std::ostringstream s;
        s << what << " must be a contiguous " << type << " tensor of shape " << text(shape) << ", not " << text(t);
        refuse(s.str());
    }
    return t.data_ptr();
}

// csa2_heads of a [tokens][heads][channels] tensor with contiguous channels.
csa2_heads heads(const at::Tensor& t, const char* what, std::initializer_list<int64_t> shape, at::ScalarType type, int index) {
    on_device(t, what, index);
    if (t.scalar_type() != type || !t.sizes().equals(at::IntArrayRef(shape))) {
        std::ostringstream s;
        s << what << " must be " << type << " of shape " << text(shape) << ", not " << text(t);
        refuse(s.str());
    }
    for (int i = 0; i < 3; ++i)
        if (t.size(i) != (int)t.size(i)) refuse(std::string(what) + " of " + text(t.sizes()) + ": sizes are counted in 32 bits");
    if (t.size(2) > 1 && t.stride(2) != 1) refuse(std::string(what) + ": the channels must be contiguous");
    return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

int type_code(const at::Tensor& t, const char* what) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return CSA2_DTYPE_BF16;
        case at::kHalf: return CSA2_DTYPE_F16;
        case at::kFloat: return CSA2_DTYPE_F32;
        default: refuse(std::string(what) + ": " + text(t) + " is not of a supported type");
    }
}

const at::Tensor& three(PyObject* o, const char* what) {
    const at::Tensor& t = tensor(o, what);
    if (t.dim() != 3) refuse(std::string(what) + " must be [tokens][heads][channels], not " + text(t));
    return t;
}

// A ctypes structure's bytes.
template <class T>
struct Descriptor {
    Py_buffer view{};
    Descriptor(PyObject* o, const char* what, int index) {
        if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE)) throw Refused{};
        if (view.len != (Py_ssize_t)sizeof(T)) {
            PyBuffer_Release(&view);
            PyErr_Format(PyExc_TypeError, "%s is not a descriptor of its kind", what);
            throw Refused{};
        }
        if (PyObject* at = PyObject_GetAttr(o, s_index)) {
            const long i = PyLong_AsLong(at);
            Py_DECREF(at);
            if (i != index) {
                PyBuffer_Release(&view);
                PyErr_Format(PyExc_ValueError, "the tensors are on CUDA device %d, %s on %ld", index, what, i);
                throw Refused{};
            }
        } else {
            PyErr_Clear();  // made by hand: its addresses are taken as they are
        }
    }
    ~Descriptor() {
        if (view.obj) PyBuffer_Release(&view);
    }
    Descriptor(const Descriptor&) = delete;
    const T* get() const { return static_cast<const T*>(view.buf); }
};

long number(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v != (int)v) refuse("a number is out of range");
    return v;
}

csa2_stream stream_of(PyObject* stream, int index) {
    if (stream == Py_None) return reinterpret_cast<csa2_stream>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream());
    PyObject* h = PyObject_GetAttr(stream, s_cuda_stream);
    if (!h) throw Refused{};
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw Refused{};
    return reinterpret_cast<csa2_stream>(p);
}

template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, const F& f) {
    if (got != want) return PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", got, want);
    try {
        return PyLong_FromLong(f());
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// rotate(rot, x, pos, out, inverse, stream)
PyObject* py_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& x = three(a[1], "x");
        const at::Tensor& y = tensor(a[3], "out");
        const int index = index_of(x);
        const csa2_heads xd = heads(x, "x", {x.size(0), x.size(1), x.size(2)}, x.scalar_type(), index);
        const csa2_heads yd = heads(y, "out", {x.size(0), x.size(1), x.size(2)}, x.scalar_type(), index);
        const Descriptor<csa2_rotary> r(a[0], "rot", index);
        const void* pos = plain(a[2], "pos", at::kInt, {r.get()->n_axes, x.size(0)}, index);
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
        return f_rotate(r.get(), &xd, &yd, type_code(x, "x"), x.size(0), (int)x.size(1), (int)x.size(2),
                        static_cast<const int32_t*>(pos), (int)number(a[4]), stream_of(a[5], index));
    });
}

// kv_append(cache, k, v, cu, max_new, start, rotary, pos, stream)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const at::Tensor& k = three(a[1], "k");
        const at::Tensor& v = tensor(a[2], "v");
        const int index = index_of(k);
        on_device(k, "k", index);
        const Descriptor<csa2_kv_cache> c(a[0], "the cache", index);
        const int64_t total = k.size(0), batch = c.get()->batch;
        const csa2_heads kd = heads(k, "k", {total, c.get()->kv_heads, c.get()->head_dim}, k.scalar_type(), index);
        const csa2_heads vd = heads(v, "v", {total, c.get()->kv_heads, c.get()->head_dim}, k.scalar_type(), index);
        const void* cu = plain(a[3], "cu", at::kInt, {batch + 1}, index);
        const void* start = a[5] == Py_None ? nullptr : plain(a[5], "start", at::kInt, {batch}, index);
        const auto call = [&](const csa2_rotary* r) {
            const void* pos = a[7] == Py_None ? nullptr : plain(a[7], "pos", at::kInt, {r ? r->n_axes : 0, total}, index);
            const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
            return f_append(c.get(), &kd, &vd, type_code(k, "k"), static_cast<const int32_t*>(cu), (int)total, (int)number(a[4]),
                            static_cast<const int32_t*>(start), r, static_cast<const int32_t*>(pos), stream_of(a[8], index));
        };
        if (a[6] == Py_None) return call(nullptr);
        const Descriptor<csa2_rotary> r(a[6], "the rotation", index);
        return call(r.get());
    });
}

// kv_attn(cache, q, cu, max_new, scale, out, ws, lse, window, stream)
PyObject* py_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor& q = three(a[1], "q");
        const at::Tensor& out = tensor(a[5], "out");
        const int index = index_of(q);
        on_device(q, "q", index);
        const Descriptor<csa2_kv_cache> c(a[0], "the cache", index);
        const int64_t total = q.size(0), H = q.size(1);
        const csa2_heads qd = heads(q, "q", {total, H, c.get()->head_dim}, q.scalar_type(), index);
        const csa2_heads od = heads(out, "out", {total, H, c.get()->head_dim}, q.scalar_type(), index);
        const void* cu = plain(a[2], "cu", at::kInt, {c.get()->batch + 1}, index);
        void* lse = a[7] == Py_None ? nullptr : plain(a[7], "lse", at::kFloat, {total, H}, index);
        void* ws = nullptr;
        size_t ws_bytes = 0;
        if (a[6] != Py_None) {
            const at::Tensor& w = tensor(a[6], "ws");
            on_device(w, "ws", index);
            if (!w.is_contiguous()) refuse("ws must be contiguous");
            ws = w.data_ptr();
            ws_bytes = (size_t)w.numel() * w.element_size();
        }
        const double scale = PyFloat_AsDouble(a[4]);
        if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
        return f_attn(c.get(), &qd, (int)H, type_code(q, "q"), static_cast<const int32_t*>(cu), (int)total, (int)number(a[3]),
                      (float)scale, (int)number(a[8]), &od, static_cast<float*>(lse), ws, ws_bytes, stream_of(a[9], index));
    });
}

// init(csa2_rotate, csa2_kv_append, csa2_kv_attn): their addresses
PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 3) return PyErr_Format(PyExc_TypeError, "3 arguments");
    void* p[3];
    for (int i = 0; i < 3; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "an address is null");
    }
    f_rotate = reinterpret_cast<decltype(f_rotate)>(p[0]);
    f_append = reinterpret_cast<decltype(f_append)>(p[1]);
    f_attn = reinterpret_cast<decltype(f_attn)>(p[2]);
    Py_RETURN_NONE;
}

#define METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("init", py_init), METHOD("rotate", py_rotate), METHOD("kv_append", py_append),
                         METHOD("kv_attn", py_attn), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() {
    s_index = PyUnicode_InternFromString("_index");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    return s_index && s_cuda_stream ? PyModule_Create(&module) : nullptr;
}
