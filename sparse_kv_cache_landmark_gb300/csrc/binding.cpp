// Native Python binding of the context-free serving calls (kvo_rope, kvo_paged_append, kvo_paged_attn,
// kvo_prompt_attn): argument checks, output allocation and stream lookup, then the C ABI.
//
// A decode loop makes these calls once per layer and token, where the same checks written in Python cost more
// host time (about 10 us a call on the Grace host) than the GPU takes.  Nothing is kept between calls.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <string>
#include <vector>

#include "kvo.h"

namespace {

PyObject* g_error = nullptr;       // KvoError(status, message)

struct Refused {
    int status;
    std::string what;
};
struct PythonError {};             // a Python exception is already set

[[noreturn]] void refuse(const std::string& what) { throw Refused{KVO_ERR_INVALID, what}; }

std::string shape_text(at::IntArrayRef s) {
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}
const char* dtype_text(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kFloat: return "torch.float32";
        case at::kByte: return "torch.uint8";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        default: return c10::toString(t);
    }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (o == Py_None) refuse(std::string(name) + " is required");
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
// Every buffer of a call is on the device of its first one.
void on_device(const at::Tensor& t, const char* name, const at::Device& dev) {
    if (t.device() != dev)
        refuse(std::string("all buffers must be on one CUDA device: ") + name + " is on " + t.device().str());
}
void of_type(const at::Tensor& t, const char* name, at::ScalarType dt) {
    if (t.scalar_type() != dt)
        refuse(std::string(name) + " must be " + dtype_text(dt) + ", got " + dtype_text(t.scalar_type()));
}
// A contiguous buffer.
const at::Tensor& need(PyObject* o, const char* name, const at::Device& dev, at::ScalarType dt,
                       std::optional<at::IntArrayRef> shape = std::nullopt) {
    const at::Tensor& t = tensor(o, name);
    of_type(t, name, dt);
    if (shape && t.sizes() != *shape)
        refuse(std::string(name) + " must have shape " + shape_text(*shape) + ", got " + shape_text(t.sizes()));
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    on_device(t, name, dev);
    return t;
}
// A bf16 [tokens][heads][d] buffer whose token stride (and head stride, where `free_heads`) is free.
struct Rows {
    const at::Tensor& t;
    int64_t tok, head;
};
Rows rows(PyObject* o, const char* name, const at::Device& dev, bool free_heads = false) {
    const at::Tensor& t = tensor(o, name);
    of_type(t, name, at::kBFloat16);
    if (t.dim() != 3) refuse(std::string(name) + " must be [tokens][heads][head_dim], got " + shape_text(t.sizes()));
    on_device(t, name, dev);
    const int64_t T = t.size(0), H = t.size(1), d = t.size(2);
    const int64_t head = H > 1 ? t.stride(1) : d;             // a dimension of one has no stride of its own
    const int64_t tok = T > 1 ? t.stride(0) : std::max(H * head, d);
    if (d > 1 && t.stride(2) != 1) refuse(std::string(name) + ": the last dimension must be contiguous");
    if (head != d && !free_heads) refuse(std::string(name) + ": heads must be contiguous");
    return {t, tok, head};
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError{};
    return v;
}
float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return (float)v;
}
int int32_size(int64_t v, const char* name) {
    if (v > INT32_MAX) refuse(std::string(name) + " must fit in 31 bits");
    return (int)v;
}

// The stream of a call: torch's current stream of the device, or the torch stream or raw handle that was given.  A
// given stream is made current for the call, so that outputs and workspace come from its own memory pool: a block of
// another stream's pool could still be in use there, or be handed out again while this call runs.
struct Stream {
    kvo_stream_t handle;                         // the legacy default stream by its name, cudaStreamLegacy
    c10::cuda::OptionalCUDAStreamGuard guard;

    Stream(PyObject* o, const at::Device& dev) {
        if (!dev.is_cuda()) refuse("all buffers must be on one CUDA device, got " + dev.str());
        uintptr_t h = 0;
        if (o == Py_None) {
            h = (uintptr_t)c10::cuda::getCurrentCUDAStream(dev.index()).stream();
        } else {
            PyObject* a = PyObject_GetAttrString(o, "cuda_stream");
            if (!a) {
                PyErr_Clear();
                a = o;
                Py_INCREF(a);
            }
            h = (uintptr_t)PyLong_AsUnsignedLongLong(a);
            Py_DECREF(a);
            if (PyErr_Occurred()) throw PythonError{};
            const bool legacy = h <= 1;
            guard.reset_stream(legacy ? c10::cuda::getDefaultCUDAStream(dev.index())
                                      : c10::cuda::getStreamFromExternal((cudaStream_t)h, dev.index()));
        }
        handle = (kvo_stream_t)(h ? h : 1);
    }
};

// Runs a C call with the device current; raises on any status but KVO_OK.
template <typename F>
void launch(const at::Device& dev, F&& call) {
    const c10::cuda::CUDAGuard guard(dev);
    const kvo_status st = call();
    if (st != KVO_OK) throw Refused{st, kvo_last_error(nullptr)};
}

// From torch's allocator, past the dispatcher (0.4 us less a tensor on the Grace host).
at::Tensor empty(at::IntArrayRef shape, at::ScalarType dt, const at::Device& dev) {
    return at::TensorBase(at::detail::empty_cuda(shape, dt, dev, std::nullopt));
}

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& body) {
    try {
        if (got != want) {
            PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
            return nullptr;
        }
        return body();
    } catch (const Refused& r) {
        if (PyObject* e = PyObject_CallFunction(g_error ? g_error : PyExc_RuntimeError, "is", r.status, r.what.c_str())) {
            PyErr_SetObject((PyObject*)Py_TYPE(e), e);
            Py_DECREF(e);
        }
    } catch (const PythonError&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject* x = THPVariable_Wrap(a);
    PyObject* y = THPVariable_Wrap(b);
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

// rope(x, pos, freq, interleaved, amplitude, out, stream)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Device dev = tensor(a[0], "x").device();
        const Rows x = rows(a[0], "x", dev, true);
        const int64_t T = x.t.size(0), H = x.t.size(1), d = x.t.size(2);
        const at::Tensor& pos = need(a[1], "pos", dev, at::kInt, {{T}});
        const at::Tensor& freq = need(a[2], "freq", dev, at::kLong);
        const bool inter = truth(a[3]);
        const float amp = number(a[4]);
        const Stream stream(a[6], dev);
        at::Tensor out;
        int64_t tok = H * d, head = d;
        if (a[5] == Py_None) {
            out = empty({T, H, d}, at::kBFloat16, dev);
        } else {
            const Rows o = rows(a[5], "out", dev, true);
            if (o.t.sizes() != x.t.sizes())
                refuse("out must have shape " + shape_text(x.t.sizes()) + ", got " + shape_text(o.t.sizes()));
            out = o.t;
            tok = o.tok;
            head = o.head;
        }
        launch(dev, [&] {
            return kvo_rope(x.t.data_ptr(), x.tok, x.head, out.data_ptr(), tok, head, (const int32_t*)pos.data_ptr(),
                            (const uint64_t*)freq.data_ptr(), T, int32_size(H, "heads"), int32_size(d, "head_dim"),
                            int32_size(2 * freq.numel(), "freq"), inter, amp, stream.handle);
        });
        return THPVariable_Wrap(out);
    });
}

// The checked descriptor of pools [n_pages][Hkv][page_size][d] and a table [batch][max_pages].
kvo_paged_cache paged(PyObject* kp, PyObject* vp, PyObject* ks, PyObject* vs, PyObject* table, const at::Device& dev) {
    const at::Tensor& k = tensor(kp, "k_pages");
    const at::Tensor& t = tensor(table, "table");
    if (k.dim() != 4 || t.dim() != 2)
        refuse("pages must be [n_pages][n_kv_heads][page_size][head_dim], table [batch][max_pages]");
    const at::ScalarType dt = k.scalar_type();
    if (dt != at::kBFloat16 && dt != at::kFloat8_e4m3fn)
        refuse(std::string("pages must be bfloat16 or float8_e4m3fn, got ") + dtype_text(dt));
    kvo_paged_cache c{};
    c.k_pages = need(kp, "k_pages", dev, dt).data_ptr();
    c.v_pages = need(vp, "v_pages", dev, dt, k.sizes()).data_ptr();
    c.table = (const int32_t*)need(table, "table", dev, at::kInt).data_ptr();
    if (dt == at::kFloat8_e4m3fn) {
        const std::vector<int64_t> s{k.size(0), k.size(1)};
        c.k_scale = (float*)need(ks, "k_scale", dev, at::kFloat, at::IntArrayRef(s)).data_ptr();
        c.v_scale = (float*)need(vs, "v_scale", dev, at::kFloat, at::IntArrayRef(s)).data_ptr();
        c.format = KVO_PAGES_E4M3;
    }
    c.batch = int32_size(t.size(0), "batch");
    c.max_pages = int32_size(t.size(1), "max_pages");
    c.n_pages = int32_size(k.size(0), "n_pages");
    c.n_kv_heads = int32_size(k.size(1), "n_kv_heads");
    c.page_size = int32_size(k.size(2), "page_size");
    c.head_dim = int32_size(k.size(3), "head_dim");
    return c;
}
int32_t* status_of(PyObject* o, const at::Device& dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = need(o, "status", dev, at::kInt);
    if (t.numel() < 1) refuse("status must hold one value");
    return (int32_t*)t.data_ptr();
}

// paged_append(k, v, k_pages, v_pages, table, start, cu, k_scale, v_scale, freq, interleaved, amplitude, q, q_out,
//              k_out, status, stream)
PyObject* py_paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 17, [&]() -> PyObject* {
        const at::Device dev = tensor(a[2], "k_pages").device();
        const kvo_paged_cache c = paged(a[2], a[3], a[7], a[8], a[4], dev);
        const Rows k = rows(a[0], "k", dev), v = rows(a[1], "v", dev);
        const int64_t T = k.t.size(0);
        const std::vector<int64_t> shape{T, c.n_kv_heads, c.head_dim};
        if (k.t.sizes() != at::IntArrayRef(shape) || v.t.sizes() != at::IntArrayRef(shape))
            refuse("k and v must have shape " + shape_text(shape) + ", got " + shape_text(k.t.sizes()) + " and " +
                   shape_text(v.t.sizes()));
        const int32_t* start = (const int32_t*)need(a[5], "start", dev, at::kInt, {{c.batch}}).data_ptr();
        const int32_t* cu =
            a[6] == Py_None ? nullptr : (const int32_t*)need(a[6], "cu", dev, at::kInt, {{(int64_t)c.batch + 1}}).data_ptr();
        const uint64_t* freq = nullptr;
        int rot = 0;
        if (a[9] != Py_None) {
            const at::Tensor& f = need(a[9], "freq", dev, at::kLong);
            freq = (const uint64_t*)f.data_ptr();
            rot = int32_size(2 * f.numel(), "freq");
        }
        const bool inter = truth(a[10]);
        const float amp = number(a[11]);
        const Stream stream(a[16], dev);
        const void* qp = nullptr;
        int64_t qt = 0, hq = 0;
        at::Tensor q_out;
        if (a[12] != Py_None) {
            const Rows q = rows(a[12], "q", dev);
            hq = q.t.size(1);
            const std::vector<int64_t> qs{T, hq, c.head_dim};
            if (q.t.sizes() != at::IntArrayRef(qs))
                refuse("q must have shape " + shape_text(qs) + ", got " + shape_text(q.t.sizes()));
            q_out = a[13] == Py_None ? empty(qs, at::kBFloat16, dev)
                                     : need(a[13], "q_out", dev, at::kBFloat16, at::IntArrayRef(qs));
            qp = q.t.data_ptr();
            qt = q.tok;
        }
        void* k_out = a[14] == Py_None ? nullptr : need(a[14], "k_out", dev, at::kBFloat16, at::IntArrayRef(shape)).data_ptr();
        int32_t* status = status_of(a[15], dev);
        launch(dev, [&] {
            return kvo_paged_append(&c, k.t.data_ptr(), k.tok, v.t.data_ptr(), v.tok, T, cu, start, freq, rot, inter, amp,
                                    qp, qt, int32_size(hq, "n_q_heads"), q_out.defined() ? q_out.data_ptr() : nullptr, k_out, status,
                                    stream.handle);
        });
        if (!q_out.defined()) Py_RETURN_NONE;          // (an empty q has no address)
        return THPVariable_Wrap(q_out);
    });
}

// paged_attn(q, k_pages, v_pages, table, lens, k_scale, v_scale, blocks, counts, max_len, o, lse, workspace, status,
//            stream)
PyObject* py_paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject* {
        const at::Device dev = tensor(a[1], "k_pages").device();
        const kvo_paged_cache c = paged(a[1], a[2], a[5], a[6], a[3], dev);
        const at::Tensor& q0 = tensor(a[0], "q");
        if (q0.dim() != 3) refuse("q must be [batch][n_q_heads][head_dim], got " + shape_text(q0.sizes()));
        const int64_t hq = q0.size(1), b = c.batch, hkv = c.n_kv_heads;
        const std::vector<int64_t> shape{b, hq, c.head_dim}, lshape{b, hq};
        const at::Tensor& q = need(a[0], "q", dev, at::kBFloat16, at::IntArrayRef(shape));
        const int32_t* lens = (const int32_t*)need(a[4], "lens", dev, at::kInt, {{b}}).data_ptr();
        const int32_t *blocks = nullptr, *counts = nullptr;
        int64_t n_blocks = 0;
        if (a[7] != Py_None) {
            const at::Tensor& t = need(a[7], "blocks", dev, at::kInt);
            n_blocks = t.dim() ? t.size(-1) : 0;
            if (n_blocks == 0 || t.numel() != b * hkv * n_blocks)
                refuse("blocks must be [batch][n_kv_heads][n], got " + shape_text(t.sizes()));
            blocks = (const int32_t*)t.data_ptr();
        }
        if (a[8] != Py_None) {
            if (!blocks) refuse("counts needs blocks");
            const at::Tensor& t = need(a[8], "counts", dev, at::kInt);
            if (t.numel() != b * hkv) refuse("counts must be [batch][n_kv_heads], got " + shape_text(t.sizes()));
            counts = (const int32_t*)t.data_ptr();
        }
        const int64_t max_len = integer(a[9]);
        const Stream stream(a[14], dev);
        at::Tensor o = a[10] == Py_None ? empty(shape, at::kBFloat16, dev) : need(a[10], "o", dev, at::kBFloat16, at::IntArrayRef(shape));
        at::Tensor lse = a[11] == Py_None ? empty(lshape, at::kFloat, dev) : need(a[11], "lse", dev, at::kFloat, at::IntArrayRef(lshape));
        int32_t* status = status_of(a[13], dev);
        at::Tensor ws;                 // from torch's allocator, like the outputs
        size_t bytes = 0;
        if (a[12] == Py_None) {
            const kvo_status st = kvo_paged_attn_workspace(&c, int32_size(hq, "n_q_heads"), int32_size(n_blocks, "n_blocks"), max_len, &bytes);
            if (st != KVO_OK) throw Refused{st, kvo_last_error(nullptr)};
            if (bytes) ws = empty({(int64_t)bytes}, at::kByte, dev);
        } else {
            ws = need(a[12], "workspace", dev, at::kByte);
            bytes = ws.numel();
        }
        launch(dev, [&] {
            return kvo_paged_attn(&c, q.data_ptr(), (int)hq, lens, max_len, blocks, counts, int32_size(n_blocks, "n_blocks"),
                                  o.data_ptr(), (float*)lse.data_ptr(), ws.defined() ? ws.data_ptr() : nullptr, bytes, status,
                                  stream.handle);
        });
        return pair(o, lse);
    });
}

// prompt_attn(q, k, v, cu_q, cu_k, causal, o, lse, status, stream)
PyObject* py_prompt_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const at::Device dev = tensor(a[0], "q").device();
        const Rows q = rows(a[0], "q", dev), k = rows(a[1], "k", dev), v = rows(a[2], "v", dev);
        const int64_t T = q.t.size(0), hq = q.t.size(1), d = q.t.size(2), m = k.t.size(0), hkv = k.t.size(1);
        const std::vector<int64_t> shape{T, hq, d}, lshape{T, hq}, kshape{m, hkv, d};
        if (k.t.sizes() != at::IntArrayRef(kshape) || v.t.sizes() != at::IntArrayRef(kshape))
            refuse("k and v must have shape " + shape_text(kshape) + ", got " + shape_text(k.t.sizes()) + " and " +
                   shape_text(v.t.sizes()));
        const at::Tensor& cq = need(a[3], "cu_q", dev, at::kInt);
        if (cq.dim() != 1 || cq.numel() < 1) refuse("cu_q must be [batch + 1], got " + shape_text(cq.sizes()));
        const at::Tensor& ck = a[4] == Py_None ? cq : need(a[4], "cu_k", dev, at::kInt, cq.sizes());
        const bool causal = truth(a[5]);
        const Stream stream(a[9], dev);
        at::Tensor o = a[6] == Py_None ? empty(shape, at::kBFloat16, dev) : need(a[6], "o", dev, at::kBFloat16, at::IntArrayRef(shape));
        at::Tensor lse = a[7] == Py_None ? empty(lshape, at::kFloat, dev) : need(a[7], "lse", dev, at::kFloat, at::IntArrayRef(lshape));
        int32_t* status = status_of(a[8], dev);
        launch(dev, [&] {
            return kvo_prompt_attn(q.t.data_ptr(), q.tok, k.t.data_ptr(), k.tok, v.t.data_ptr(), v.tok,
                                   (const int32_t*)cq.data_ptr(), (const int32_t*)ck.data_ptr(),
                                   int32_size(cq.numel() - 1, "batch"), T, m, int32_size(hq, "n_q_heads"),
                                   int32_size(hkv, "n_kv_heads"), int32_size(d, "head_dim"), causal, o.data_ptr(),
                                   (float*)lse.data_ptr(), status, stream.handle);
        });
        return pair(o, lse);
    });
}

// raise_with(cls): the exception class, called as cls(status, message)
PyObject* py_raise_with(PyObject*, PyObject* cls) {
    Py_XINCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"rope", (PyCFunction)(void*)py_rope, METH_FASTCALL, nullptr},
                         {"paged_append", (PyCFunction)(void*)py_paged_append, METH_FASTCALL, nullptr},
                         {"paged_attn", (PyCFunction)(void*)py_paged_attn, METH_FASTCALL, nullptr},
                         {"prompt_attn", (PyCFunction)(void*)py_prompt_attn, METH_FASTCALL, nullptr},
                         {"raise_with", py_raise_with, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvo_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvo_binding(void) { return PyModule_Create(&module); }
