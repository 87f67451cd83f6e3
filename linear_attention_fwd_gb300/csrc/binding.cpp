// Python binding of the linear-attention and paged-cache calls: argument checks, output allocation and the
// current stream, in C++.  A decode step's calls take a few microseconds on the GPU; the same work done
// in Python around ctypes cost 8 to 20 us of host time per call, here 3 to 6.
//
// The library itself is reached through the addresses that `bind` is given, so that the module works with
// whichever build of it the Python side has loaded.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <initializer_list>
#include <optional>

#include "../../include/kda.h"

namespace {

decltype(&kda_lin_chunk_fwd) f_chunk;
decltype(&kda_lin_chunk_fwd_workspace_bytes) f_chunk_bytes;
decltype(&kda_lin_recurrent_step) f_step;
decltype(&kda_paged_append) f_append;
decltype(&kda_paged_attention) f_attend;
decltype(&kda_paged_attention_workspace_bytes) f_attend_bytes;
PyObject *raise_status;   // called with (status, name); raises

struct Refused {};        // a Python error is set

[[noreturn]] void refuse(PyObject *type, const char *form, ...) {
    va_list args;
    va_start(args, form);
    PyErr_FormatV(type, form, args);
    va_end(args);
    throw Refused{};
}

using Shape = std::initializer_list<int64_t>;

// An argument that may be None.
struct Arg {
    const at::Tensor *t = nullptr;
    const char *name;
    Arg(PyObject *o, const char *n) : name(n) {
        if (o == Py_None) return;
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor, got %s", n, Py_TYPE(o)->tp_name);
        t = &THPVariable_Unpack(o);
    }
    explicit operator bool() const { return t != nullptr; }
    void *ptr() const { return t ? t->data_ptr() : nullptr; }
    int64_t size(int64_t d) const { return t->size(d); }
    const Arg &need(int64_t dims, const char *what) const {
        if (!t || t->dim() != dims) refuse(PyExc_ValueError, "%s must be %s", name, what);
        return *this;
    }
    // a contiguous tensor of this type and shape on the CUDA device (nothing to check where it is None)
    void check(at::ScalarType type, int dev, Shape shape) const {
        if (!t) return;
        if (t->scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t->scalar_type()));
        if (!t->is_cuda() || t->get_device() != dev) refuse(PyExc_ValueError, "%s must be on cuda:%d", name, dev);
        if (!t->sizes().equals(at::IntArrayRef(shape))) {
            std::string want, got;
            for (const int64_t x : shape) want += (want.empty() ? "" : ", ") + std::to_string(x);
            for (const int64_t x : t->sizes()) got += (got.empty() ? "" : ", ") + std::to_string(x);
            refuse(PyExc_ValueError, "%s must have shape (%s), got (%s)", name, want.c_str(), got.c_str());
        }
        if (!t->is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    }
};

int device_of(const Arg &a) {
    if (!a.t->is_cuda()) refuse(PyExc_ValueError, "%s must be on a CUDA device", a.name);
    const int dev = a.t->get_device();
    if (dev != c10::cuda::current_device()) refuse(PyExc_ValueError, "%s must be on the current CUDA device", a.name);
    return dev;
}

kda_dtype_t dtype_of(const Arg &a) {
    switch (a.t->scalar_type()) {
        case at::kFloat: return KDA_F32;
        case at::kBFloat16: return KDA_BF16;
        default: refuse(PyExc_TypeError, "unsupported dtype %s (fp32 or bf16)", c10::toString(a.t->scalar_type()));
    }
}

// The caller's stream (a handle, or None: the current one).  Tensors are allocated for it: memory that the
// allocator hands out for another stream may still be in use there.
struct Stream {
    int dev;
    cudaStream_t handle;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    Stream(PyObject *o, int device) : dev(device) {
        if (o == Py_None) {
            handle = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
            return;
        }
        handle = static_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
        if (PyErr_Occurred()) throw Refused{};
        guard.emplace(c10::cuda::getStreamFromExternal(handle, (c10::DeviceIndex)device));
    }
    at::Tensor make(Shape shape, at::ScalarType type) const {
        return at::detail::empty_cuda(at::IntArrayRef(shape), type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
    }
};

int32_t narrow(int64_t x, const char *what) {
    if (x > 0x7fffffffLL) refuse(PyExc_ValueError, "%s is too large", what);
    return (int32_t)x;
}

bool truth(PyObject *o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw Refused{};   // (asking raised)
    return r != 0;
}

void finish(kda_status_t st, const char *name) {
    if (st == KDA_OK) return;
    PyObject *r = PyObject_CallFunction(raise_status, "is", (int)st, name);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
    throw Refused{};
}

// `given`, or a new tensor in `made`
const at::Tensor *or_made(const Arg &given, at::Tensor &made, const Stream &s, Shape shape, at::ScalarType type) {
    if (given) return given.t;
    made = s.make(shape, type);
    return &made;
}

PyObject *wrap(PyObject *given, const at::Tensor &made) {
    if (given != Py_None) return Py_NewRef(given);
    return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(Py_None);
}

PyObject *pair(PyObject *a, PyObject *b) {
    PyObject *r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

void count(Py_ssize_t n, Py_ssize_t want, const char *name) {
    if (n != want) refuse(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
}

template <typename F> PyObject *guarded(F body) {
    HANDLE_TH_ERRORS
    try {
        return body();
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (q, k, v, g, head_g, initial_state, cu_seqlens, out, final_state, want_final, workspace, stream)
PyObject *lin_chunk(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 12, "lin_chunk");
        const Arg q(a[0], "q"), k(a[1], "k"), v(a[2], "v"), g(a[3], "g"), hg(a[4], "head_g"), s0(a[5], "initial_state");
        const Arg cu(a[6], "cu_seqlens"), out(a[7], "out"), fin(a[8], "final_state"), ws(a[10], "workspace");
        q.need(4, "[B, T, Hk, dk]"), v.need(4, "[B, T, H, dv]"), k.need(4, "shaped like q");
        const int dev = device_of(q);
        const kda_dtype_t code = dtype_of(q);
        const at::ScalarType dt = q.t->scalar_type();
        const int64_t B = q.size(0), T = q.size(1), Hk = q.size(2), dk = q.size(3), H = v.size(2), dv = v.size(3);
        int64_t N = B;
        if (cu) {
            N = cu.t->numel() - 1;
            if (N < 1) refuse(PyExc_ValueError, "cu_seqlens must be [N + 1] with N >= 1");
        }
        q.check(dt, dev, {B, T, Hk, dk});
        k.check(dt, dev, {B, T, Hk, dk});
        v.check(dt, dev, {B, T, H, dv});
        g.check(at::kFloat, dev, {B, T, H});
        hg.check(at::kFloat, dev, {H});
        s0.check(at::kFloat, dev, {N, H, dk, dv});
        cu.check(at::kInt, dev, {N + 1});
        out.check(dt, dev, {B, T, H, dv});
        fin.check(at::kFloat, dev, {N, H, dk, dv});
        if (ws) ws.check(at::kByte, dev, {ws.t->numel()});
        const kda_lin_dims_t d{narrow(B, "B"), narrow(T, "T"), narrow(N, "N"), narrow(H, "H"), narrow(Hk, "Hk"), narrow(dk, "dk"), narrow(dv, "dv"), code};
        const Stream s(a[11], dev);
        at::Tensor o, f, w;
        const at::Tensor *op = or_made(out, o, s, {B, T, H, dv}, dt), *fp = nullptr;
        if (fin || truth(a[9])) fp = or_made(fin, f, s, {N, H, dk, dv}, at::kFloat);
        const at::Tensor *wp = ws.t;
        if (!wp)
            if (const size_t bytes = f_chunk_bytes(&d, cu ? 1 : 0)) wp = or_made(ws, w, s, {(int64_t)bytes}, at::kByte);
        finish(f_chunk(q.ptr(), k.ptr(), v.ptr(), static_cast<const float *>(g.ptr()), static_cast<const float *>(hg.ptr()),
                       static_cast<const float *>(s0.ptr()), static_cast<const int32_t *>(cu.ptr()), op->data_ptr(),
                       fp ? static_cast<float *>(fp->data_ptr()) : nullptr, wp ? wp->data_ptr() : nullptr, wp ? (size_t)wp->numel() : 0, &d, s.handle),
               "kda_lin_chunk_fwd");
        return pair(wrap(a[7], o), wrap(a[8], f));
    });
}

// (q, k, v, g, head_g, state, state_indices, out, stream)
PyObject *lin_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 9, "lin_step");
        const Arg q(a[0], "q"), k(a[1], "k"), v(a[2], "v"), g(a[3], "g"), hg(a[4], "head_g"), state(a[5], "state"), idx(a[6], "state_indices"), out(a[7], "out");
        q.need(3, "[N, Hk, dk]"), v.need(3, "[N, H, dv]"), state.need(4, "[P, H, dk, dv]"), k.need(3, "shaped like q");
        const int dev = device_of(q);
        const kda_dtype_t code = dtype_of(q);
        const at::ScalarType dt = q.t->scalar_type();
        const int64_t N = q.size(0), Hk = q.size(1), dk = q.size(2), H = v.size(1), dv = v.size(2), slots = state.size(0);
        q.check(dt, dev, {N, Hk, dk});
        k.check(dt, dev, {N, Hk, dk});
        v.check(dt, dev, {N, H, dv});
        g.check(at::kFloat, dev, {N, H});
        hg.check(at::kFloat, dev, {H});
        state.check(at::kFloat, dev, {slots, H, dk, dv});
        idx.check(at::kInt, dev, {N});
        out.check(dt, dev, {N, H, dv});
        const kda_lin_dims_t d{narrow(N, "N"), 1, narrow(slots, "P"), narrow(H, "H"), narrow(Hk, "Hk"), narrow(dk, "dk"), narrow(dv, "dv"), code};
        const Stream s(a[8], dev);
        at::Tensor o;
        const at::Tensor *op = or_made(out, o, s, {N, H, dv}, dt);
        finish(f_step(q.ptr(), k.ptr(), v.ptr(), static_cast<const float *>(g.ptr()), static_cast<const float *>(hg.ptr()),
                      static_cast<float *>(state.ptr()), static_cast<const int32_t *>(idx.ptr()), op->data_ptr(), &d, s.handle),
               "kda_lin_recurrent_step");
        return wrap(a[7], o);
    });
}

kda_paged_dims_t paged_dims(const Arg &kc, const Arg &vc, const Arg &table, int64_t rows, int64_t heads, at::ScalarType dt, kda_dtype_t code, int dev) {
    kc.need(4, "[pages, page_size, Hkv, d]"), vc.need(4, "shaped like k_cache"), table.need(2, "[N, max_pages]");
    const int64_t pages = kc.size(0), ps = kc.size(1), hkv = kc.size(2), d = kc.size(3), width = table.size(1);
    kc.check(dt, dev, {pages, ps, hkv, d});
    vc.check(dt, dev, {pages, ps, hkv, d});
    table.check(at::kInt, dev, {rows, width});
    return {narrow(rows, "N"), narrow(heads ? heads : hkv, "Hq"), narrow(hkv, "Hkv"), narrow(d, "d"), narrow(pages, "pages"), narrow(ps, "page_size"),
            narrow(width, "max_pages"), code};
}

// (k, v, k_cache, v_cache, block_table, positions, cu_seqlens, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 8, "append");
        const Arg k(a[0], "k"), v(a[1], "v"), kc(a[2], "k_cache"), vc(a[3], "v_cache"), table(a[4], "block_table"), pos(a[5], "positions"), cu(a[6], "cu_seqlens");
        k.need(3, "[tokens, Hkv, d]"), v.need(3, "shaped like k"), pos.need(1, "[N]");
        const int dev = device_of(k);
        const at::ScalarType dt = k.t->scalar_type();
        const int64_t N = pos.size(0), tokens = k.size(0);
        const kda_paged_dims_t d = paged_dims(kc, vc, table, N, 0, dt, dtype_of(k), dev);
        k.check(dt, dev, {tokens, d.kv_heads, d.head_dim});
        v.check(dt, dev, {tokens, d.kv_heads, d.head_dim});
        pos.check(at::kInt, dev, {N});
        cu.check(at::kInt, dev, {N + 1});
        const Stream s(a[7], dev);
        finish(f_append(k.ptr(), v.ptr(), kc.ptr(), vc.ptr(), static_cast<const int32_t *>(table.ptr()), static_cast<const int32_t *>(pos.ptr()),
                        static_cast<const int32_t *>(cu.ptr()), tokens, &d, s.handle),
               "kda_paged_append");
        return Py_NewRef(Py_None);
    });
}

// (q, k_cache, v_cache, block_table, seq_lens, scale, out, lse, want_lse, workspace, stream)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 11, "attend");
        const Arg q(a[0], "q"), kc(a[1], "k_cache"), vc(a[2], "v_cache"), table(a[3], "block_table"), lens(a[4], "seq_lens");
        const Arg out(a[6], "out"), lse(a[7], "lse"), ws(a[9], "workspace");
        q.need(3, "[N, Hq, d]"), lens.need(1, "[N]");
        const int dev = device_of(q);
        const at::ScalarType dt = q.t->scalar_type();
        const int64_t N = q.size(0), Hq = q.size(1);
        kda_paged_dims_t d = paged_dims(kc, vc, table, N, Hq, dt, dtype_of(q), dev);
        d.heads = narrow(Hq, "Hq");
        q.check(dt, dev, {N, Hq, d.head_dim});
        lens.check(at::kInt, dev, {N});
        out.check(dt, dev, {N, Hq, d.head_dim});
        lse.check(at::kFloat, dev, {N, Hq});
        if (ws) ws.check(at::kByte, dev, {ws.t->numel()});
        const double scale = PyFloat_AsDouble(a[5]);
        if (PyErr_Occurred()) throw Refused{};
        const Stream s(a[10], dev);
        at::Tensor o, l, w;
        const at::Tensor *op = or_made(out, o, s, {N, Hq, d.head_dim}, dt), *lp = nullptr;
        if (lse || truth(a[8])) lp = or_made(lse, l, s, {N, Hq}, at::kFloat);
        const at::Tensor *wp = ws.t;
        if (!wp)
            if (const size_t bytes = f_attend_bytes(&d)) wp = or_made(ws, w, s, {(int64_t)bytes}, at::kByte);
        finish(f_attend(q.ptr(), kc.ptr(), vc.ptr(), static_cast<const int32_t *>(table.ptr()), static_cast<const int32_t *>(lens.ptr()), (float)scale,
                        op->data_ptr(), lp ? static_cast<float *>(lp->data_ptr()) : nullptr, wp ? wp->data_ptr() : nullptr,
                        wp ? (size_t)wp->numel() : 0, &d, s.handle),
               "kda_paged_attention");
        return pair(wrap(a[6], o), wrap(a[7], l));
    });
}

// (raise_status, six addresses in the order of the declarations above)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 7, "bind");
        void *p[6];
        for (int i = 0; i < 6; ++i) p[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (PyErr_Occurred()) throw Refused{};
        f_chunk = reinterpret_cast<decltype(f_chunk)>(p[0]);
        f_chunk_bytes = reinterpret_cast<decltype(f_chunk_bytes)>(p[1]);
        f_step = reinterpret_cast<decltype(f_step)>(p[2]);
        f_append = reinterpret_cast<decltype(f_append)>(p[3]);
        f_attend = reinterpret_cast<decltype(f_attend)>(p[4]);
        f_attend_bytes = reinterpret_cast<decltype(f_attend_bytes)>(p[5]);
        Py_XSETREF(raise_status, Py_NewRef(a[0]));
        return Py_NewRef(Py_None);
    });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(lin_chunk), METHOD(lin_step), METHOD(append), METHOD(attend), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
