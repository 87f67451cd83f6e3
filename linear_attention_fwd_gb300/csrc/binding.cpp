// Python binding of the linear-attention, paged-cache and branching-decode calls: argument checks, output allocation and the
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
#include <tuple>

#include "../../include/kda.h"

namespace {

decltype(&kda_lin_chunk_fwd) f_chunk;
decltype(&kda_lin_chunk_fwd_workspace_bytes) f_chunk_bytes;
decltype(&kda_lin_recurrent_step) f_step;
decltype(&kda_paged_append) f_append;
decltype(&kda_paged_attention) f_attend;
decltype(&kda_paged_attention_workspace_bytes) f_attend_bytes;
decltype(&kda_recurrent_tree) f_tree;
decltype(&kda_recurrent_tree_qknorm) f_tree_norm;
decltype(&kda_recurrent_tree_commit) f_replay;
decltype(&kda_recurrent_tree_commit_qknorm) f_replay_norm;
decltype(&kda_paged_tree_attention) f_tree_attend;
decltype(&kda_paged_tree_attention_workspace_bytes) f_tree_attend_bytes;
decltype(&kda_paged_tree_commit) f_keep;
decltype(&kda_paged_fork) f_fork;
decltype(&kda_paged_compact) f_compact;
decltype(&kda_paged_copy) f_copy;
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
    const int32_t *ints() const { return static_cast<const int32_t *>(ptr()); }
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

// The inputs that kda_recurrent_tree (q given) and kda_recurrent_tree_commit share.
kda_dims_t tree_dims(const Arg &q, const Arg &k, const Arg &v, const Arg &g, const Arg &beta, const Arg &state, const Arg &parents, const Arg &idx, const Arg &num, int &dev) {
    k.need(4, "[N, T, H, dk]"), v.need(4, "[N, T, H, dv]"), g.need(4, "shaped like k"), beta.need(3, "[N, T, H]"), state.need(4, "[P, H, dk, dv]");
    dev = device_of(k);
    const kda_dtype_t code = dtype_of(k);
    const at::ScalarType dt = k.t->scalar_type();
    const int64_t N = k.size(0), T = k.size(1), H = k.size(2), dk = k.size(3), dv = v.size(3), slots = state.size(0);
    q.check(dt, dev, {N, T, H, dk});
    k.check(dt, dev, {N, T, H, dk});
    g.check(dt, dev, {N, T, H, dk});
    v.check(dt, dev, {N, T, H, dv});
    beta.check(dt, dev, {N, T, H});
    state.check(at::kFloat, dev, {slots, H, dk, dv});
    parents.check(at::kInt, dev, {N, T});
    idx.check(at::kInt, dev, {N});
    num.check(at::kInt, dev, {N});
    return {narrow(N, "N"), narrow(T, "T"), narrow(slots, "P"), narrow(H, "H"), narrow(dk, "dk"), narrow(dv, "dv"), code};
}

// None, or a number
std::optional<float> epsilon(PyObject *o) {
    if (o == Py_None) return std::nullopt;
    const double x = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) throw Refused{};
    return (float)x;
}

// (q, k, v, g, beta, state, parents, state_indices, num_tokens, out, qk_eps, stream)
PyObject *tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 12, "tree");
        const Arg q(a[0], "q"), k(a[1], "k"), v(a[2], "v"), g(a[3], "g"), beta(a[4], "beta"), state(a[5], "state"), parents(a[6], "parents");
        const Arg idx(a[7], "state_indices"), num(a[8], "num_tokens"), out(a[9], "out");
        q.need(4, "[N, T, H, dk]");
        int dev;
        const kda_dims_t d = tree_dims(q, k, v, g, beta, state, parents, idx, num, dev);
        const at::ScalarType dt = k.t->scalar_type();
        out.check(dt, dev, {d.batch, d.seqlen, d.heads, d.dv});
        const std::optional<float> eps = epsilon(a[10]);
        const Stream s(a[11], dev);
        at::Tensor o;
        const at::Tensor *op = or_made(out, o, s, {d.batch, d.seqlen, d.heads, d.dv}, dt);
        const float *S = static_cast<const float *>(state.ptr());
        if (eps)
            finish(f_tree_norm(q.ptr(), k.ptr(), v.ptr(), g.ptr(), beta.ptr(), *eps, S, idx.ints(), parents.ints(), num.ints(), op->data_ptr(), &d, s.handle),
                   "kda_recurrent_tree_qknorm");
        else
            finish(f_tree(q.ptr(), k.ptr(), v.ptr(), g.ptr(), beta.ptr(), S, idx.ints(), parents.ints(), num.ints(), op->data_ptr(), &d, s.handle), "kda_recurrent_tree");
        return wrap(a[9], o);
    });
}

// (k, v, g, beta, state, parents, accepted, state_indices, num_tokens, qk_eps, stream)
PyObject *replay(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 11, "replay");
        const Arg q(Py_None, "q"), k(a[0], "k"), v(a[1], "v"), g(a[2], "g"), beta(a[3], "beta"), state(a[4], "state"), parents(a[5], "parents");
        const Arg accepted(a[6], "accepted"), idx(a[7], "state_indices"), num(a[8], "num_tokens");
        accepted.need(1, "[N]");
        int dev;
        const kda_dims_t d = tree_dims(q, k, v, g, beta, state, parents, idx, num, dev);
        accepted.check(at::kInt, dev, {d.batch});
        const std::optional<float> eps = epsilon(a[9]);
        const Stream s(a[10], dev);
        float *S = static_cast<float *>(state.ptr());
        if (eps)
            finish(f_replay_norm(k.ptr(), v.ptr(), g.ptr(), beta.ptr(), *eps, S, idx.ints(), parents.ints(), num.ints(), accepted.ints(), &d, s.handle),
                   "kda_recurrent_tree_commit_qknorm");
        else
            finish(f_replay(k.ptr(), v.ptr(), g.ptr(), beta.ptr(), S, idx.ints(), parents.ints(), num.ints(), accepted.ints(), &d, s.handle),
                   "kda_recurrent_tree_commit");
        return Py_NewRef(Py_None);
    });
}

// (q, k_cache, v_cache, block_table, seq_lens, parents, scale, num_tokens, out, lse, want_lse, workspace, stream)
PyObject *tree_attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 13, "tree_attend");
        const Arg q(a[0], "q"), kc(a[1], "k_cache"), vc(a[2], "v_cache"), table(a[3], "block_table"), lens(a[4], "seq_lens"), parents(a[5], "parents");
        const Arg num(a[7], "num_tokens"), out(a[8], "out"), lse(a[9], "lse"), ws(a[11], "workspace");
        q.need(4, "[N, T, Hq, d]"), lens.need(1, "[N]");
        const int dev = device_of(q);
        const at::ScalarType dt = q.t->scalar_type();
        const int64_t N = q.size(0), T = q.size(1), Hq = q.size(2);
        kda_paged_dims_t d = paged_dims(kc, vc, table, N, Hq, dt, dtype_of(q), dev);
        d.heads = narrow(Hq, "Hq");
        q.check(dt, dev, {N, T, Hq, d.head_dim});
        lens.check(at::kInt, dev, {N});
        parents.check(at::kInt, dev, {N, T});
        num.check(at::kInt, dev, {N});
        out.check(dt, dev, {N, T, Hq, d.head_dim});
        lse.check(at::kFloat, dev, {N, T, Hq});
        if (ws) ws.check(at::kByte, dev, {ws.t->numel()});
        const double scale = PyFloat_AsDouble(a[6]);
        if (PyErr_Occurred()) throw Refused{};
        const int32_t tokens = narrow(T, "T");
        const Stream s(a[12], dev);
        at::Tensor o, l, w;
        const at::Tensor *op = or_made(out, o, s, {N, T, Hq, d.head_dim}, dt), *lp = nullptr;
        if (lse || truth(a[10])) lp = or_made(lse, l, s, {N, T, Hq}, at::kFloat);
        const at::Tensor *wp = ws.t;
        if (!wp)
            if (const size_t bytes = f_tree_attend_bytes(tokens, &d)) wp = or_made(ws, w, s, {(int64_t)bytes}, at::kByte);
        finish(f_tree_attend(q.ptr(), kc.ptr(), vc.ptr(), table.ints(), lens.ints(), parents.ints(), num.ints(), tokens, (float)scale, op->data_ptr(),
                             lp ? static_cast<float *>(lp->data_ptr()) : nullptr, wp ? wp->data_ptr() : nullptr, wp ? (size_t)wp->numel() : 0, &d, s.handle),
               "kda_paged_tree_attention");
        return pair(wrap(a[8], o), wrap(a[9], l));
    });
}

// (k_cache, v_cache, block_table, seq_lens, parents, accepted, num_tokens, tokens, new_lens, stream)
PyObject *keep(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 10, "keep");
        const Arg kc(a[0], "k_cache"), vc(a[1], "v_cache"), table(a[2], "block_table"), lens(a[3], "seq_lens"), parents(a[4], "parents");
        const Arg accepted(a[5], "accepted"), num(a[6], "num_tokens"), to(a[8], "new_lens");
        kc.need(4, "[pages, page_size, Hkv, d]"), lens.need(1, "[N]"), accepted.need(1, "[N]");
        const int dev = device_of(kc);
        const int64_t N = lens.size(0);
        int64_t T = 0;
        if (parents) {
            T = parents.need(2, "[N, T]").size(1);
        } else {
            T = PyLong_AsLongLong(a[7]);
            if (PyErr_Occurred()) throw Refused{};
        }
        const kda_paged_dims_t d = paged_dims(kc, vc, table, N, 0, kc.t->scalar_type(), dtype_of(kc), dev);
        lens.check(at::kInt, dev, {N});
        parents.check(at::kInt, dev, {N, T});
        accepted.check(at::kInt, dev, {N});
        num.check(at::kInt, dev, {N});
        to.check(at::kInt, dev, {N});
        const Stream s(a[9], dev);
        at::Tensor made;
        const at::Tensor *tp = or_made(to, made, s, {N}, at::kInt);
        finish(f_keep(kc.ptr(), vc.ptr(), table.ints(), lens.ints(), parents.ints(), num.ints(), accepted.ints(), narrow(T, "T"),
                      static_cast<int32_t *>(tp->data_ptr()), &d, s.handle),
               "kda_paged_tree_commit");
        return wrap(a[8], made);
    });
}

kda_paged_dims_t pool_dims(const Arg &table, const Arg &refs, int64_t page_size) {
    return {narrow(table.size(0), "N"), 1, 1, 64, narrow(refs.size(0), "pages"), narrow(page_size, "page_size"), narrow(table.size(1), "max_pages"), KDA_BF16};
}

// (block_table, seq_lens, page_refs, sources, new_tokens, page_size, new_table, new_lens, new_refs, copies, short_of, stream)
PyObject *fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 12, "fork");
        const Arg table(a[0], "block_table"), lens(a[1], "seq_lens"), refs(a[2], "page_refs"), sources(a[3], "sources"), more(a[4], "new_tokens");
        const Arg out[5] = {{a[6], "new_table"}, {a[7], "new_lens"}, {a[8], "new_refs"}, {a[9], "copies"}, {a[10], "short_of"}};
        table.need(2, "[N, max_pages]"), lens.need(1, "[N]"), refs.need(1, "[pages]"), sources.need(1, "[N]");
        const int dev = device_of(table);
        const int64_t N = table.size(0), W = table.size(1), pages = refs.size(0), ps = PyLong_AsLongLong(a[5]);
        if (PyErr_Occurred()) throw Refused{};
        table.check(at::kInt, dev, {N, W});
        lens.check(at::kInt, dev, {N});
        refs.check(at::kInt, dev, {pages});
        sources.check(at::kInt, dev, {N});
        more.check(at::kInt, dev, {N});
        out[0].check(at::kInt, dev, {N, W});
        out[1].check(at::kInt, dev, {N});
        out[2].check(at::kInt, dev, {pages});
        out[3].check(at::kInt, dev, {N, 2});
        out[4].check(at::kInt, dev, {1});
        const kda_paged_dims_t d = pool_dims(table, refs, ps);
        const Stream s(a[11], dev);
        at::Tensor made[5];
        int32_t *p[5];
        p[0] = static_cast<int32_t *>(or_made(out[0], made[0], s, {N, W}, at::kInt)->data_ptr());
        p[1] = static_cast<int32_t *>(or_made(out[1], made[1], s, {N}, at::kInt)->data_ptr());
        p[2] = static_cast<int32_t *>(or_made(out[2], made[2], s, {pages}, at::kInt)->data_ptr());
        p[3] = static_cast<int32_t *>(or_made(out[3], made[3], s, {N, 2}, at::kInt)->data_ptr());
        p[4] = static_cast<int32_t *>(or_made(out[4], made[4], s, {1}, at::kInt)->data_ptr());
        finish(f_fork(table.ints(), lens.ints(), refs.ints(), sources.ints(), more.ints(), p[0], p[1], p[2], p[3], p[4], &d, s.handle), "kda_paged_fork");
        PyObject *r = PyTuple_New(5);
        for (int i = 0; r && i < 5; ++i) PyTuple_SET_ITEM(r, i, wrap(a[6 + i], made[i]));
        return r;
    });
}

// (block_table, page_refs, new_table, new_refs, copies, stream)
PyObject *compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 6, "compact");
        const Arg table(a[0], "block_table"), refs(a[1], "page_refs"), nt(a[2], "new_table"), nr(a[3], "new_refs"), copies(a[4], "copies");
        table.need(2, "[N, max_pages]"), refs.need(1, "[pages]");
        const int dev = device_of(table);
        const int64_t N = table.size(0), W = table.size(1), pages = refs.size(0);
        table.check(at::kInt, dev, {N, W});
        refs.check(at::kInt, dev, {pages});
        nt.check(at::kInt, dev, {N, W});
        nr.check(at::kInt, dev, {pages});
        copies.check(at::kInt, dev, {pages / 2, 2});
        const kda_paged_dims_t d = pool_dims(table, refs, 1);
        const Stream s(a[5], dev);
        at::Tensor made[3];
        int32_t *p[3];
        p[0] = static_cast<int32_t *>(or_made(nt, made[0], s, {N, W}, at::kInt)->data_ptr());
        p[1] = static_cast<int32_t *>(or_made(nr, made[1], s, {pages}, at::kInt)->data_ptr());
        p[2] = static_cast<int32_t *>(or_made(copies, made[2], s, {pages / 2, 2}, at::kInt)->data_ptr());
        finish(f_compact(table.ints(), refs.ints(), p[0], p[1], p[2], &d, s.handle), "kda_paged_compact");
        PyObject *r = PyTuple_New(3);
        for (int i = 0; r && i < 3; ++i) PyTuple_SET_ITEM(r, i, wrap(a[2 + i], made[i]));
        return r;
    });
}

// (k_cache, v_cache, copies, stream)
PyObject *copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 4, "copy");
        const Arg kc(a[0], "k_cache"), vc(a[1], "v_cache"), copies(a[2], "copies");
        kc.need(4, "[pages, page_size, Hkv, d]"), vc.need(4, "shaped like k_cache"), copies.need(2, "[M, 2]");
        const int dev = device_of(kc);
        const at::ScalarType dt = kc.t->scalar_type();
        const int64_t pages = kc.size(0), ps = kc.size(1), hkv = kc.size(2), d = kc.size(3), M = copies.size(0);
        const kda_dtype_t code = dtype_of(kc);
        kc.check(dt, dev, {pages, ps, hkv, d});
        vc.check(dt, dev, {pages, ps, hkv, d});
        copies.check(at::kInt, dev, {M, 2});
        const kda_paged_dims_t dims{0, narrow(hkv, "Hkv"), narrow(hkv, "Hkv"), narrow(d, "d"), narrow(pages, "pages"), narrow(ps, "page_size"), 1, code};
        const Stream s(a[3], dev);
        finish(f_copy(kc.ptr(), vc.ptr(), copies.ints(), M, &dims, s.handle), "kda_paged_copy");
        return Py_NewRef(Py_None);
    });
}

// (raise_status, the addresses in the order of the declarations above)
template <typename F> void take(F &f, PyObject *o) { f = reinterpret_cast<F>(PyLong_AsVoidPtr(o)); }

PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 17, "bind");
        PyObject *const *p = a + 1;
        std::apply([&](auto &...f) { (take(f, *p++), ...); },
                   std::tie(f_chunk, f_chunk_bytes, f_step, f_append, f_attend, f_attend_bytes, f_tree, f_tree_norm, f_replay, f_replay_norm, f_tree_attend,
                            f_tree_attend_bytes, f_keep, f_fork, f_compact, f_copy));
        if (PyErr_Occurred()) throw Refused{};
        Py_XSETREF(raise_status, Py_NewRef(a[0]));
        return Py_NewRef(Py_None);
    });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(lin_chunk), METHOD(lin_step), METHOD(append), METHOD(attend), METHOD(tree), METHOD(replay), METHOD(tree_attend),
                         METHOD(keep), METHOD(fork), METHOD(compact), METHOD(copy), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
