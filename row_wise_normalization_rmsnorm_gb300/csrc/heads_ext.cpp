// heads_ext.cpp -- the Python binding of the entry points on head rows
// (rotary positions, the paged cache, its attention): argument checks and
// marshalling, with no computation.
//
// A module in C++ because these calls serve single tokens: the same checks in
// Python took 10 to 20 us a call on a Grace host (rope_fwd of 8 tokens 23 us,
// 5 here, of a kernel of 3).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <optional>
#include <string>

#include "../../include/rmsnorm.h"

namespace {

// A Python exception to raise; thrown inside, set at the entry points.
struct Bad {
    PyObject *type;
    std::string what;
};
// A Python exception that is already set.
struct AlreadySet {};

[[noreturn]] void value_error(std::string s) { throw Bad{PyExc_ValueError, std::move(s)}; }
[[noreturn]] void type_error(std::string s) { throw Bad{PyExc_TypeError, std::move(s)}; }

std::string str(int64_t v) { return std::to_string(v); }
std::string shape_of(const at::Tensor &t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + str(t.size(i));
    return s + "]";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// RMSNORM_* code of a tensor's type.
int dtype_code(const at::Tensor &t) {
    switch (t.scalar_type()) {
    case at::kFloat: return RMSNORM_F32;
    case at::kBFloat16: return RMSNORM_BF16;
    case at::kHalf: return RMSNORM_F16;
    default: type_error("unsupported dtype; use torch.float32, torch.bfloat16 or torch.float16");
    }
}

// [tokens, heads, head_dim] on a GPU with head_dim contiguous, of one type
// and device with `like`.
void head_rows(const at::Tensor &t, const char *name, const at::Tensor *like) {
    if (t.layout() != at::kStrided || t.dim() != 3 || !t.is_cuda())
        value_error(std::string(name) + " must be a CUDA tensor [tokens, heads, head_dim], has " + shape_of(t));
    if (t.stride(2) != 1 && t.size(2) > 1) value_error(std::string(name) + "'s last dimension must be contiguous");
    if (like && (t.scalar_type() != like->scalar_type() || t.device() != like->device()))
        value_error(std::string(name) + " must match dtype/device of the other head rows");
}

// A vector or table beside the head rows.
void beside(const at::Tensor &t, const char *name, at::ScalarType a, at::ScalarType b, const at::Tensor &like,
            bool contiguous = true) {
    if (t.device() != like.device()) value_error(std::string(name) + " must be on the input's device");
    if (t.scalar_type() != a && t.scalar_type() != b)
        value_error(std::string(name) + " must be " + c10::toString(a) + (a == b ? "" : std::string(" or ") + c10::toString(b)) +
                    ", is " + c10::toString(t.scalar_type()));
    if (contiguous && !t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}

void *ptr(const at::Tensor &t) { return t.data_ptr(); }

// The stream that a call launches on: the device's current one (None), a
// handle, or an object with one.
struct LaunchStream {
    rmsnorm_stream_t handle;
    std::optional<c10::cuda::CUDAStream> named;  // where the caller named one
    LaunchStream(PyObject *stream, const at::Tensor &like) {
        const c10::DeviceIndex device = like.device().index();
        if (stream == Py_None) {
            handle = reinterpret_cast<rmsnorm_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
            return;
        }
        PyObject *h = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
        if (!h) throw AlreadySet{};
        void *p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!p && PyErr_Occurred()) throw AlreadySet{};
        if (p == static_cast<void *>(cudaStreamLegacy)) p = nullptr;  // the same stream; PyTorch knows it as 0
        handle = static_cast<rmsnorm_stream_t>(p);
        named = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), device);
    }
};

// A contiguous tensor on `like`'s device, from PyTorch's allocator (its CUDA
// entry itself: the dispatched at::empty takes 0.9 us a tensor longer). For a
// named stream the memory is that stream's own: the current stream's may still
// be in use by what was queued there before its last owner dropped it, and the
// named stream waits for none of that. Its first reader is likely to be the
// current stream, so the memory is not given out again, once dropped, before
// that one is done with it either.
at::Tensor new_tensor(at::IntArrayRef size, at::ScalarType type, const at::Tensor &like, const LaunchStream &s) {
    if (!s.named) return at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
    const c10::cuda::CUDAStream reader = c10::cuda::getCurrentCUDAStream(like.device().index());
    at::Tensor t;
    {
        c10::cuda::CUDAStreamGuard on(*s.named);
        t = at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
    }
    if (t.numel() > 0) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), reader);
    return t;
}

// Rows x (given as `in`) written to `out`, a tensor made here when None. The
// result is a new reference.
PyObject *rows_to(const at::Tensor &in, PyObject *out, const char *name, const LaunchStream &s, rope_rows_t &r) {
    std::string out_name = std::string(name) + "_out";
    at::Tensor made;
    const at::Tensor *o = &made;
    PyObject *result;
    if (out == Py_None) {
        made = new_tensor(in.sizes(), in.scalar_type(), in, s);
        result = THPVariable_Wrap(made);
        if (!result) throw AlreadySet{};
    } else {
        o = &tensor(out, out_name.c_str());
        head_rows(*o, out_name.c_str(), &in);
        if (o->sizes() != in.sizes())
            value_error(out_name + " must have " + name + "'s shape " + shape_of(in) + ", has " + shape_of(*o));
        result = Py_NewRef(out);
    }
    r = rope_rows_t{ptr(in), ptr(*o), in.stride(0), in.stride(1), o->stride(0), o->stride(1)};
    return result;
}

int pairing_of(PyObject *o) {
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (s && !std::strcmp(s, "half")) return ROPE_HALF;
    if (s && !std::strcmp(s, "adjacent")) return ROPE_ADJACENT;
    PyErr_Clear();
    value_error("pairing must be 'half' or 'adjacent'");
}

// The angles, and the axes' bytes (NULL: one axis).
const uint8_t *angles_of(PyObject *positions, PyObject *inv_freq, PyObject *axes, PyObject *pairing,
                         const at::Tensor &like, rope_angles_t &a) {
    const int64_t tokens = like.size(0), head_dim = like.size(2);
    const at::Tensor &p = tensor(positions, "positions"), &f = tensor(inv_freq, "inv_freq");
    beside(p, "positions", at::kInt, at::kLong, like, false);
    beside(f, "inv_freq", at::kFloat, at::kFloat, like);
    const int64_t n = p.dim() == 2 ? p.size(0) : 1;
    if ((p.dim() != 1 && p.dim() != 2) || p.size(-1) != tokens || n < 1 || n > ROPE_MAX_AXES)
        value_error("positions must be [" + str(tokens) + "] or [axes, " + str(tokens) + "] with 1 to 4 axes, has " +
                    shape_of(p));
    if (tokens > 1 && p.stride(-1) != 1) value_error("positions must be contiguous over the tokens");
    const int64_t half = f.dim() == 1 ? f.size(0) : 0;
    if (half < 1 || half > head_dim / 2)
        value_error("inv_freq must have 1 to " + str(head_dim / 2) + " frequencies for head_dim " + str(head_dim) + ", has " +
                    shape_of(f));
    const uint8_t *ax = nullptr;
    if (axes == Py_None) {
        if (n > 1) value_error("several axes need `axes` (rope_axes(sections))");
    } else {
        bool fine = PyBytes_Check(axes) && PyBytes_GET_SIZE(axes) == half;
        if (fine) {
            ax = reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(axes));
            for (int64_t i = 0; i < half; ++i) fine = fine && ax[i] < n;
        }
        if (!fine) value_error("axes must be " + str(half) + " bytes below " + str(n) + " (rope_axes(sections))");
    }
    a.positions = ptr(p);
    a.inv_freq = static_cast<const float *>(ptr(f));
    a.axis_stride = p.dim() == 2 ? p.stride(0) : 0;
    a.position_bytes = (int32_t)p.element_size();
    a.n_axes = (int32_t)n;
    a.rotary_dim = (int32_t)(2 * half);
    a.pairing = pairing_of(pairing);
    return ax;
}

void cache_of(PyObject *k_cache, PyObject *v_cache, const at::Tensor &like, paged_cache_t &c) {
    const at::Tensor &k = tensor(k_cache, "k_cache"), &v = tensor(v_cache, "v_cache");
    const at::Tensor *both[2] = {&k, &v};
    for (int i = 0; i < 2; ++i) {
        const at::Tensor &t = *both[i];
        const std::string name = i ? "v_cache" : "k_cache";
        if (t.layout() != at::kStrided || t.dim() != 4 || t.size(3) != like.size(2))
            value_error(name + " must be [pages, page_size, heads, " + str(like.size(2)) + "], has " + shape_of(t));
        if (t.scalar_type() != like.scalar_type() || t.device() != like.device())
            value_error(name + " must match dtype/device of the head rows");
        if (t.stride(3) != 1 && t.size(3) > 1) value_error(name + "'s last dimension must be contiguous");
        if (t.size(1) > 0x7fffffff || t.size(2) > 0x7fffffff) value_error(name + "'s pages are too large");
    }
    if (k.sizes() != v.sizes()) value_error("k_cache and v_cache must have one shape");
    c = paged_cache_t{ptr(k),      ptr(v),      k.size(0),   k.stride(0), k.stride(1), k.stride(2),
                      v.stride(0), v.stride(1), v.stride(2), (int32_t)k.size(1), (int32_t)k.size(2)};
}

int32_t size32(int64_t v, const char *name) {
    if (v < 0 || v > 0x7fffffff) value_error(std::string(name) + " is out of range");
    return (int32_t)v;
}

int32_t int_arg(PyObject *o, const char *name) {
    PyObject *n = PyNumber_Index(o);
    if (!n) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(n, &overflow);
    Py_DECREF(n);
    if (overflow) value_error(std::string(name) + " is out of range");
    return size32(v, name);
}

float float_arg(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be a number");
    }
    return (float)v;
}

// The tensors' device made current for the call, where it is not.
struct OnDevice {
    std::optional<c10::cuda::CUDAGuard> guard;
    explicit OnDevice(const at::Tensor &t) {
        if (t.device().index() != c10::cuda::current_device()) guard.emplace(t.device());
    }
};

// _binding._raise(status, what): the library's error as RMSNormError
void check(rmsnorm_status_t st, const char *what) {
    if (st == RMSNORM_SUCCESS) return;
    PyObject *m = PyImport_ImportModule("row_wise_normalization_rmsnorm_gb300._binding");
    PyObject *r = m ? PyObject_CallMethod(m, "_raise", "is", (int)st, what) : nullptr;
    Py_XDECREF(m);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, what);
    throw AlreadySet{};
}

// A new reference that is dropped unless taken.
struct Ref {
    PyObject *o = nullptr;
    ~Ref() { Py_XDECREF(o); }
    PyObject *take() {
        PyObject *r = o;
        o = nullptr;
        return r;
    }
};

template <class F> PyObject *guarded(F &&f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Bad &b) {
        PyErr_SetString(b.type, b.what.c_str());
    } catch (const AlreadySet &) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

bool count(Py_ssize_t have, Py_ssize_t want) {
    if (have == want) return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return false;
}

// rope(gradient, q, k, positions, inv_freq, axes, pairing, q_out, k_out, stream)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 10)) return nullptr;
    return guarded([&]() -> PyObject * {
        const bool grad = a[0] == Py_True;
        const char *qn = grad ? "dq" : "q", *kn = grad ? "dk" : "k";
        const at::Tensor &q = tensor(a[1], qn);
        rope_call_t c;
        std::memset(&c, 0, sizeof c);
        c.dtype = dtype_code(q);
        head_rows(q, qn, nullptr);
        Ref qo, ko;
        if (a[2] != Py_None) {
            const at::Tensor &k = tensor(a[2], kn);
            head_rows(k, kn, &q);
            if (k.size(0) != q.size(0) || k.size(2) != q.size(2))
                value_error(std::string(kn) + " must be [" + str(q.size(0)) + ", heads, " + str(q.size(2)) + "], has " + shape_of(k));
            c.k_heads = size32(k.size(1), kn);
        } else if (a[8] != Py_None) {
            value_error(std::string(kn) + "_out needs " + kn);
        }
        const uint8_t *axes = angles_of(a[3], a[4], a[5], a[6], q, c.angles);
        const LaunchStream s(a[9], q);
        qo.o = rows_to(q, a[7], qn, s, c.q);
        if (a[2] != Py_None) ko.o = rows_to(tensor(a[2], kn), a[8], kn, s, c.k);
        c.tokens = q.size(0);
        c.q_heads = size32(q.size(1), qn);
        c.head_dim = size32(q.size(2), qn);
        OnDevice on(q);
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = grad ? rope_bwd(&c, axes, s.handle) : rope_fwd(&c, axes, s.handle);
        Py_END_ALLOW_THREADS
        check(st, grad ? "rope_bwd" : "rope_fwd");
        PyObject *k_result = ko.o ? ko.take() : Py_NewRef(Py_None);
        PyObject *r = PyTuple_New(2);
        if (!r) {
            Py_DECREF(k_result);
            throw AlreadySet{};
        }
        PyTuple_SET_ITEM(r, 0, qo.take());
        PyTuple_SET_ITEM(r, 1, k_result);
        return r;
    });
}

// append(k, v, k_cache, v_cache, slots, positions, inv_freq, axes, pairing, q, q_out, wq, wk, eps, offset, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 16)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        paged_append_call_t c;
        std::memset(&c, 0, sizeof c);
        c.dtype = dtype_code(k);
        head_rows(k, "k", nullptr);
        head_rows(v, "v", &k);
        if (v.sizes() != k.sizes()) value_error("v must have k's shape " + shape_of(k) + ", has " + shape_of(v));
        const int64_t tokens = k.size(0), dim = k.size(2);
        const bool has_q = a[9] != Py_None;
        if (has_q) {
            const at::Tensor &q = tensor(a[9], "q");
            head_rows(q, "q", &k);
            if (q.size(0) != tokens || q.size(2) != dim)
                value_error("q must be [" + str(tokens) + ", heads, " + str(dim) + "], has " + shape_of(q));
            c.q_heads = size32(q.size(1), "q");
        } else if (a[10] != Py_None || a[11] != Py_None) {
            value_error("wq and q_out need q");
        }
        const uint8_t *axes = nullptr;
        if (a[5] != Py_None)
            axes = angles_of(a[5], a[6], a[7], a[8], k, c.angles);
        else if (a[6] != Py_None || a[7] != Py_None)
            value_error("inv_freq and axes need positions");
        cache_of(a[2], a[3], k, c.cache);
        if (c.cache.heads != k.size(1)) value_error("the cache holds " + str(c.cache.heads) + " heads, k has " + str(k.size(1)));
        const at::Tensor &slots = tensor(a[4], "slots");
        beside(slots, "slots", at::kLong, at::kLong, k);
        if (slots.numel() != tokens) value_error("slots must have " + str(tokens) + " elements, has " + str(slots.numel()));
        const void **to[2] = {&c.wq, &c.wk};
        const at::Tensor *first = nullptr;
        for (int i = 0; i < 2; ++i) {
            if (a[11 + i] == Py_None) continue;
            const char *name = i ? "wk" : "wq";
            const at::Tensor &w = tensor(a[11 + i], name);
            beside(w, name, k.scalar_type(), at::kFloat, k);
            if (w.numel() != dim || (first && w.scalar_type() != first->scalar_type()))
                value_error(std::string(name) + " must have " + str(dim) + " elements, and wq and wk one type");
            first = &w;
            *to[i] = ptr(w);
        }
        if (first && first->scalar_type() == at::kFloat && c.dtype != RMSNORM_F32) c.dtype |= RMSNORM_WEIGHT_F32;
        c.eps = float_arg(a[13], "eps");
        c.offset = float_arg(a[14], "offset");
        Ref qo;
        const LaunchStream s(a[15], k);
        if (has_q) qo.o = rows_to(tensor(a[9], "q"), a[10], "q", s, c.q);
        c.k = rope_rows_t{ptr(k), nullptr, k.stride(0), k.stride(1), 0, 0};
        c.v = rope_rows_t{ptr(v), nullptr, v.stride(0), v.stride(1), 0, 0};
        c.slots = static_cast<const int64_t *>(ptr(slots));
        c.tokens = tokens;
        c.head_dim = size32(dim, "k");
        OnDevice on(k);
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = paged_kv_append(&c, axes, s.handle);
        Py_END_ALLOW_THREADS
        check(st, "paged_kv_append");
        return has_q ? qo.take() : Py_NewRef(Py_None);
    });
}

// attn(q, k_cache, v_cache, block_table, kv_lens, cu_q, max_q, max_kv, scale, causal, out, lse, workspace, stream)
PyObject *attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 14)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &q = tensor(a[0], "q");
        paged_attn_call_t c;
        std::memset(&c, 0, sizeof c);
        c.dtype = dtype_code(q);
        head_rows(q, "q", nullptr);
        cache_of(a[1], a[2], q, c.cache);
        const at::Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "kv_lens"), &cu = tensor(a[5], "cu_q");
        beside(table, "block_table", at::kInt, at::kInt, q, false);
        beside(lens, "kv_lens", at::kInt, at::kInt, q);
        beside(cu, "cu_q", at::kInt, at::kInt, q);
        const int64_t batch = lens.dim() == 1 ? lens.size(0) : -1;
        if (batch < 0 || table.dim() != 2 || table.size(0) != batch || (table.size(1) > 1 && table.stride(1) != 1))
            value_error("block_table must be [batch, width] with contiguous rows, kv_lens [batch]");
        if (cu.dim() != 1 || cu.size(0) != batch + 1) value_error("cu_q must have " + str(batch + 1) + " elements");
        const int64_t tokens = q.size(0), heads = q.size(1);
        c.max_q = int_arg(a[6], "max_q");
        c.max_kv = int_arg(a[7], "max_kv");
        c.scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)q.size(2))) : float_arg(a[8], "scale");
        const int causal = PyObject_IsTrue(a[9]);
        if (causal < 0) throw AlreadySet{};
        c.causal = causal;
        rope_rows_t r;
        Ref out, lse;
        const LaunchStream s(a[13], q);
        out.o = rows_to(q, a[10], "q", s, r);
        if (a[11] == Py_True) {
            const at::Tensor t = new_tensor({tokens, heads}, at::kFloat, q, s);
            c.lse = static_cast<float *>(ptr(t));
            lse.o = THPVariable_Wrap(t);
            if (!lse.o) throw AlreadySet{};
        } else if (a[11] != Py_None && a[11] != Py_False) {
            const at::Tensor &t = tensor(a[11], "lse");
            beside(t, "lse", at::kFloat, at::kFloat, q);
            if (t.numel() != tokens * heads) value_error("lse must have " + str(tokens * heads) + " elements, has " + str(t.numel()));
            c.lse = static_cast<float *>(ptr(t));
            lse.o = Py_NewRef(a[11]);
        } else {
            lse.o = Py_NewRef(Py_None);
        }
        c.q = r.in;
        c.out = r.out;
        c.q_token = r.in_token;
        c.q_head = r.in_head;
        c.out_token = r.out_token;
        c.out_head = r.out_head;
        c.block_table = static_cast<const int32_t *>(ptr(table));
        c.kv_lens = static_cast<const int32_t *>(ptr(lens));
        c.cu_q = static_cast<const int32_t *>(ptr(cu));
        c.table_stride = table.stride(0);
        c.tokens = tokens;
        c.batch = size32(batch, "batch");
        c.table_width = size32(table.size(1), "block_table");
        c.q_heads = size32(heads, "q");
        c.head_dim = size32(q.size(2), "q");
        OnDevice on(q);
        at::Tensor made;
        if (a[12] != Py_None) {
            const at::Tensor &w = tensor(a[12], "workspace");
            if (!w.is_cuda() || w.device() != q.device() || !w.is_contiguous())
                value_error("workspace must be a contiguous CUDA tensor on the input's device");
            c.workspace = ptr(w);
            c.workspace_bytes = (size_t)w.numel() * w.element_size();
        } else if (!s.named) {
            // torch's allocator, on the current stream; for another stream the
            // library takes stream-ordered memory there
            const size_t bytes = paged_attn_workspace_bytes(&c);
            if (bytes > 0) {
                made = new_tensor({(int64_t)bytes}, at::kByte, q, s);
                c.workspace = ptr(made);
                c.workspace_bytes = bytes;
            }
        }
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = paged_attn_fwd(&c, s.handle);
        Py_END_ALLOW_THREADS
        check(st, "paged_attn_fwd");
        PyObject *result = PyTuple_New(2);
        if (!result) throw AlreadySet{};
        PyTuple_SET_ITEM(result, 0, out.take());
        PyTuple_SET_ITEM(result, 1, lse.take());
        return result;
    });
}

// attn_workspace(tokens, batch, heads, kv_heads, head_dim, max_q, max_kv)
PyObject *attn_workspace(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 7)) return nullptr;
    return guarded([&]() -> PyObject * {
        paged_attn_call_t c;
        std::memset(&c, 0, sizeof c);
        c.dtype = RMSNORM_BF16;
        c.tokens = int_arg(a[0], "tokens");
        c.batch = int_arg(a[1], "batch");
        c.q_heads = int_arg(a[2], "heads");
        c.cache.heads = int_arg(a[3], "kv_heads");
        c.head_dim = int_arg(a[4], "head_dim");
        c.max_q = int_arg(a[5], "max_q");
        c.max_kv = int_arg(a[6], "max_kv");
        return PyLong_FromSize_t(paged_attn_workspace_bytes(&c));
    });
}

PyMethodDef methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attn)), METH_FASTCALL, nullptr},
    {"attn_workspace", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attn_workspace)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_heads_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__heads_ext(void) { return PyModule_Create(&module); }
