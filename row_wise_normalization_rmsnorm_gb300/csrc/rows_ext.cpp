// rows_ext.cpp -- the Python binding of the entry points on training rows
// (8-bit checkpoints, group norm, embedding rows): argument checks and
// marshalling, with no computation.
#include "ext_args.h"

using namespace ext;

extern PyMethodDef rows_methods[];

namespace {

// A contiguous CUDA tensor, of `like`'s type and device where there is one.
const at::Tensor &rows_arg(PyObject *o, const char *name, const at::Tensor *like = nullptr) {
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
    if (t.layout() != at::kStrided || !t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    if (like && (t.scalar_type() != like->scalar_type() || t.device() != like->device()))
        value_error(std::string(name) + " must match dtype/device of the input");
    return t;
}
void numel_is(const at::Tensor &t, const char *name, int64_t n) {
    if (t.numel() != n) value_error(std::string(name) + " must have " + str(n) + " elements, has " + str(t.numel()));
}
void same_shape(const at::Tensor &t, const char *name, const at::Tensor &like) {
    if (t.sizes() != like.sizes()) value_error(std::string(name) + " must have shape " + shape_of(like) + ", has " + shape_of(t));
}

// Rows x columns of the last dimension.
struct Matrix {
    int64_t M, N;
    explicit Matrix(const at::Tensor &x, const char *name) {
        N = x.dim() > 0 ? x.size(-1) : 0;
        if (N < 1) value_error(std::string(name) + " must have a last dimension of 1 or more, has " + shape_of(x));
        M = x.numel() / N;
    }
};

// A weight in the activations' type or fp32: its pointer (None: NULL) and
// RMSNORM_WEIGHT_F32 into `flag`. `first`: the weight that it has to agree with.
const void *weight_arg(PyObject *o, const char *name, const at::Tensor &x, int64_t n, int &flag, const at::Tensor **first = nullptr) {
    if (o == Py_None) return nullptr;
    const at::Tensor &w = tensor(o, name);
    beside(w, name, x.scalar_type(), at::kFloat, x);
    numel_is(w, name, n);
    if (first) {
        if (*first && (*first)->scalar_type() != w.scalar_type()) value_error(std::string(name) + " must have the other parameters' type");
        *first = &w;
    }
    if (w.scalar_type() == at::kFloat && x.scalar_type() != at::kFloat) flag = RMSNORM_WEIGHT_F32;
    return ptr(w);
}

// A result: the caller's tensor, checked, or a new one.
struct Result {
    Ref ref;
    void *p = nullptr;
    Result(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like, const LaunchStream &s) {
        if (o == Py_None) {
            const at::Tensor t = new_tensor(shape, type, like, s);
            ref.o = THPVariable_Wrap(t);
            if (!ref.o) throw AlreadySet{};
            p = ptr(t);
            return;
        }
        const at::Tensor &t = rows_arg(o, name);
        if (t.device() != like.device()) value_error(std::string(name) + " must be on the input's device");
        if (t.scalar_type() != type)
            value_error(std::string(name) + " must be " + c10::toString(type) + ", is " + c10::toString(t.scalar_type()));
        int64_t n = 1;
        for (int64_t d : shape) n *= d;
        numel_is(t, name, n);
        ref.o = Py_NewRef(o);
        p = ptr(t);
    }
};

// 8-bit codes (torch.int8) of x's shape and their scales (torch.uint8).
std::vector<int64_t> scales_shape(at::IntArrayRef x) {
    std::vector<int64_t> s(x.begin(), x.end());
    s.back() = (s.back() + CKPT8_BLOCK - 1) / CKPT8_BLOCK;
    return s;
}
const at::Tensor &codes_arg(PyObject *codes, PyObject *scales, const at::Tensor **sc) {
    const at::Tensor &c = rows_arg(codes, "codes"), &s = rows_arg(scales, "scales");
    if (c.scalar_type() != at::kChar || s.scalar_type() != at::kByte) value_error("codes must be int8 and scales uint8");
    if (s.device() != c.device()) value_error("scales must be on the codes' device");
    const Matrix m(c, "codes");
    numel_is(s, "scales", m.M * ((m.N + CKPT8_BLOCK - 1) / CKPT8_BLOCK));
    *sc = &s;
    return c;
}

// The caller's workspace, or (on the current stream) one of torch's allocator;
// for a named stream the library takes stream-ordered memory there.
struct Workspace {
    void *p = nullptr;
    size_t bytes = 0;
    at::Tensor made;
    Workspace(PyObject *o, size_t need, const at::Tensor &like, const LaunchStream &s) {
        if (o != Py_None) {
            const at::Tensor &w = tensor(o, "workspace");
            if (!w.is_cuda() || w.device() != like.device() || !w.is_contiguous())
                value_error("workspace must be a contiguous CUDA tensor on the input's device");
            p = ptr(w);
            bytes = (size_t)w.numel() * w.element_size();
        } else if (!s.named && need > 0) {
            made = new_tensor({(int64_t)need}, at::kByte, like, s);
            p = ptr(made);
            bytes = need;
        }
    }
};

PyObject *tuple(std::initializer_list<PyObject *> items) {  // steals the references
    PyObject *r = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (r)
            PyTuple_SET_ITEM(r, i++, o);
        else
            Py_XDECREF(o);
    }
    if (!r) throw AlreadySet{};
    return r;
}

rmsnorm_dtype_t code(int dt) { return (rmsnorm_dtype_t)dt; }

// pack(x, codes, scales, stream) -> codes, scales
PyObject *pack(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 4)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = rows_arg(a[0], "x");
        const int dt = dtype_code(x);
        const Matrix m(x, "x");
        const LaunchStream s(a[3], x);
        Result codes(a[1], "codes", x.sizes(), at::kChar, x, s), scales(a[2], "scales", scales_shape(x.sizes()), at::kByte, x, s);
        OnDevice on(x);
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = ckpt8_pack(ptr(x), codes.p, static_cast<uint8_t *>(scales.p), m.M, m.N, code(dt), s.handle);
        Py_END_ALLOW_THREADS
        check(st, "ckpt8_pack");
        return tuple({codes.ref.take(), scales.ref.take()});
    });
}

at::ScalarType torch_type(PyObject *o, const char *name) {
    if (!THPDtype_Check(o)) type_error(std::string(name) + " must be a torch.dtype");
    const at::ScalarType t = reinterpret_cast<THPDtype *>(o)->scalar_type;
    if (t != at::kFloat && t != at::kBFloat16 && t != at::kHalf)
        type_error("unsupported dtype; use torch.float32, torch.bfloat16 or torch.float16");
    return t;
}
int code_of(at::ScalarType t) { return t == at::kFloat ? RMSNORM_F32 : t == at::kBFloat16 ? RMSNORM_BF16 : RMSNORM_F16; }

// unpack(codes, scales, dtype, x, stream) -> x
PyObject *unpack(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 5)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor *sc;
        const at::Tensor &c = codes_arg(a[0], a[1], &sc);
        const at::ScalarType type = torch_type(a[2], "dtype");
        const Matrix m(c, "codes");
        const LaunchStream s(a[4], c);
        Result x(a[3], "x", c.sizes(), type, c, s);
        OnDevice on(c);
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = ckpt8_unpack(ptr(c), static_cast<const uint8_t *>(ptr(*sc)), x.p, m.M, m.N, code(code_of(type)), s.handle);
        Py_END_ALLOW_THREADS
        check(st, "ckpt8_unpack");
        return x.ref.take();
    });
}

// norm_keep(x, w, residual, eps, offset, y, residual_out, rstd, codes, scales, stream)
//   -> y, residual_out, rstd, codes, scales
PyObject *norm_keep(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 11)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = rows_arg(a[0], "x");
        int flag = 0;
        const int dt = dtype_code(x);
        const Matrix m(x, "x");
        const void *w = weight_arg(a[1], "w", x, m.N, flag);
        const at::Tensor *res = nullptr;
        if (a[2] != Py_None) {
            res = &rows_arg(a[2], "residual", &x);
            numel_is(*res, "residual", x.numel());
        } else if (a[6] != Py_None) {
            value_error("residual_out needs residual");
        }
        const float eps = float_arg(a[3], "eps"), offset = float_arg(a[4], "offset");
        const LaunchStream s(a[10], x);
        Result y(a[5], "y", x.sizes(), x.scalar_type(), x, s);
        std::optional<Result> h;
        if (res) h.emplace(a[6], "residual_out", x.sizes(), x.scalar_type(), x, s);
        Result rstd(a[7], "rstd", x.sizes().slice(0, x.dim() - 1), at::kFloat, x, s);
        Result codes(a[8], "codes", x.sizes(), at::kChar, x, s), scales(a[9], "scales", scales_shape(x.sizes()), at::kByte, x, s);
        OnDevice on(x);
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = rmsnorm_fwd_ckpt8(ptr(x), res ? ptr(*res) : nullptr, w, y.p, h ? h->p : nullptr, static_cast<float *>(rstd.p), codes.p,
                               static_cast<uint8_t *>(scales.p), m.M, m.N, code(dt | flag), eps, offset, s.handle);
        Py_END_ALLOW_THREADS
        check(st, "rmsnorm_fwd_ckpt8");
        return tuple({y.ref.take(), h ? h->ref.take() : Py_NewRef(Py_None), rstd.ref.take(), codes.ref.take(), scales.ref.take()});
    });
}

// norm_bwd(dy, codes, scales, w, rstd, dresidual_out, offset, dx, dw, workspace, stream) -> dx, dw
PyObject *norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 11)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &dy = rows_arg(a[0], "dy");
        int flag = 0;
        const int dt = dtype_code(dy);
        const at::Tensor *sc;
        const at::Tensor &c = codes_arg(a[1], a[2], &sc);
        const Matrix m(dy, "dy");
        if (c.device() != dy.device()) value_error("codes must be on the input's device");
        same_shape(c, "codes", dy);
        const void *w = weight_arg(a[3], "w", dy, m.N, flag);
        const at::Tensor &rstd = rows_arg(a[4], "rstd");
        beside(rstd, "rstd", at::kFloat, at::kFloat, dy);
        numel_is(rstd, "rstd", m.M);
        const at::Tensor *dres = nullptr;
        if (a[5] != Py_None) {
            dres = &rows_arg(a[5], "dresidual_out", &dy);
            numel_is(*dres, "dresidual_out", dy.numel());
        }
        const float offset = float_arg(a[6], "offset");
        const LaunchStream s(a[10], dy);
        Result dx(a[7], "dx", dy.sizes(), dy.scalar_type(), dy, s);
        std::optional<Result> dw;
        if (w)
            dw.emplace(a[8], "dw", tensor(a[3], "w").sizes(), tensor(a[3], "w").scalar_type(), dy, s);
        else if (a[8] != Py_None)
            value_error("dw needs w");
        OnDevice on(dy);
        Workspace ws(a[9], w && a[9] == Py_None ? rmsnorm_bwd_ckpt8_workspace_bytes(m.M, m.N, code(dt | flag)) : 0, dy, s);
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = rmsnorm_bwd_ckpt8(ptr(dy), dres ? ptr(*dres) : nullptr, ptr(c), static_cast<const uint8_t *>(ptr(*sc)), w,
                               static_cast<const float *>(ptr(rstd)), dx.p, dw ? dw->p : nullptr, ws.p, ws.bytes, m.M, m.N,
                               code(dt | flag), offset, s.handle);
        Py_END_ALLOW_THREADS
        check(st, "rmsnorm_bwd_ckpt8");
        return tuple({dx.ref.take(), dw ? dw->ref.take() : Py_NewRef(Py_None)});
    });
}

int64_t long_arg(PyObject *o, const char *name) {
    PyObject *i = PyNumber_Index(o);
    if (!i) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(i, &overflow);
    Py_DECREF(i);
    if (overflow || v < 0) value_error(std::string(name) + " is out of range");
    return v;
}

rmsnorm_act_t act_arg(PyObject *o) {
    if (o == Py_None) return ROWS_ACT_NONE;
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (s && !std::strcmp(s, "silu")) return ROWS_ACT_SILU;
    if (s && !std::strcmp(s, "gelu")) return ROWS_ACT_GELU;
    PyErr_Clear();
    value_error("act must be None, 'silu' or 'gelu'");
}

// [batch, ..., channels] as batch, places, channels.
struct Places {
    int64_t B, S, C, G;
    Places(const at::Tensor &x, const char *name, PyObject *groups) {
        if (x.dim() < 2 || x.size(-1) < 1) value_error(std::string(name) + " must be [batch, ..., channels], has " + shape_of(x));
        B = x.size(0);
        C = x.size(-1);
        S = 1;
        for (int64_t d = 1; d + 1 < x.dim(); ++d) S *= x.size(d);
        G = long_arg(groups, "groups");
        if (G < 1 || C % G != 0) value_error("groups must divide the " + str(C) + " channels, is " + str(G));
    }
};

// The largest power of two, up to 16, that the addresses are multiples of.
int32_t align_of(std::initializer_list<const void *> at) {
    uintptr_t all = 16;
    for (const void *q : at) all |= reinterpret_cast<uintptr_t>(q);
    return (int32_t)(all & (~all + 1));
}
// Workspace bytes of a group norm whose row arrays (and codes, or NULL) lie
// there; 0 for a call that will be refused.
size_t gn_need(const Places &p, int dt, bool backward, std::initializer_list<const void *> rows, const void *codes) {
    groupnorm_plan_t plan;
    const rmsnorm_status_t st = groupnorm_plan_query(p.B, p.S, p.C, p.G, (rmsnorm_dtype_t)dt, backward, codes != nullptr,
                                                     align_of(rows), align_of({codes}), 0, 0, &plan);
    return st == RMSNORM_SUCCESS ? (size_t)plan.workspace_bytes : 0;
}

// gn_fwd(x, gamma, beta, groups, act, eps, keep, y, mean, rstd, codes, scales, workspace, stream)
//   -> y, mean, rstd, codes, scales
PyObject *gn_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 14)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = rows_arg(a[0], "x");
        int flag = 0;
        const int dt = dtype_code(x);
        const Places p(x, "x", a[3]);
        const at::Tensor *first = nullptr;
        const void *gamma = weight_arg(a[1], "gamma", x, p.C, flag, &first), *beta = weight_arg(a[2], "beta", x, p.C, flag, &first);
        const rmsnorm_act_t act = act_arg(a[4]);
        const float eps = float_arg(a[5], "eps");
        const bool keep = a[6] == Py_True;
        const LaunchStream s(a[13], x);
        Result y(a[7], "y", x.sizes(), x.scalar_type(), x, s);
        Result mean(a[8], "mean", {p.B, p.G}, at::kFloat, x, s), rstd(a[9], "rstd", {p.B, p.G}, at::kFloat, x, s);
        std::optional<Result> codes, scales;
        if (keep) {
            codes.emplace(a[10], "codes", x.sizes(), at::kChar, x, s);
            scales.emplace(a[11], "scales", scales_shape(x.sizes()), at::kByte, x, s);
        }
        OnDevice on(x);
        Workspace ws(a[12], a[12] == Py_None && !s.named ? gn_need(p, dt, false, {ptr(x), y.p}, keep ? codes->p : nullptr) : 0, x, s);
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = groupnorm_fwd(ptr(x), gamma, beta, y.p, static_cast<float *>(mean.p), static_cast<float *>(rstd.p),
                           keep ? codes->p : nullptr, keep ? static_cast<uint8_t *>(scales->p) : nullptr, ws.p, ws.bytes, p.B, p.S,
                           p.C, p.G, act, code(dt | flag), eps, s.handle);
        Py_END_ALLOW_THREADS
        check(st, keep ? "groupnorm_fwd_ckpt8" : "groupnorm_fwd");
        return tuple({y.ref.take(), mean.ref.take(), rstd.ref.take(), keep ? codes->ref.take() : Py_NewRef(Py_None),
                      keep ? scales->ref.take() : Py_NewRef(Py_None)});
    });
}

// gn_bwd(dy, x, codes, scales, gamma, beta, mean, rstd, groups, act, want_dgamma, want_dbeta, dx, dgamma, dbeta,
//        workspace, stream) -> dx, dgamma, dbeta
PyObject *gn_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 17)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &dy = rows_arg(a[0], "dy");
        int flag = 0;
        const int dt = dtype_code(dy);
        const Places p(dy, "dy", a[8]);
        const at::Tensor *x = nullptr, *codes = nullptr, *scales = nullptr;
        if (a[1] != Py_None) {
            x = &rows_arg(a[1], "x", &dy);
            same_shape(*x, "x", dy);
        } else {
            codes = &codes_arg(a[2], a[3], &scales);
            if (codes->device() != dy.device()) value_error("codes must be on the input's device");
            same_shape(*codes, "codes", dy);
        }
        const at::Tensor *first = nullptr;
        const void *gamma = weight_arg(a[4], "gamma", dy, p.C, flag, &first), *beta = weight_arg(a[5], "beta", dy, p.C, flag, &first);
        const at::Tensor &mean = rows_arg(a[6], "mean"), &rstd = rows_arg(a[7], "rstd");
        beside(mean, "mean", at::kFloat, at::kFloat, dy);
        beside(rstd, "rstd", at::kFloat, at::kFloat, dy);
        numel_is(mean, "mean", p.B * p.G);
        numel_is(rstd, "rstd", p.B * p.G);
        const rmsnorm_act_t act = act_arg(a[9]);
        const bool want_gamma = a[10] == Py_True && gamma, want_beta = a[11] == Py_True;
        const at::ScalarType pt = first ? first->scalar_type() : dy.scalar_type();
        const LaunchStream s(a[16], dy);
        Result dx(a[12], "dx", dy.sizes(), dy.scalar_type(), dy, s);
        std::optional<Result> dgamma, dbeta;
        if (want_gamma) dgamma.emplace(a[13], "dgamma", at::IntArrayRef{p.C}, pt, dy, s);
        if (want_beta) dbeta.emplace(a[14], "dbeta", at::IntArrayRef{p.C}, pt, dy, s);
        OnDevice on(dy);
        Workspace ws(a[15], a[15] == Py_None && !s.named ? gn_need(p, dt, true, {ptr(dy), dx.p, x ? ptr(*x) : nullptr}, codes ? ptr(*codes) : nullptr) : 0,
                     dy, s);
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = groupnorm_bwd(ptr(dy), x ? ptr(*x) : nullptr, codes ? ptr(*codes) : nullptr,
                           scales ? static_cast<const uint8_t *>(ptr(*scales)) : nullptr, gamma, beta,
                           static_cast<const float *>(ptr(mean)), static_cast<const float *>(ptr(rstd)), dx.p,
                           dgamma ? dgamma->p : nullptr, dbeta ? dbeta->p : nullptr, ws.p, ws.bytes, p.B, p.S, p.C, p.G, act,
                           code(dt | flag), s.handle);
        Py_END_ALLOW_THREADS
        check(st, x ? "groupnorm_bwd" : "groupnorm_bwd_ckpt8");
        return tuple({dx.ref.take(), dgamma ? dgamma->ref.take() : Py_NewRef(Py_None), dbeta ? dbeta->ref.take() : Py_NewRef(Py_None)});
    });
}

// ids: int32 or int64, contiguous, on the table's (or dh's) device.
const at::Tensor &ids_arg(PyObject *o, const at::Tensor &like) {
    const at::Tensor &ids = tensor(o, "ids");
    beside(ids, "ids", at::kInt, at::kLong, like);
    return ids;
}
std::vector<int64_t> with_columns(at::IntArrayRef ids, int64_t N) {
    std::vector<int64_t> s(ids.begin(), ids.end());
    s.push_back(N);
    return s;
}

// embed(ids, table, w, norm, scale, eps, offset, y, h, rstd, stream) -> y, h, rstd
PyObject *embed(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 11)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &table = rows_arg(a[1], "table");
        int flag = 0;
        const int dt = dtype_code(table);
        if (table.dim() != 2 || table.size(1) < 1) value_error("table must be [rows, columns], has " + shape_of(table));
        const at::Tensor &ids = ids_arg(a[0], table);
        const int64_t T = ids.numel(), rows = table.size(0), N = table.size(1);
        const bool norm = a[3] == Py_True;
        const void *w = norm ? weight_arg(a[2], "w", table, N, flag) : nullptr;
        const float scale = float_arg(a[4], "scale"), eps = float_arg(a[5], "eps"), offset = float_arg(a[6], "offset");
        const LaunchStream s(a[10], table);
        const std::vector<int64_t> shape = with_columns(ids.sizes(), N);
        std::optional<Result> y, rstd;
        if (norm) y.emplace(a[7], "y", shape, table.scalar_type(), table, s);
        Result h(a[8], norm ? "residual_out" : "out", shape, table.scalar_type(), table, s);
        if (norm) rstd.emplace(a[9], "rstd", ids.sizes(), at::kFloat, table, s);
        OnDevice on(table);
        const int ib = (int)ids.element_size();
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = norm ? rmsnorm_embed_fwd(ptr(ids), ptr(table), w, y->p, h.p, static_cast<float *>(rstd->p), T, N, rows, ib,
                                      code(dt | flag), scale, eps, offset, s.handle)
                  : embed_fwd(ptr(ids), ptr(table), h.p, T, N, rows, ib, code(dt), scale, s.handle);
        Py_END_ALLOW_THREADS
        check(st, norm ? "rmsnorm_embed_fwd" : "embed_fwd");
        if (!norm) return h.ref.take();
        return tuple({y->ref.take(), h.ref.take(), rstd->ref.take()});
    });
}

// embed_grad(dh, ids, rows, scale, dtype, dtable, accumulate, workspace, stream) -> dtable
PyObject *embed_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 9)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &dh = rows_arg(a[0], "dh");
        const int dt = dtype_code(dh);
        const at::Tensor &ids = ids_arg(a[1], dh);
        const Matrix m(dh, "dh");
        if (ids.numel() != m.M) value_error("ids must have " + str(m.M) + " elements, has " + str(ids.numel()));
        const int64_t rows = long_arg(a[2], "rows");
        const float scale = float_arg(a[3], "scale");
        at::ScalarType type = a[4] != Py_None                                    ? torch_type(a[4], "dtype")
                              : a[5] != Py_None && THPVariable_Check(a[5]) ? THPVariable_Unpack(a[5]).scalar_type()
                                                                                 : dh.scalar_type();
        if (type != dh.scalar_type() && type != at::kFloat) value_error("dtable must have dh's type or be float32");
        const int accumulate = PyObject_IsTrue(a[6]);
        if (accumulate < 0) throw AlreadySet{};
        if (accumulate && a[5] == Py_None) value_error("accumulate needs dtable");
        const LaunchStream s(a[8], dh);
        Result out(a[5], "dtable", {rows, m.N}, type, dh, s);
        OnDevice on(dh);
        Workspace ws(a[7], a[7] == Py_None ? embed_bwd_workspace_bytes(m.M, m.N, rows) : 0, dh, s);
        const int flag = type != dh.scalar_type() ? RMSNORM_WEIGHT_F32 : 0, ib = (int)ids.element_size();
        rmsnorm_status_t st;
        Py_BEGIN_ALLOW_THREADS
        st = embed_bwd(ptr(dh), ptr(ids), out.p, ws.p, ws.bytes, m.M, m.N, rows, ib, code(dt | flag), scale, accumulate, s.handle);
        Py_END_ALLOW_THREADS
        check(st, "embed_bwd");
        return out.ref.take();
    });
}

// gn_workspace(batch, places, channels, groups, dtype code, backward), norm_workspace(M, N, code),
// embed_workspace(tokens, columns, rows): bytes on the current device
PyObject *workspace(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n == 6)
            return PyLong_FromSize_t(groupnorm_workspace_bytes(long_arg(a[0], "batch"), long_arg(a[1], "places"), long_arg(a[2], "channels"),
                                                               long_arg(a[3], "groups"), code((int)long_arg(a[4], "dtype")),
                                                               a[5] == Py_True));
        if (n == 4)
            return PyLong_FromSize_t(rmsnorm_bwd_ckpt8_workspace_bytes(long_arg(a[0], "M"), long_arg(a[1], "N"),
                                                                       code((int)long_arg(a[2], "dtype"))));
        if (!count(n, 3)) return nullptr;
        return PyLong_FromSize_t(embed_bwd_workspace_bytes(long_arg(a[0], "tokens"), long_arg(a[1], "columns"), long_arg(a[2], "rows")));
    });
}

#define METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}

}  // namespace

PyMethodDef rows_methods[] = {METHOD("pack", pack),         METHOD("unpack", unpack),         METHOD("norm_keep", norm_keep),
                              METHOD("norm_bwd", norm_bwd), METHOD("gn_fwd", gn_fwd),         METHOD("gn_bwd", gn_bwd),
                              METHOD("embed", embed),       METHOD("embed_grad", embed_grad), METHOD("workspace", workspace),
                              {nullptr, nullptr, 0, nullptr}};
