// torch_ops.cpp -- the operators around the verification for torch tensors: checks
// of arguments, outputs from torch's allocator, the current stream.
//
// A decoding step of few tokens is bound by the host: written in Python over ctypes
// these calls took 11 to 18 us each (tensor attributes 0.1 us apiece, torch.empty
// 1.7, an argument of ctypes 0.15), of which a launch is 3.  binding.py has the
// signatures and the documentation; None stands for an argument left out.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <string>

#include "spec_verify.h"

namespace {

using at::Tensor;

struct Raised {};  // a Python exception is set
PyObject* g_error = nullptr;  // binding.SpecVerifyError

[[noreturn]] void bad(const std::string& what) {
    PyErr_SetString(PyExc_ValueError, what.c_str());
    throw Raised();
}
[[noreturn]] void bad_type(const std::string& what) {
    PyErr_SetString(PyExc_TypeError, what.c_str());
    throw Raised();
}

struct Ref {  // an owned reference
    PyObject* p;
    explicit Ref(PyObject* q) : p(q) {
        if (!p) throw Raised();
    }
    Ref(const Ref&) = delete;
    ~Ref() { Py_DECREF(p); }
};

// Attribute names, made once.
#define NAMES(X) X(_ref) X(k) X(v) X(k_scale) X(v_scale) X(turns) X(positions) X(slots) X(masks) X(context_len) X(page_table) X(page_size) \
    X(num_pages) X(buffer) X(workspace) X(q_weight) X(k_weight) X(eps) X(num_tokens) X(num_keys) X(q_heads) X(kv_heads) X(prompts) X(stream_id) X(device_index) X(device_type)
struct Names {
#define X(n) PyObject* n = nullptr;
    NAMES(X)
#undef X
} N;

PyObject* attr(PyObject* o, PyObject* name) {
    PyObject* a = PyObject_GetAttr(o, name);
    if (!a) throw Raised();
    return a;
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
int64_t int_attr(PyObject* o, PyObject* name) {
    Ref a(attr(o, name));
    return integer(a.p);
}

// The calls have no backward: a tensor whose history they would drop is refused.
void without_history(const Tensor& t, const char* name) {
    if (!t.unsafeGetTensorImpl()->autograd_meta()) return;  // (most tensors, and every one of integers)
    if ((t.requires_grad() && c10::GradMode::is_enabled()) ||
        (t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode()))
        bad(std::string(name) + " carries a gradient, which this call would drop: detach it, or call under torch.no_grad()");
}

// None: not given
const Tensor* maybe(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
    const Tensor& t = THPVariable_Unpack(o);
    without_history(t, name);
    return &t;
}
const Tensor& tensor(PyObject* o, const char* name) {
    const Tensor* t = maybe(o, name);
    if (!t) bad_type(std::string(name) + " must be a tensor");
    return *t;
}
Tensor tensor_attr(PyObject* o, PyObject* name, const char* what) {
    Ref a(attr(o, name));
    return tensor(a.p, what);
}

std::string shape_str(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

void on_device(const Tensor& t, const char* name, c10::Device dev) {
    if (!t.is_cuda()) bad(std::string(name) + " must be a CUDA tensor");
    if (t.device() != dev) bad(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
}
void of_type(const Tensor& t, const char* name, at::ScalarType ty) {
    if (t.scalar_type() != ty)
        bad(std::string(name) + " must be " + c10::toString(ty) + ", got " + c10::toString(t.scalar_type()));
}
void check(const Tensor& t, const char* name, at::ScalarType ty, at::IntArrayRef shape, c10::Device dev) {
    on_device(t, name, dev);
    of_type(t, name, ty);
    if (t.sizes() != shape)
        bad(std::string(name) + " must have shape " + shape_str(shape) + ", got " + shape_str(t.sizes()));
    if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
}
// a contiguous tensor of n entries
void flat(const Tensor& t, const char* name, at::ScalarType ty, int64_t n, c10::Device dev) {
    on_device(t, name, dev);
    of_type(t, name, ty);
    if (t.numel() != n)
        bad(std::string(name) + " has " + std::to_string(t.numel()) + " entries for " + std::to_string(n) + " tokens");
    if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
}
int32_t* status_word(PyObject* o, c10::Device dev) {
    const Tensor* t = maybe(o, "dev_status");
    if (!t) return nullptr;
    check(*t, "dev_status", at::kInt, {1}, dev);
    return static_cast<int32_t*>(t->data_ptr());
}
spec_dtype dtype_of(const Tensor& t, const char* name) {
    switch (t.scalar_type()) {
        case at::kFloat: return SPEC_F32;
        case at::kBFloat16: return SPEC_BF16;
        case at::kHalf: return SPEC_F16;
        default: bad(std::string(name) + " must be float32, bfloat16 or float16, got " + c10::toString(t.scalar_type()));
    }
}

// [..., heads, D] as tokens of heads: the leading dimensions are one run of tokens.
struct Rows {
    void* p = nullptr;
    int64_t n = 0, step = 0, head = 0;
    int heads = 0;
};
Rows rows(const Tensor& t, const char* name, int64_t heads, int64_t D, at::ScalarType ty, c10::Device dev,
          int64_t tokens) {
    on_device(t, name, dev);
    of_type(t, name, ty);
    const int64_t d = t.dim();
    const auto sh = t.sizes(), st = t.strides();
    if (d < 3 || sh[d - 1] != D || (heads >= 0 && sh[d - 2] != heads))
        bad(std::string(name) + " must be [tokens, " + (heads >= 0 ? std::to_string(heads) : "heads") + ", " +
            std::to_string(D) + "], got " + shape_str(sh));
    if (D > 1 && st[d - 1] != 1) bad(std::string("the channels of ") + name + " must be contiguous");
    int64_t n = sh[d - 3], step = st[d - 3];
    for (int64_t i = d - 4; i >= 0; --i) {
        if (sh[i] != 1 && n > 1 && st[i] != n * step)
            bad(std::string("the leading dimensions of ") + name + " must be one run of tokens");
        if (n == 1) step = st[i];
        n *= sh[i];
    }
    if (tokens >= 0 && n != tokens)
        bad(std::string(name) + " has " + std::to_string(n) + " tokens, expected " + std::to_string(tokens));
    if (sh[d - 2] > INT32_MAX) bad(std::string(name) + " has too many heads");
    return {t.data_ptr(), n, step, st[d - 2], int(sh[d - 2])};
}

Tensor empty(at::IntArrayRef shape, at::ScalarType ty, c10::Device dev) {
    return at::detail::empty_cuda(shape, ty, dev, c10::nullopt);
}

// The call's stream: `stream` (a torch.cuda.Stream) is made current for its duration, so
// that what is allocated belongs to the stream that the kernels run on, and the
// allocator is told of every other tensor the call uses there (`uses`), so that the
// memory of one that is dropped meanwhile is not given away before they ran.
struct OnStream {
    c10::cuda::OptionalCUDAStreamGuard guard;
    std::optional<c10::cuda::CUDAStream> given;
    explicit OnStream(PyObject* s) {
        if (s == Py_None) return;
        given = c10::cuda::CUDAStream::unpack3(int_attr(s, N.stream_id), c10::DeviceIndex(int_attr(s, N.device_index)),
                                               c10::DeviceType(int_attr(s, N.device_type)));
        guard.reset_stream(*given);
    }
    void uses(std::initializer_list<const Tensor*> ts) const {
        if (!given) return;
        for (const Tensor* t : ts)
            if (t && t->defined()) c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(), *given);
    }
    void uses_attrs(PyObject* o, std::initializer_list<PyObject*> names) const {
        if (!given) return;
        for (PyObject* n : names) {
            Ref a(attr(o, n));
            uses({maybe(a.p, "tensor")});
        }
    }
    void uses_cache(PyObject* o) const { uses_attrs(o, {N.k, N.v, N.k_scale, N.v_scale}); }
};

// f(stream) with the device current, without the interpreter's lock
template <class F>
void run(const char* what, c10::Device dev, F&& f) {
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != dev.index()) guard.set_index(dev.index());
    const spec_stream_t st = reinterpret_cast<spec_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    PyThreadState* save = PyEval_SaveThread();
    const spec_status rc = f(st);
    PyEval_RestoreThread(save);
    if (rc == SPEC_OK) return;
    Ref e(PyObject_CallFunction(g_error, "is", int(rc), what));
    PyErr_SetObject(g_error, e.p);
    throw Raised();
}

PyObject* same(PyObject* given, const Tensor& t) {
    if (given == Py_None) return THPVariable_Wrap(t);
    Py_INCREF(given);
    return given;
}

struct Cache {
    const spec_kv_cache* c;
    Tensor k;  // one of its tensors: device and type
    explicit Cache(PyObject* o)
        : c(reinterpret_cast<const spec_kv_cache*>(int_attr(o, N._ref))), k(tensor_attr(o, N.k, "cache")) {}
    c10::Device device() const { return k.device(); }
};

// A norm as it is at this call: what is checked here is what the kernel reads (a module can give
// its weights other memory, or another type, after the norm was made of them).
struct Norm {
    Tensor q, k;  // weights, where there are some
    spec_head_norm n = {};
    explicit Norm(PyObject* o) {
        Ref x(attr(o, N.q_weight)), y(attr(o, N.k_weight)), e(attr(o, N.eps));
        if (const Tensor* t = maybe(x.p, "q_weight")) q = *t;
        if (const Tensor* t = maybe(y.p, "k_weight")) k = *t;
        const double eps = PyFloat_AsDouble(e.p);
        if (eps == -1.0 && PyErr_Occurred()) throw Raised();
        n.eps = float(eps);
        n.dtype = SPEC_F32;
    }
    void fits(int64_t D, c10::Device dev) {
        n.q_weight = weight(q, "q_weight", D, dev);
        n.k_weight = weight(k, "k_weight", D, dev);
        if (q.defined() && k.defined() && q.scalar_type() != k.scalar_type()) bad("q_weight and k_weight must have one type");
    }
    const void* weight(const Tensor& t, const char* name, int64_t D, c10::Device dev) {
        if (!t.defined()) return nullptr;
        on_device(t, name, dev);
        n.dtype = dtype_of(t, name);
        if (t.numel() != D) bad(std::string(name) + " has " + std::to_string(t.numel()) + " entries for heads of " + std::to_string(D));
        if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
};

// rope(q, k, positions, table, out_q, out_k, inverse, stream)
PyObject* rope(PyObject* const* a) {
    OnStream on(a[7]);
    const Tensor& q = tensor(a[0], "q");
    const Tensor* k = maybe(a[1], "k");
    const Tensor& pos = tensor(a[2], "positions");
    const auto* table = reinterpret_cast<const spec_rope_table*>(int_attr(a[3], N._ref));
    const int inverse = PyObject_IsTrue(a[6]);
    if (inverse < 0) throw Raised();
    const c10::Device dev = q.device();
    const at::ScalarType ty = q.scalar_type();
    const int64_t D = q.dim() ? q.size(-1) : 0;
    const Rows rq = rows(q, "q", -1, D, ty, dev, -1);
    const spec_dtype dt = dtype_of(q, "q");
    const Tensor oq = a[4] == Py_None ? empty(q.sizes(), ty, dev) : tensor(a[4], "out_q");
    const Rows ro = rows(oq, "out_q", rq.heads, D, ty, dev, rq.n);
    Rows rk, rp;
    Tensor ok;
    if (k) {
        rk = rows(*k, "k", -1, D, ty, dev, rq.n);
        ok = a[5] == Py_None ? empty(k->sizes(), ty, dev) : tensor(a[5], "out_k");
        rp = rows(ok, "out_k", rk.heads, D, ty, dev, rq.n);
    }
    flat(pos, "positions", at::kInt, rq.n, dev);
    const auto* pp = static_cast<const int32_t*>(pos.data_ptr());
    on.uses({&q, k, &pos, &oq, &ok});
    on.uses_attrs(a[3], {N.turns});
    run("spec_rope", dev, [&](spec_stream_t st) {
        return spec_rope(rq.p, rq.heads, rq.step, rq.head, ro.p, ro.step, ro.head, rk.p, rk.heads, rk.step, rk.head,
                         rp.p, rp.step, rp.head, dt, int(D), rq.n, pp, table, inverse, st);
    });
    if (!k) return same(a[4], oq);
    Ref x(same(a[4], oq)), y(same(a[5], ok));
    return PyTuple_Pack(2, x.p, y.p);
}

// kv_write(cache, k, v, slots, positions, table, q, out_q, dev_status, stream)
PyObject* kv_write(PyObject* const* a) {
    OnStream on(a[9]);
    const Cache c(a[0]);
    const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &slots = tensor(a[3], "slots");
    const Tensor *pos = maybe(a[4], "positions"), *q = maybe(a[6], "q");
    const c10::Device dev = c.device();
    const at::ScalarType ty = k.scalar_type();
    const int64_t D = c.c->head_dim;
    const Rows rk = rows(k, "k", c.c->heads, D, ty, dev, -1), rv = rows(v, "v", c.c->heads, D, ty, dev, rk.n);
    const spec_dtype dt = dtype_of(k, "k");
    flat(slots, "slots", at::kLong, rk.n, dev);
    if (!pos != (a[5] == Py_None)) bad("a rotation needs positions and a table");
    const spec_rope_table* table = nullptr;
    const int32_t* pp = nullptr;
    if (pos) {
        flat(*pos, "positions", at::kInt, rk.n, dev);
        table = reinterpret_cast<const spec_rope_table*>(int_attr(a[5], N._ref));
        pp = static_cast<const int32_t*>(pos->data_ptr());
    }
    Rows rq, ro;
    Tensor oq;
    if (q) {
        if (!table) bad("q is taken along only to be rotated");
        rq = rows(*q, "q", -1, D, ty, dev, rk.n);
        oq = a[7] == Py_None ? empty(q->sizes(), ty, dev) : tensor(a[7], "out_q");
        ro = rows(oq, "out_q", rq.heads, D, ty, dev, rk.n);
    }
    int32_t* st_word = status_word(a[8], dev);
    const auto* sp = static_cast<const int64_t*>(slots.data_ptr());
    on.uses({&k, &v, &slots, pos, q, &oq, maybe(a[8], "dev_status")});
    on.uses_cache(a[0]);
    if (table) on.uses_attrs(a[5], {N.turns});
    run("spec_kv_write", dev, [&](spec_stream_t st) {
        return spec_kv_write(c.c, rk.p, rk.step, rk.head, rv.p, rv.step, rv.head, dt, rk.n, sp, pp, table, rq.p, rq.heads,
                             rq.step, rq.head, ro.p, ro.step, ro.head, st_word, st);
    });
    if (!q) Py_RETURN_NONE;
    return same(a[7], oq);
}

// kv_read(cache, slots, dtype, out_k, out_v, stream)
PyObject* kv_read(PyObject* const* a) {
    OnStream on(a[5]);
    const Cache c(a[0]);
    const Tensor& slots = tensor(a[1], "slots");
    const c10::Device dev = c.device();
    flat(slots, "slots", at::kLong, slots.numel(), dev);
    at::ScalarType ty = c.c->dtype == SPEC_E4M3 ? at::kBFloat16 : c.k.scalar_type();
    if (a[2] != Py_None) {
        if (!THPDtype_Check(a[2])) bad_type("dtype must be a torch.dtype");
        ty = reinterpret_cast<THPDtype*>(a[2])->scalar_type;
    }
    c10::SmallVector<int64_t, 6> shape(slots.sizes().begin(), slots.sizes().end());
    shape.push_back(c.c->heads);
    shape.push_back(c.c->head_dim);
    Tensor out[2];
    for (int i = 0; i < 2; ++i) {
        const char* name = i ? "out_v" : "out_k";
        if (a[3 + i] == Py_None) {
            out[i] = empty(shape, ty, dev);
        } else {
            out[i] = tensor(a[3 + i], name);
            check(out[i], name, ty, shape, dev);
        }
    }
    const spec_dtype dt = dtype_of(out[0], "dtype");
    on.uses({&slots, &out[0], &out[1]});
    on.uses_cache(a[0]);
    run("spec_kv_read", dev, [&](spec_stream_t st) {
        return spec_kv_read(c.c, slots.numel(), static_cast<const int64_t*>(slots.data_ptr()), dt, out[0].data_ptr(),
                            out[1].data_ptr(), st);
    });
    Ref x(same(a[3], out[0])), y(same(a[4], out[1]));
    return PyTuple_Pack(2, x.p, y.p);
}

// tree_plan(tree_parents, num_nodes, context_len, page_table, cache, dev_status, stream):
// (positions, slots, masks, buffer)
PyObject* tree_plan(PyObject* const* a) {
    OnStream on(a[6]);
    const Tensor &par = tensor(a[0], "tree_parents"), &nodes = tensor(a[1], "num_nodes"),
                 &ctx = tensor(a[2], "context_len"), &table = tensor(a[3], "page_table");
    const Cache c(a[4]);
    const c10::Device dev = c.device();
    if (par.dim() != 2 || table.dim() != 2) bad("tree_parents must be [B, N] and page_table [B, max_pages]");
    const int64_t B = par.size(0), NN = par.size(1), width = table.size(1);
    check(par, "tree_parents", at::kInt, {B, NN}, dev);
    check(nodes, "num_nodes", at::kInt, {B}, dev);
    check(ctx, "context_len", at::kInt, {B}, dev);
    check(table, "page_table", at::kInt, {B, width}, dev);
    if (B > INT32_MAX || NN > INT32_MAX || width > INT32_MAX) bad("too many requests, nodes or pages");
    int32_t* st_word = status_word(a[5], dev);
    const size_t n = spec_tree_plan_size(int(B));
    const Tensor buffer = empty({int64_t(n)}, at::kByte, dev), positions = empty({B, NN}, at::kInt, dev),
                 masks = empty({B, NN}, at::kInt, dev), slots = empty({B, NN}, at::kLong, dev);
    on.uses({&par, &nodes, &ctx, &table, maybe(a[5], "dev_status")});
    run("spec_tree_plan", dev, [&](spec_stream_t st) {
        return spec_tree_plan(static_cast<const int32_t*>(par.data_ptr()), static_cast<const int32_t*>(nodes.data_ptr()),
                              static_cast<const int32_t*>(ctx.data_ptr()), static_cast<const int32_t*>(table.data_ptr()),
                              int(B), int(NN), int(width), c.c->page_size, c.c->num_pages,
                              static_cast<int32_t*>(positions.data_ptr()), static_cast<int64_t*>(slots.data_ptr()),
                              static_cast<uint32_t*>(masks.data_ptr()), buffer.data_ptr(), n, st_word, st);
    });
    Ref x(THPVariable_Wrap(positions)), y(THPVariable_Wrap(slots)), z(THPVariable_Wrap(masks)), w(THPVariable_Wrap(buffer));
    return PyTuple_Pack(4, x.p, y.p, z.p, w.p);
}

// The tensors of a plan that a call reads, for B requests of N nodes: a caller can set the
// plan's fields.
struct AttentionPlan {
    Tensor masks, table, buffer;
    AttentionPlan(PyObject* o, int64_t B, int64_t NN, c10::Device dev)
        : masks(tensor_attr(o, N.masks, "plan.masks")), table(tensor_attr(o, N.page_table, "plan.page_table")),
          buffer(tensor_attr(o, N.buffer, "plan.buffer")) {
        check(masks, "plan.masks", at::kInt, {B, NN}, dev);
        if (table.dim() != 2) bad("plan.page_table must be [B, max_pages]");
        check(table, "plan.page_table", at::kInt, {B, table.size(1)}, dev);
        on_device(buffer, "plan.buffer", dev);
        if (!buffer.is_contiguous() || buffer.nbytes() < spec_tree_plan_size(int(B))) bad("plan.buffer is not the plan's");
    }
};
struct CommitPlan {
    Tensor masks, slots, ctx;
    CommitPlan(PyObject* o, int64_t B, int64_t NN, c10::Device dev)
        : masks(tensor_attr(o, N.masks, "plan.masks")), slots(tensor_attr(o, N.slots, "plan.slots")),
          ctx(tensor_attr(o, N.context_len, "plan.context_len")) {
        check(masks, "plan.masks", at::kInt, {B, NN}, dev);
        check(slots, "plan.slots", at::kLong, {B, NN}, dev);
        check(ctx, "plan.context_len", at::kInt, {B}, dev);
    }
};

void check_pages(PyObject* plan, const Cache& c, c10::Device dev) {
    if (int_attr(plan, N.page_size) != c.c->page_size || int_attr(plan, N.num_pages) != c.c->num_pages ||
        c.device() != dev)
        bad("the plan was made for a cache of other pages");
}

// tree_attention(q, cache, plan, scale, masks, out, lse, workspace, dev_status, stream)
PyObject* tree_attention(PyObject* const* a) {
    OnStream on(a[9]);
    const Tensor& q = tensor(a[0], "q");
    const Cache c(a[1]);
    PyObject* plan = a[2];
    const c10::Device dev = c.device();
    if (q.dim() != 4 || q.size(3) != c.c->head_dim) bad("q must be [B, N, q_heads, head_dim]");
    const int64_t B = q.size(0), NN = q.size(1), Hq = q.size(2), D = q.size(3);
    on_device(q, "q", dev);
    if (q.stride(3) != 1) bad("the channels of q must be contiguous");
    const Tensor positions = tensor_attr(plan, N.positions, "plan.positions");
    if (positions.dim() != 2 || positions.size(0) != B || positions.size(1) != NN)
        bad("the plan is for " + shape_str(positions.sizes()) + ", q for " + shape_str({B, NN}));
    check_pages(plan, c, positions.device());
    const AttentionPlan P(plan, B, NN, dev);
    const spec_dtype dt = dtype_of(q, "q");
    Tensor masks = P.masks;
    if (a[4] != Py_None) {
        masks = tensor(a[4], "masks");
        check(masks, "masks", at::kInt, {B, NN}, dev);
    }
    Tensor out;
    if (a[5] == Py_None) {
        out = empty({B, NN, Hq, D}, q.scalar_type(), dev);
    } else {
        out = tensor(a[5], "out");
        check(out, "out", q.scalar_type(), {B, NN, Hq, D}, dev);
    }
    const Tensor* lse = maybe(a[6], "lse");
    if (lse) check(*lse, "lse", at::kFloat, {B, NN, Hq}, dev);
    int32_t* st_word = status_word(a[8], dev);
    double scale = 1.0 / std::sqrt(double(D));
    if (a[3] != Py_None) {
        scale = PyFloat_AsDouble(a[3]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised();
    }
    if (Hq < 1 || Hq > 65536 || Hq % c.c->heads)
        bad("unsupported: " + std::to_string(Hq) + " query heads over " + std::to_string(c.c->heads));
    Tensor ws;
    if (a[7] != Py_None) {
        ws = tensor(a[7], "workspace");
        on_device(ws, "workspace", dev);
        if (!ws.is_contiguous()) bad("workspace must be contiguous");
    } else {  // one for each stream, so that its memory is never another's while a kernel uses it
        Ref kept(attr(plan, N.workspace));
        const auto raw = reinterpret_cast<unsigned long long>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
        Ref key(Py_BuildValue("(KLL)", raw, (long long)c.c->heads, (long long)D));
        PyObject* w = PyDict_GetItemWithError(kept.p, key.p);
        if (w) {
            ws = tensor(w, "workspace");
        } else {
            if (PyErr_Occurred()) throw Raised();
            size_t n = 0;
            {
                c10::cuda::CUDAGuard guard(dev.index());
                n = spec_tree_attention_workspace_size(c.c, int(Hq));
            }
            if (n == 0)
                bad("unsupported: " + std::to_string(Hq) + " query heads over " + std::to_string(c.c->heads) + " of " +
                    std::to_string(D));
            ws = empty({int64_t(n)}, at::kByte, dev);
            Ref t(THPVariable_Wrap(ws));
            if (PyDict_SetItem(kept.p, key.p, t.p)) throw Raised();
        }
    }
    on.uses({&q, &P.buffer, &P.table, &masks, &out, lse, &ws, maybe(a[8], "dev_status")});
    on.uses_cache(a[1]);
    run("spec_tree_attention", dev, [&](spec_stream_t st) {
        return spec_tree_attention(q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), dt, int(B), int(NN), int(Hq), c.c,
                                   static_cast<const int32_t*>(P.table.data_ptr()), int(P.table.size(1)),
                                   static_cast<const uint32_t*>(masks.data_ptr()), P.buffer.data_ptr(), float(scale),
                                   out.data_ptr(), lse ? static_cast<float*>(lse->data_ptr()) : nullptr, ws.data_ptr(),
                                   ws.nbytes(), st_word, st);
    });
    return same(a[5], out);
}

// kv_commit(caches, plan, last_node, new_context_len, dev_status, stream)
PyObject* kv_commit(PyObject* const* a) {
    OnStream on(a[5]);
    Ref list(PySequence_Fast(a[0], "caches must be a list"));
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(list.p);
    if (count == 0) bad("no caches");
    PyObject* plan = a[1];
    const Tensor &last = tensor(a[2], "last_node"), positions = tensor_attr(plan, N.positions, "plan.positions");
    if (positions.dim() != 2) bad("plan.positions must be [B, N]");
    const int64_t B = positions.size(0), NN = positions.size(1);
    const c10::Device dev = positions.device();
    const CommitPlan P(plan, B, NN, dev);
    check(last, "last_node", at::kInt, {B}, dev);
    Tensor len;
    if (a[3] == Py_None) {
        len = empty({B}, at::kInt, dev);
    } else {
        len = tensor(a[3], "new_context_len");
        check(len, "new_context_len", at::kInt, {B}, dev);
    }
    int32_t* st_word = status_word(a[4], dev);
    for (Py_ssize_t i = 0; i < count; ++i) {
        check_pages(plan, Cache(PySequence_Fast_GET_ITEM(list.p, i)), dev);
        on.uses_cache(PySequence_Fast_GET_ITEM(list.p, i));
    }
    on.uses({&last, &P.masks, &P.slots, &P.ctx, &len, maybe(a[4], "dev_status")});
    // the lengths are written once, by the last group of caches: it may be the
    // plan's own context_len, which the earlier groups still read
    Tensor scratch;
    if (count > SPEC_MAX_COMMIT_CACHES) scratch = empty({B}, at::kInt, dev);
    for (Py_ssize_t i = 0; i < count; i += SPEC_MAX_COMMIT_CACHES) {
        spec_kv_cache group[SPEC_MAX_COMMIT_CACHES];
        const int n = int(std::min<Py_ssize_t>(count - i, SPEC_MAX_COMMIT_CACHES));
        for (int j = 0; j < n; ++j) group[j] = *Cache(PySequence_Fast_GET_ITEM(list.p, i + j)).c;
        const Tensor& to = i + n == count ? len : scratch;
        run("spec_kv_commit", dev, [&](spec_stream_t st) {
            return spec_kv_commit(group, n, static_cast<const uint32_t*>(P.masks.data_ptr()),
                                  static_cast<const int64_t*>(P.slots.data_ptr()), static_cast<const int32_t*>(last.data_ptr()),
                                  static_cast<const int32_t*>(P.ctx.data_ptr()), int(B), int(NN),
                                  static_cast<int32_t*>(to.data_ptr()), st_word, st);
        });
    }
    return same(a[3], len);
}

// norm_rope(q, k, positions, table, norm, out_q, out_k, stream)
PyObject* norm_rope(PyObject* const* a) {
    OnStream on(a[7]);
    const Tensor& q = tensor(a[0], "q");
    const Tensor *k = maybe(a[1], "k"), *pos = maybe(a[2], "positions");
    Norm norm(a[4]);
    if (!pos != (a[3] == Py_None)) bad("a rotation needs positions and a table");
    const spec_rope_table* table = nullptr;
    if (pos) table = reinterpret_cast<const spec_rope_table*>(int_attr(a[3], N._ref));
    const c10::Device dev = q.device();
    const at::ScalarType ty = q.scalar_type();
    const int64_t D = q.dim() ? q.size(-1) : 0;
    norm.fits(D, dev);
    const Rows rq = rows(q, "q", -1, D, ty, dev, -1);
    const spec_dtype dt = dtype_of(q, "q");
    const Tensor oq = a[5] == Py_None ? empty(q.sizes(), ty, dev) : tensor(a[5], "out_q");
    const Rows ro = rows(oq, "out_q", rq.heads, D, ty, dev, rq.n);
    Rows rk, rp;
    Tensor ok;
    if (k) {
        rk = rows(*k, "k", -1, D, ty, dev, rq.n);
        ok = a[6] == Py_None ? empty(k->sizes(), ty, dev) : tensor(a[6], "out_k");
        rp = rows(ok, "out_k", rk.heads, D, ty, dev, rq.n);
    }
    const int32_t* pp = nullptr;
    if (pos) {
        flat(*pos, "positions", at::kInt, rq.n, dev);
        pp = static_cast<const int32_t*>(pos->data_ptr());
    }
    on.uses({&q, k, pos, &oq, &ok, &norm.q, &norm.k});
    if (pos) on.uses_attrs(a[3], {N.turns});
    run("spec_norm_rope", dev, [&](spec_stream_t st) {
        return spec_norm_rope(&norm.n, rq.p, rq.heads, rq.step, rq.head, ro.p, ro.step, ro.head, rk.p, rk.heads, rk.step,
                              rk.head, rp.p, rp.step, rp.head, dt, int(D), rq.n, pp, table, st);
    });
    if (!k) return same(a[5], oq);
    Ref x(same(a[5], oq)), y(same(a[6], ok));
    return PyTuple_Pack(2, x.p, y.p);
}

// norm_kv_write(cache, k, v, slots, positions, table, q, out_q, out_k, norm, dev_status, stream)
PyObject* norm_kv_write(PyObject* const* a) {
    OnStream on(a[11]);
    const Cache c(a[0]);
    const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &slots = tensor(a[3], "slots");
    const Tensor *pos = maybe(a[4], "positions"), *q = maybe(a[6], "q"), *ok = maybe(a[8], "out_k");
    std::optional<Norm> norm;
    if (a[9] != Py_None) norm.emplace(a[9]);
    const c10::Device dev = c.device();
    const at::ScalarType ty = k.scalar_type();
    const int64_t D = c.c->head_dim;
    if (norm) norm->fits(D, dev);
    const Rows rk = rows(k, "k", c.c->heads, D, ty, dev, -1), rv = rows(v, "v", c.c->heads, D, ty, dev, rk.n);
    const spec_dtype dt = dtype_of(k, "k");
    flat(slots, "slots", at::kLong, rk.n, dev);
    if (!pos != (a[5] == Py_None)) bad("a rotation needs positions and a table");
    const spec_rope_table* table = nullptr;
    const int32_t* pp = nullptr;
    if (pos) {
        flat(*pos, "positions", at::kInt, rk.n, dev);
        table = reinterpret_cast<const spec_rope_table*>(int_attr(a[5], N._ref));
        pp = static_cast<const int32_t*>(pos->data_ptr());
    }
    Rows rq, ro, rp;
    Tensor oq;
    if (ok) rp = rows(*ok, "out_k", c.c->heads, D, ty, dev, rk.n);
    if (q) {
        if (!table && !norm) bad("q is taken along only to be normalised or rotated");
        rq = rows(*q, "q", -1, D, ty, dev, rk.n);
        oq = a[7] == Py_None ? empty(q->sizes(), ty, dev) : tensor(a[7], "out_q");
        ro = rows(oq, "out_q", rq.heads, D, ty, dev, rk.n);
    }
    int32_t* st_word = status_word(a[10], dev);
    const auto* sp = static_cast<const int64_t*>(slots.data_ptr());
    on.uses({&k, &v, &slots, pos, q, &oq, ok, maybe(a[10], "dev_status")});
    if (norm) on.uses({&norm->q, &norm->k});
    on.uses_cache(a[0]);
    if (table) on.uses_attrs(a[5], {N.turns});
    run("spec_norm_kv_write", dev, [&](spec_stream_t st) {
        return spec_norm_kv_write(c.c, norm ? &norm->n : nullptr, rk.p, rk.step, rk.head, rp.p, rp.step, rp.head, rv.p, rv.step,
                                  rv.head, dt, rk.n, sp, pp, table, rq.p, rq.heads, rq.step, rq.head, ro.p, ro.step,
                                  ro.head, st_word, st);
    });
    if (!q) Py_RETURN_NONE;
    return same(a[7], oq);
}

// prompt_plan(offsets, num_tokens, q_heads, kv_heads, k_offsets, num_keys, page_table, cache, dev_status, stream):
// (positions, slots, buffer)
PyObject* prompt_plan(PyObject* const* a) {
    OnStream on(a[9]);
    const Tensor& off = tensor(a[0], "offsets");
    const Tensor *koff = maybe(a[4], "k_offsets"), *table = maybe(a[6], "page_table");
    const int64_t T = integer(a[1]), Hq = integer(a[2]), Hkv = integer(a[3]), M = a[5] == Py_None ? T : integer(a[5]);
    const c10::Device dev = off.device();
    if (off.dim() != 1 || off.size(0) < 1) bad("offsets must be [prompts + 1]");
    const int64_t B = off.size(0) - 1;
    check(off, "offsets", at::kInt, {B + 1}, dev);
    if (koff) check(*koff, "k_offsets", at::kInt, {B + 1}, dev);
    if (!koff && M != T) bad("num_keys differs from num_tokens without k_offsets");
    if (!table != (a[7] == Py_None)) bad("slots need a page table and a cache");
    std::optional<Cache> c;
    if (table) {
        c.emplace(a[7]);
        if (table->dim() != 2 || table->size(1) > INT32_MAX) bad("page_table must be [prompts, max_pages]");
        check(*table, "page_table", at::kInt, {B, table->size(1)}, dev);
        if (c->device() != dev) bad("the cache is on another device than the offsets");
    }
    if (B > INT32_MAX || Hq < 1 || Hq > INT32_MAX || Hkv < 1 || Hkv > INT32_MAX || T < 0 || M < 0) bad("sizes out of range");
    int32_t* st_word = status_word(a[8], dev);
    const size_t n = spec_prompt_plan_size(int(B), T, int(Hq), int(Hkv));
    if (n == 0)
        bad("unsupported: " + std::to_string(B) + " prompts of " + std::to_string(T) + " tokens, " + std::to_string(Hq) +
            " query heads over " + std::to_string(Hkv));
    const Tensor buffer = empty({int64_t(n)}, at::kByte, dev), positions = empty({T}, at::kInt, dev);
    Tensor slots;
    if (table) slots = empty({T}, at::kLong, dev);
    on.uses({&off, koff, table, maybe(a[8], "dev_status")});
    run("spec_prompt_plan", dev, [&](spec_stream_t st) {
        return spec_prompt_plan(static_cast<const int32_t*>(off.data_ptr()),
                                koff ? static_cast<const int32_t*>(koff->data_ptr()) : nullptr, int(B), T, M, int(Hq), int(Hkv),
                                table ? static_cast<const int32_t*>(table->data_ptr()) : nullptr, table ? int(table->size(1)) : 0,
                                table ? c->c->page_size : 0, table ? c->c->num_pages : 0,
                                static_cast<int32_t*>(positions.data_ptr()),
                                table ? static_cast<int64_t*>(slots.data_ptr()) : nullptr, buffer.data_ptr(), n, st_word, st);
    });
    Ref x(THPVariable_Wrap(positions)), w(THPVariable_Wrap(buffer));
    if (!table) return PyTuple_Pack(3, x.p, Py_None, w.p);
    Ref y(THPVariable_Wrap(slots));
    return PyTuple_Pack(3, x.p, y.p, w.p);
}

// prompt_attention(q, k, v, plan, scale, window, out, lse, dev_status, stream)
PyObject* prompt_attention(PyObject* const* a) {
    OnStream on(a[9]);
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    PyObject* plan = a[3];
    const c10::Device dev = q.device();
    const at::ScalarType ty = q.scalar_type();
    const int64_t B = int_attr(plan, N.prompts), T = int_attr(plan, N.num_tokens), M = int_attr(plan, N.num_keys),
                  Hq = int_attr(plan, N.q_heads), Hkv = int_attr(plan, N.kv_heads);
    if (q.dim() != 3) bad("q must be [tokens, q_heads, head_dim]");
    if (k.dim() != 3 || v.dim() != 3) bad("k and v must be [keys, kv_heads, head_dim]");
    const int64_t D = q.size(2);
    const Rows rq = rows(q, "q", Hq, D, ty, dev, T), rk = rows(k, "k", Hkv, D, ty, dev, M), rv = rows(v, "v", Hkv, D, ty, dev, M);
    const spec_dtype dt = dtype_of(q, "q");
    const Tensor buffer = tensor_attr(plan, N.buffer, "plan.buffer");
    on_device(buffer, "plan.buffer", dev);
    if (B < 0 || B > INT32_MAX || Hq > INT32_MAX || Hkv > INT32_MAX || D > INT32_MAX || !buffer.is_contiguous() ||
        buffer.nbytes() < spec_prompt_plan_size(int(B), T, int(Hq), int(Hkv)))
        bad("plan.buffer is not the plan's");
    double scale = 1.0 / std::sqrt(double(D));
    if (a[4] != Py_None) {
        scale = PyFloat_AsDouble(a[4]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised();
    }
    const int64_t window = integer(a[5]);
    if (window < 0 || window > INT32_MAX) bad("window must be a number of tokens, or 0");
    Tensor out;
    if (a[6] == Py_None) {
        out = empty({T, Hq, D}, ty, dev);
    } else {
        out = tensor(a[6], "out");
        check(out, "out", ty, {T, Hq, D}, dev);
    }
    const Tensor* lse = maybe(a[7], "lse");
    if (lse) check(*lse, "lse", at::kFloat, {T, Hq}, dev);
    int32_t* st_word = status_word(a[8], dev);
    on.uses({&q, &k, &v, &buffer, &out, lse, maybe(a[8], "dev_status")});
    run("spec_prompt_attention", dev, [&](spec_stream_t st) {
        return spec_prompt_attention(rq.p, rq.step, rq.head, rk.p, rk.step, rk.head, rv.p, rv.step, rv.head, dt, int(B), T, M,
                                     int(Hq), int(Hkv), int(D), buffer.data_ptr(), float(scale), int(window), out.data_ptr(),
                                     lse ? static_cast<float*>(lse->data_ptr()) : nullptr, st_word, st);
    });
    return same(a[6], out);
}

// token_logprobs(logits, tokens, rows, temperature, top, entropy, workspace, dev_status, stream):
// (logprobs, entropy, top_ids, top_logprobs)
PyObject* token_logprobs(PyObject* const* a) {
    OnStream on(a[8]);
    const Tensor &logits = tensor(a[0], "logits"), &tokens = tensor(a[1], "tokens");
    const Tensor *row = maybe(a[2], "rows"), *temp = maybe(a[3], "temperature");
    const int64_t top = integer(a[4]);
    const int ent = PyObject_IsTrue(a[5]);
    if (ent < 0) throw Raised();
    const c10::Device dev = logits.device();
    const int64_t d = logits.dim();
    if (d < 1 || logits.size(-1) < 1) bad("logits must be [..., V]");
    on_device(logits, "logits", dev);
    const spec_dtype dt = dtype_of(logits, "logits");
    const int64_t V = logits.size(-1);
    if (V > 1 && logits.stride(-1) != 1) bad("the vocabulary of logits must be contiguous");
    // the leading dimensions are one run of rows
    int64_t R = 1, step = V;
    for (int64_t i = d - 2; i >= 0; --i) {
        const int64_t n = logits.size(i), s = logits.stride(i);
        if (n != 1 && R > 1 && s != R * step) bad("the leading dimensions of logits must be one run of rows");
        if (R == 1 && n != 1) step = s;
        R *= n;
    }
    if (R <= 1) step = V;
    const int64_t E = tokens.numel();
    check(tokens, "tokens", at::kInt, tokens.sizes(), dev);
    if (row) check(*row, "rows", at::kInt, tokens.sizes(), dev);
    else if (E != R) bad("tokens are " + std::to_string(E) + " for " + std::to_string(R) + " rows of logits");
    if (temp) check(*temp, "temperature", at::kFloat, tokens.sizes(), dev);
    if (top < 0 || top > SPEC_MAX_TOP) bad("top must be 0 to " + std::to_string(SPEC_MAX_TOP));
    if (V > (1 << 24)) bad("unsupported: a vocabulary of " + std::to_string(V));
    int32_t* st_word = status_word(a[7], dev);
    size_t n = 0;
    {
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != dev.index()) guard.set_index(dev.index());
        n = spec_token_logprobs_workspace_size(E, int(V));
    }
    if (n == 0) bad("unsupported: " + std::to_string(E) + " tokens");
    Tensor ws;
    if (a[6] != Py_None) {
        ws = tensor(a[6], "workspace");
        on_device(ws, "workspace", dev);
        if (!ws.is_contiguous()) bad("workspace must be contiguous");
    } else {  // of the stream's own pool, so that nothing else has it before the kernels have run
        ws = empty({int64_t(n)}, at::kByte, dev);
    }
    c10::SmallVector<int64_t, 6> shape(tokens.sizes().begin(), tokens.sizes().end());
    const Tensor lp = empty(shape, at::kFloat, dev);
    Tensor h, ids, lps;
    if (ent) h = empty(shape, at::kFloat, dev);
    if (top) {
        shape.push_back(top);
        ids = empty(shape, at::kInt, dev);
        lps = empty(shape, at::kFloat, dev);
    }
    on.uses({&logits, &tokens, row, temp, &ws, maybe(a[7], "dev_status")});
    auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    run("spec_token_logprobs", dev, [&](spec_stream_t st) {
        return spec_token_logprobs(logits.data_ptr(), dt, R, step, int(V), row ? static_cast<const int32_t*>(row->data_ptr()) : nullptr,
                                   static_cast<const int32_t*>(tokens.data_ptr()),
                                   temp ? static_cast<const float*>(temp->data_ptr()) : nullptr, E, int(top),
                                   static_cast<float*>(lp.data_ptr()), static_cast<float*>(ptr(h)), static_cast<int32_t*>(ptr(ids)),
                                   static_cast<float*>(ptr(lps)), ws.data_ptr(), ws.nbytes(), st_word, st);
    });
    auto wrap = [](const Tensor& t) {
        if (t.defined()) return THPVariable_Wrap(t);
        Py_INCREF(Py_None);
        return Py_None;
    };
    Ref x(wrap(lp)), y(wrap(h)), z(wrap(ids)), w(wrap(lps));
    return PyTuple_Pack(4, x.p, y.p, z.p, w.p);
}

template <PyObject* (*F)(PyObject* const*), int COUNT>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != COUNT) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", COUNT, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// error_class(cls): what a refused call raises
PyObject* error_class(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

#define ENTRY(name, count) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<name, count>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(rope, 8),           ENTRY(kv_write, 10),  ENTRY(kv_read, 6), ENTRY(tree_plan, 7),
                         ENTRY(tree_attention, 10), ENTRY(kv_commit, 6), ENTRY(norm_rope, 8), ENTRY(norm_kv_write, 12),
                         ENTRY(prompt_plan, 10), ENTRY(prompt_attention, 10), ENTRY(token_logprobs, 9),
                         {"error_class", error_class, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "specverify_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_specverify_torch() {
#define X(n) \
    if (!(N.n = PyUnicode_InternFromString(#n))) return nullptr;
    NAMES(X)
#undef X
    return PyModule_Create(&module_def);
}
