// serve_binding.cpp -- the Python side of the drafted-token verification calls:
// argument checks, output and workspace allocation and the C call, in native
// code.  A call of a few microseconds on the GPU spent three times that in
// Python (17 us of 20 for one token over 1000 keys); here it is 2 us beside
// the launches.  The functions take positional arguments only and run on the
// current stream of their tensors' device; int8_bit_weight_amd/__init__.py
// documents them and handles streams.  Checks raise ValueError, a status
// of the library goes to the callback given to set_error.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "qmm.h"

namespace {

PyObject *g_error = nullptr;

#define NEED(cond, what)                           \
    do {                                           \
        if (!(cond)) {                             \
            PyErr_SetString(PyExc_ValueError, what); \
            return nullptr;                        \
        }                                          \
    } while (0)

// The tensor behind an argument; None gives an empty one if it may be missing.
struct Arg {
    at::Tensor t;
    bool ok = true;
    Arg(PyObject *o, bool optional = false) {
        if (THPVariable_Check(o)) {
            t = THPVariable_Unpack(o);
        } else if (!(optional && o == Py_None)) {
            PyErr_Format(PyExc_ValueError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
            ok = false;
        }
    }
    const at::Tensor *operator->() const { return &t; }
    explicit operator bool() const { return t.defined(); }
    void *data() const { return t.defined() ? t.data_ptr() : nullptr; }
};

// An integer argument; false with an exception set if it is none.
bool integer(PyObject *o, int64_t &v) {
    v = PyLong_AsLongLong(o);
    return !(v == -1 && PyErr_Occurred());
}

constexpr int kNone = -1;
int type_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
    case at::kFloat: return QMM_T_F32;
    case at::kHalf: return QMM_T_F16;
    case at::kBFloat16: return QMM_T_BF16;
    case at::kChar: return QMM_T_S8;
    default: return kNone;
    }
}
bool is_float(int t) { return t == QMM_T_F32 || t == QMM_T_F16 || t == QMM_T_BF16; }

// Elements of a row follow one another (or there is no second one).
bool rows(const at::Tensor &t) {
    const int64_t last = t.dim() - 1;
    return t.stride(last) == 1 || t.size(last) < 2 || t.numel() == 0;
}
// Row stride of a matrix; a single row's stride means nothing and may be anything.
int64_t ld(const at::Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

bool vector_of(const at::Tensor &t, at::ScalarType type) {
    return t.dim() == 1 && t.scalar_type() == type && (t.stride(0) == 1 || t.numel() < 2);
}

bool on_device(c10::Device d, std::initializer_list<const at::Tensor *> ts) {
    if (!d.is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "expected device (cuda) tensors");
        return false;
    }
    for (const at::Tensor *t : ts)
        if (t->defined() && t->device() != d) {
            PyErr_Format(PyExc_ValueError, "tensors on %s and %s", d.str().c_str(), t->device().str().c_str());
            return false;
        }
    return true;
}

void *stream_of(c10::Device d) { return c10::hip::getCurrentHIPStream(d.index()).stream(); }

at::Tensor bytes(size_t n, c10::Device d) { return at::empty({(int64_t)n}, at::TensorOptions().dtype(at::kByte).device(d)); }

size_t size_in_bytes(const at::Tensor &t) { return t.defined() ? (size_t)t.numel() * t.element_size() : 0; }
// A workspace's bytes follow one another (or there is none).
bool is_workspace(const at::Tensor &t) { return !t.defined() || t.is_contiguous(); }

bool done(const char *fn, qmm_status s) {
    if (s == QMM_OK) return true;
    PyObject *r = PyObject_CallFunction(g_error, "si", fn, (int)s);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", fn, (int)s);
    return false;
}

PyObject *set_error(PyObject *, PyObject *f) {
    Py_INCREF(f);
    Py_XSETREF(g_error, f);
    Py_RETURN_NONE;
}

// q4_group_matmul(X, data, K, N, group, out, ws) -> out
PyObject *group_matmul(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    NEED(n == 7, "seven arguments");
    Arg X(args[0]), W(args[1]), out(args[5], true), ws(args[6], true);
    int64_t K, N, group;
    if (!X.ok || !W.ok || !out.ok || !ws.ok || !integer(args[2], K) || !integer(args[3], N) || !integer(args[4], group))
        return nullptr;
    NEED(X->dim() == 2 && X->size(1) == K, "X must be [M, K]");
    const int xt = type_of(X.t);
    NEED(is_float(xt), "X must be fp32, fp16 or bf16");
    NEED(rows(X.t), "rows of X must be contiguous");
    // the C call takes the weight's sizes on trust
    NEED(W->scalar_type() == at::kByte && W->is_contiguous() &&
             size_in_bytes(W.t) >= qmm_q4_group_packed_bytes(K, N, group),
         "the packed weight must be contiguous uint8 and hold K x N of its group");
    NEED(is_workspace(ws.t), "ws must be contiguous");
    const int64_t M = X->size(0);
    const c10::Device d = X->device();
    if (!on_device(d, {&W.t, &out.t, &ws.t})) return nullptr;
    const c10::DeviceGuard guard(d);
    if (!out) out.t = at::empty({M, N}, X->options().requires_grad(false));
    NEED(out->scalar_type() == X->scalar_type() && out->dim() == 2 && out->size(0) == M && out->size(1) == N && rows(out.t),
         "out must be [M, N] of X's type with contiguous rows");
    const size_t need = qmm_q4_group_matmul_workspace_bytes(M, K, N, group, (qmm_dtype)xt);
    if (!ws && need) ws.t = bytes(need, d);
    if (!done("q4_group_matmul", q4_group_matmul(X.data(), (qmm_dtype)xt, M, K, ld(X.t), W.data(), N, group, out.data(),
                                                 ld(out.t), ws.data(), size_in_bytes(ws.t), stream_of(d))))
        return nullptr;
    return THPVariable_Wrap(out.t);
    END_HANDLE_TH_ERRORS
}

// kv_plan(ctx, new, table, free, page_size, max_tokens, free_begin, cu, slots, positions, info) -> (cu, slots, positions, info)
PyObject *plan(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    NEED(n == 11, "eleven arguments");
    Arg ctx(args[0]), add(args[1]), table(args[2]), free_pages(args[3]), begin(args[6], true);
    Arg out[4] = {{args[7], true}, {args[8], true}, {args[9], true}, {args[10], true}};
    int64_t page, max_tokens;
    if (!ctx.ok || !add.ok || !table.ok || !free_pages.ok || !begin.ok || !out[0].ok || !out[1].ok || !out[2].ok ||
        !out[3].ok || !integer(args[4], page) || !integer(args[5], max_tokens))
        return nullptr;
    NEED(vector_of(ctx.t, at::kInt) && vector_of(add.t, at::kInt) && vector_of(free_pages.t, at::kInt),
         "lengths and free_pages must be contiguous int32 vectors");
    const int64_t R = ctx->size(0);
    NEED(add->size(0) == R, "new_lens must have the length of ctx_lens");
    NEED(table->dim() == 2 && table->size(0) == R && table->scalar_type() == at::kInt, "block_table must be int32 [R, width]");
    NEED(rows(table.t), "rows of block_table must be contiguous");
    NEED(!begin || (begin->scalar_type() == at::kInt && begin->numel() == 1), "free_begin must be one int32");
    const c10::Device d = ctx->device();
    if (!on_device(d, {&add.t, &table.t, &free_pages.t, &begin.t})) return nullptr;
    const c10::DeviceGuard guard(d);
    const int64_t sizes[4] = {R + 1, max_tokens, max_tokens, 4};
    const at::ScalarType types[4] = {at::kInt, at::kLong, at::kInt, at::kInt};
    NEED(max_tokens >= 0, "max_tokens must not be negative");
    const bool given = (bool)out[0];
    for (int i = 0; i < 4; ++i) {
        if (!given) out[i].t = at::empty({sizes[i]}, at::TensorOptions().dtype(types[i]).device(d));
        NEED(out[i] && out[i]->dim() == 1 && out[i]->size(0) == sizes[i] && out[i]->scalar_type() == types[i] &&
                 out[i]->is_contiguous() && out[i]->device() == d,
             "out must hold cu_new [R + 1], slots (int64) and positions [max_tokens] and info [4]");
    }
    if (!done("kv_plan",
              kv_plan((const int32_t *)ctx.data(), (const int32_t *)add.data(), R, (int32_t *)table.data(), ld(table.t),
                      table->size(1), page, (const int32_t *)free_pages.data(), free_pages->size(0), (const int32_t *)begin.data(),
                      max_tokens, (int32_t *)out[0].data(), (int64_t *)out[1].data(), (int32_t *)out[2].data(),
                      (int32_t *)out[3].data(), stream_of(d))))
        return nullptr;
    PyObject *r = PyTuple_New(4);
    if (!r) return nullptr;
    for (int i = 0; i < 4; ++i) {
        PyObject *o = given ? args[7 + i] : THPVariable_Wrap(out[i].t);
        if (given) Py_INCREF(o);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i, o);
    }
    return r;
    END_HANDLE_TH_ERRORS
}

// Whether two tensors of one shape have the same strides wherever a stride counts.
bool alike(const at::Tensor &a, const at::Tensor &b) {
    for (int64_t i = 0; i < a.dim(); ++i)
        if (a.stride(i) != b.stride(i) && a.size(i) > 1) return false;
    return true;
}

// The C description of a paged cache; NULL or what is wrong with it.
const char *describe(const Arg &k, const Arg &v, const Arg &ks, const Arg &vs, qmm_kv_cache &c) {
    if (k->dim() != 4 || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type())
        return "k_cache and v_cache must be [pages, page_size, heads, dim] of one type";
    const int ct = type_of(k.t);
    if (ct == kNone || ct == QMM_T_F32) return "the cache must be fp16, bf16 or int8";
    if (!alike(k.t, v.t) || (k->stride(3) != 1 && k->size(3) != 1)) return "k_cache and v_cache must share strides, rows contiguous";
    c = {};
    c.k = k.data();
    c.v = v.data();
    c.type = (qmm_dtype)ct;
    c.num_pages = k->size(0);
    c.page_size = k->size(1);
    c.n_heads = k->size(2);
    c.head_dim = k->size(3);
    c.page_stride = k->stride(0);
    c.token_stride = k->stride(1);
    c.head_stride = k->stride(2);
    if (ct == QMM_T_S8) {
        if (!ks || !vs) return "an int8 cache needs k_scale and v_scale";
        if (ks->dim() != 3 || ks->size(0) != c.num_pages || ks->size(1) != c.page_size || ks->size(2) != c.n_heads ||
            vs->sizes() != ks->sizes() || ks->scalar_type() != at::kFloat || vs->scalar_type() != at::kFloat || !alike(ks.t, vs.t))
            return "scales must be fp32 [pages, page_size, heads] with equal strides";
        c.k_scale = (float *)ks.data();
        c.v_scale = (float *)vs.data();
        c.scale_page_stride = ks->stride(0);
        c.scale_token_stride = ks->stride(1);
        c.scale_head_stride = ks->stride(2);
    } else if (ks || vs) {
        return "only an int8 cache has scales";
    }
    return nullptr;
}

// kv_append(K, V, slots, k_cache, v_cache, k_scale, v_scale)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    NEED(n == 7, "seven arguments");
    Arg K(args[0]), V(args[1]), slots(args[2]), kc(args[3]), vc(args[4]), ks(args[5], true), vs(args[6], true);
    if (!K.ok || !V.ok || !slots.ok || !kc.ok || !vc.ok || !ks.ok || !vs.ok) return nullptr;
    qmm_kv_cache c;
    const char *wrong = describe(kc, vc, ks, vs, c);
    NEED(!wrong, wrong);
    const int xt = type_of(K.t);
    NEED(is_float(xt) && V->scalar_type() == K->scalar_type(), "K and V must both be fp32, fp16 or bf16");
    NEED(K->dim() == 3 && K->sizes() == V->sizes() && K->size(1) == c.n_heads && K->size(2) == c.head_dim,
         "K and V must be [T, heads, dim]");
    const int64_t T = K->size(0);
    NEED(slots->dim() == 1 && slots->size(0) == T && slots->scalar_type() == at::kLong && slots->is_contiguous(),
         "slots must be int64 [T]");
    NEED(rows(K.t) && rows(V.t), "rows of K and V must be contiguous");
    const c10::Device d = K->device();
    if (!on_device(d, {&V.t, &slots.t, &kc.t, &vc.t, &ks.t, &vs.t})) return nullptr;
    const c10::DeviceGuard guard(d);
    if (!done("kv_append", kv_append(K.data(), K->stride(0), K->stride(1), V.data(), V->stride(0), V->stride(1), (qmm_dtype)xt, T,
                                     (const int64_t *)slots.data(), &c, stream_of(d))))
        return nullptr;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// tree_attention(Q, k_cache, v_cache, table, ctx, cu, mask, scale, k_scale, v_scale, out, ws) -> out
PyObject *attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    NEED(n == 12, "twelve arguments");
    Arg Q(args[0]), kc(args[1]), vc(args[2]), table(args[3]), ctx(args[4]), cu(args[5]), mask(args[6], true), ks(args[8], true),
        vs(args[9], true), out(args[10], true), ws(args[11], true);
    if (!Q.ok || !kc.ok || !vc.ok || !table.ok || !ctx.ok || !cu.ok || !mask.ok || !ks.ok || !vs.ok || !out.ok || !ws.ok)
        return nullptr;
    qmm_kv_cache c;
    const char *wrong = describe(kc, vc, ks, vs, c);
    NEED(!wrong, wrong);
    NEED(Q->dim() == 3 && Q->size(2) == c.head_dim && rows(Q.t), "Q must be [T, q_heads, dim]");
    const int64_t T = Q->size(0), Hq = Q->size(1), D = Q->size(2);
    const int xt = type_of(Q.t);
    NEED(is_float(xt), "Q must be fp16 or bf16");
    NEED(is_workspace(ws.t), "ws must be contiguous");
    double scale = 1.0 / std::sqrt((double)(D > 0 ? D : 1));
    if (args[7] != Py_None) {
        scale = PyFloat_AsDouble(args[7]);
        if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    }
    NEED(ctx->dim() == 1 && ctx->scalar_type() == at::kInt && ctx->is_contiguous() && cu->dim() == 1 &&
             cu->scalar_type() == at::kInt && cu->size(0) == ctx->size(0) + 1 && cu->is_contiguous(),
         "ctx_lens and cu_new must be int32 [R] and [R + 1]");
    const int64_t R = ctx->size(0);
    NEED(table->dim() == 2 && table->size(0) == R && table->scalar_type() == at::kInt, "block_table must be int32 [R, width]");
    NEED(rows(table.t), "rows of block_table must be contiguous");
    int64_t cols = 0, ld_mask = 0;
    const void *mask_at = nullptr;
    if (mask) {
        NEED(mask->dim() == 2 && mask->size(0) == T && (mask->scalar_type() == at::kBool || mask->scalar_type() == at::kByte),
             "mask must be bool or uint8 [T, columns]");
        NEED(rows(mask.t), "rows of mask must be contiguous");
        cols = mask->size(1);
        ld_mask = ld(mask.t);
        mask_at = mask.data() ? mask.data() : cu.data();  // a mask of no columns has no memory, and is still a mask
    }
    const c10::Device d = Q->device();
    if (!on_device(d, {&kc.t, &vc.t, &ks.t, &vs.t, &table.t, &ctx.t, &cu.t, &mask.t, &out.t, &ws.t})) return nullptr;
    const c10::DeviceGuard guard(d);
    if (!out) out.t = at::empty({T, Hq, D}, Q->options().requires_grad(false));
    NEED(out->sizes() == Q->sizes() && out->scalar_type() == Q->scalar_type() && rows(out.t),
         "out must have Q's shape and type with contiguous rows");
    const size_t need = qmm_tree_attention_workspace_bytes(T, Hq, R, c.n_heads, D);
    if (!ws && need) ws.t = bytes(need, d);
    if (!done("tree_attention",
              tree_attention(Q.data(), Q->stride(0), Q->stride(1), (qmm_dtype)xt, T, Hq, &c, (const int32_t *)table.data(),
                             ld(table.t), table->size(1), (const int32_t *)ctx.data(), (const int32_t *)cu.data(), R,
                             (const uint8_t *)mask_at, ld_mask, cols, (float)scale, out.data(), out->stride(0), out->stride(1),
                             ws.data(), size_in_bytes(ws.t), stream_of(d))))
        return nullptr;
    return THPVariable_Wrap(out.t);
    END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"set_error", set_error, METH_O, nullptr},
    {"q4_group_matmul", (PyCFunction)(void (*)(void))group_matmul, METH_FASTCALL, nullptr},
    {"kv_plan", (PyCFunction)(void (*)(void))plan, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"tree_attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve() { return PyModule_Create(&kModule); }
