// The draft calls' arguments from torch tensors: a CPython module that checks
// each tensor (type, device, layout, size), fills the C ABI's arguments and
// makes the call on torch's current stream.  The same in Python takes 4 to 10
// us a call on the machine's Arm cores, more than most of these kernels run.
//
// Each function takes its arguments by position (the named and default ones are
// in __init__.py) and returns the abg_status; a wrong tensor is a ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <stdexcept>
#include <string>

#include "../../include/abg.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Wrong : std::runtime_error {
    using std::runtime_error::runtime_error;
};

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw Wrong(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

const char *type_name(ScalarType t) {
    switch (t) {
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    default: return "the other tensors' type";
    }
}

// Device pointer of a contiguous CUDA tensor of this type with at least numel elements.
void *need(const Tensor &t, ScalarType type, int64_t numel, const char *name) {
    if (t.scalar_type() == type && t.is_cuda() && t.is_contiguous() && t.numel() >= numel) return t.data_ptr();
    throw Wrong(std::string(name) + " must be a contiguous " + type_name(type) + " CUDA tensor of at least " +
                std::to_string(numel) + " elements");
}
template <typename P>
P *need(PyObject *o, ScalarType type, int64_t numel, const char *name) {
    return static_cast<P *>(need(tensor(o, name), type, numel, name));
}
template <typename P>
P *need_or_null(PyObject *o, ScalarType type, int64_t numel, const char *name) {
    return o == Py_None ? nullptr : need<P>(o, type, numel, name);
}
int32_t *i32(PyObject *o, int64_t numel, const char *name) { return need<int32_t>(o, ScalarType::Int, numel, name); }

int abg_type(const Tensor &t, const char *name) {
    switch (t.scalar_type()) {
    case ScalarType::Float: return ABG_SB_F32;
    case ScalarType::BFloat16: return ABG_SB_BF16;
    case ScalarType::Half: return ABG_SB_F16;
    default: throw Wrong(std::string(name) + " must be float32, bfloat16 or float16");
    }
}

int64_t number(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Wrong("a size must be an integer");
    }
    return v;
}

// The stream given as a handle, or (None) torch's current one on t's device
// (t has been checked to be on one).
void *stream_of(PyObject *o, const Tensor &t) {
    if (o != Py_None) return reinterpret_cast<void *>(static_cast<uintptr_t>(number(o)));
    return c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
}

// The library's call, without the interpreter's lock: a launch waits while the
// stream's queue is full, and what it waits for may need the lock.
template <typename F>
int unlocked(F call) {
    PyThreadState *const state = PyEval_SaveThread();
    const int status = call();
    PyEval_RestoreThread(state);
    return status;
}

struct Caches {
    int type;
    ScalarType scalar;
    int64_t pages, Hkv, page, D;
    void *K, *V;
};
Caches caches(PyObject *k, PyObject *v) {
    const Tensor &K = tensor(k, "Kc"), &V = tensor(v, "Vc");
    if (K.dim() != 4 || V.sizes() != K.sizes() || V.scalar_type() != K.scalar_type())
        throw Wrong("the caches must be [pages][Hkv][page][D] tensors of one shape and type");
    const ScalarType s = K.scalar_type();
    return {abg_type(K, "Kc"), s,         K.size(0), K.size(1), K.size(2), K.size(3), need(K, s, 0, "Kc"),
            need(V, s, 0, "Vc")};
}

// A [rows][heads][D] CUDA tensor with contiguous columns.
struct Rows {
    const void *p;
    int64_t rows, row, head;
};
Rows strided(PyObject *o, int64_t heads, int64_t D, ScalarType type, const char *name) {
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || !t.is_cuda() || t.dim() != 3 || t.size(1) != heads || t.size(2) != D ||
        t.stride(2) != 1)
        throw Wrong(std::string(name) + " must be a " + type_name(type) + " CUDA tensor [rows][" +
                    std::to_string(heads) + "][" + std::to_string(D) + "] with contiguous columns");
    // (the stride of a single row or head is never used, and can be anything)
    return {t.data_ptr(), t.size(0), t.size(0) > 1 ? t.stride(0) : heads * D, heads > 1 ? t.stride(1) : D};
}

int page_plan(PyObject *const *a) {
    const Tensor &lens = tensor(a[0], "lens"), &ring = tensor(a[5], "ring"), &table = tensor(a[6], "table"),
                 &slots = tensor(a[8], "slots");
    const int64_t B = lens.numel(), N = slots.numel(), R = ring.numel(), width = B ? table.numel() / B : 0;
    auto *lens_p = static_cast<int32_t *>(need(lens, ScalarType::Int, B, "lens"));
    auto *add = i32(a[1], B, "add"), *cu = i32(a[2], B + 1, "cu"), *held = i32(a[3], B, "held");
    auto *ends = need<int64_t>(a[4], ScalarType::Long, 2, "ends");
    auto *ring_p = static_cast<int32_t *>(need(ring, ScalarType::Int, R, "ring"));
    auto *table_p = static_cast<int32_t *>(need(table, ScalarType::Int, 0, "table"));
    auto *slots_p = static_cast<int64_t *>(need(slots, ScalarType::Long, N, "slots"));
    auto *pos = i32(a[9], N, "pos"), *lens_out = i32(a[10], B, "lens_out"), *held_out = i32(a[11], B, "held_out");
    auto *ends_out = need<int64_t>(a[12], ScalarType::Long, 2, "ends_out");
    auto *info = i32(a[13], 2, "info");
    const int64_t page = number(a[7]);
    void *stream = stream_of(a[14], lens);
    return unlocked([&] {
        return abg_page_plan(lens_p, add, cu, held, ends, ring_p, table_p, slots_p, pos, lens_out, held_out, ends_out,
                             info, B, N, page, width, R, stream);
    });
}

int tree_plan(PyObject *const *a) {
    const Tensor &parent = tensor(a[0], "parent"), &lens = tensor(a[1], "lens"), &mask = tensor(a[3], "mask");
    const int64_t B = lens.numel(), N = parent.numel();
    if (mask.dim() != 2 || mask.size(0) != N) throw Wrong("mask must be [N][words]");
    auto *parent_p = static_cast<int32_t *>(need(parent, ScalarType::Int, N, "parent"));
    auto *lens_p = static_cast<int32_t *>(need(lens, ScalarType::Int, B, "lens"));
    auto *cu = i32(a[2], B + 1, "cu");
    auto *mask_p = static_cast<uint64_t *>(need(mask, ScalarType::Long, N, "mask"));
    auto *pos = i32(a[4], N, "pos");
    const int64_t words = mask.size(1);
    void *stream = stream_of(a[5], parent);
    return unlocked([&] { return abg_tree_plan(parent_p, lens_p, cu, mask_p, pos, B, N, words, stream); });
}

// k v Kc Vc slots rows q qo qn_w kn_w cos sin pos eps stream
int kv_put(PyObject *const *a) {
    if ((a[10] == Py_None) != (a[11] == Py_None)) throw Wrong("cos and sin must both be given, or neither");
    if ((a[6] == Py_None) != (a[7] == Py_None)) throw Wrong("q and qo must both be given, or neither");
    const Caches c = caches(a[2], a[3]);
    const Tensor &kt = tensor(a[0], "k");
    const ScalarType src = kt.scalar_type();
    const int src_type = abg_type(kt, "k");
    const Rows k = strided(a[0], c.Hkv, c.D, src, "k"), v = strided(a[1], c.Hkv, c.D, src, "v");
    abg_kv_put_args p = {};
    p.k = k.p, p.k_row = k.row, p.k_head = k.head;
    p.v = v.p, p.v_row = v.row, p.v_head = v.head;
    p.src_rows = std::min(k.rows, v.rows);
    p.N = a[5] != Py_None ? tensor(a[5], "rows").numel() : a[4] != Py_None ? tensor(a[4], "slots").numel() : p.src_rows;
    p.slots = need_or_null<int64_t>(a[4], ScalarType::Long, p.N, "slots");
    p.rows = need_or_null<int32_t>(a[5], ScalarType::Int, p.N, "rows");
    p.Hkv = c.Hkv, p.D = c.D, p.page = c.page, p.pages = c.pages, p.Kc = c.K, p.Vc = c.V, p.type = c.type;
    p.src_type = src_type;
    if (a[6] != Py_None) {
        const Tensor &qt = tensor(a[6], "q");
        p.Hq = qt.dim() == 3 ? qt.size(1) : 0;
        const Rows q = strided(a[6], p.Hq, c.D, src, "q");
        p.q = q.p, p.q_row = q.row, p.q_head = q.head;
        p.src_rows = std::min(p.src_rows, q.rows);
        p.qo = need<void>(a[7], c.scalar, p.N * p.Hq * c.D, "qo");
        p.qn_w = need_or_null<float>(a[8], ScalarType::Float, c.D, "qn_w");
    }
    p.kn_w = need_or_null<float>(a[9], ScalarType::Float, c.D, "kn_w");
    if (a[10] != Py_None) {
        const Tensor &cos = tensor(a[10], "cos"), &sin = tensor(a[11], "sin");
        for (const Tensor *t : {&cos, &sin})  // (or flat)
            if (t->dim() > 1 ? t->size(-1) != c.D / 2 : t->numel() % (c.D / 2) != 0)
                throw Wrong("cos and sin must be [positions][" + std::to_string(c.D / 2) + "]");
        p.cos_rows = cos.numel() / (c.D / 2);
        p.cos = static_cast<float *>(need(cos, ScalarType::Float, p.cos_rows * (c.D / 2), "cos"));
        p.sin = need<float>(a[11], ScalarType::Float, p.cos_rows * (c.D / 2), "sin");
        p.pos = i32(a[12], p.N, "pos");
    }
    const double eps = PyFloat_AsDouble(a[13]);
    if (eps == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Wrong("eps must be a number");
    }
    p.eps = static_cast<float>(eps);
    void *stream = stream_of(a[14], kt);
    return unlocked([&] { return abg_kv_put(&p, stream); });
}

// q Kc Vc table lens cu Kd Vd mask y max_span gate ysum ws stream
int tree_attn(PyObject *const *a) {
    const Caches c = caches(a[1], a[2]);
    const Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "table"), &lens = tensor(a[4], "lens"),
                 &Kd = tensor(a[6], "Kd"), &Vd = tensor(a[7], "Vd"), &mask = tensor(a[8], "mask"), &y = tensor(a[9], "y"),
                 &ws = tensor(a[13], "ws");
    if (q.dim() != 3 || q.size(2) != c.D || Kd.dim() != 3 || Kd.size(0) != c.Hkv || Kd.size(2) != c.D ||
        Vd.sizes() != Kd.sizes())
        throw Wrong("q must be [N][Hq][D], Kd and Vd [Hkv][drafts][D]");
    if (mask.dim() != 2) throw Wrong("mask must be [N][words]");
    const int64_t B = lens.numel(), N = q.size(0), Hq = q.size(1), n = N * Hq * c.D;
    abg_tree_attn_args p = {};
    p.q = need(q, c.scalar, n, "q"), p.Kc = c.K, p.Vc = c.V;
    p.table = static_cast<int32_t *>(need(table, ScalarType::Int, 0, "table"));
    p.lens = static_cast<int32_t *>(need(lens, ScalarType::Int, B, "lens"));
    p.cu = i32(a[5], B + 1, "cu");
    p.Kd = need(Kd, c.scalar, 0, "Kd"), p.Vd = need(Vd, c.scalar, 0, "Vd");
    p.mask = static_cast<uint64_t *>(need(mask, ScalarType::Long, N * mask.size(1), "mask"));
    p.y_type = abg_type(y, "y");
    p.y = need(y, y.scalar_type(), n, "y");
    p.gate = need_or_null<float>(a[11], ScalarType::Float, n, "gate");
    p.ysum = need_or_null<float>(a[12], ScalarType::Float, n / 64, "ysum");
    p.B = B, p.N = N, p.Hq = Hq, p.Hkv = c.Hkv, p.D = c.D, p.page = c.page, p.pages = c.pages;
    p.width = B ? table.numel() / B : 0, p.drafts = Kd.size(1), p.words = mask.size(1);
    p.max_span = number(a[10]), p.type = c.type;
    void *ws_p = need(ws, ScalarType::Byte, 0, "ws"), *stream = stream_of(a[14], q);
    const int64_t ws_bytes = ws.numel();
    return unlocked([&] { return abg_tree_attn(&p, ws_p, ws_bytes, stream); });
}

// logits tok parent cu best rows add last ws stream
int tree_accept(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "logits"), &add = tensor(a[6], "add"), &ws = tensor(a[8], "ws");
    if (x.dim() != 2 || x.scalar_type() != ScalarType::Float || !x.is_cuda() || (x.stride(1) != 1 && x.size(1) > 1))
        throw Wrong("logits must be a float32 CUDA tensor [N][V] with contiguous rows");
    const int64_t N = x.size(0), V = x.size(1), B = add.numel();
    auto *logits = static_cast<float *>(x.data_ptr());
    const int64_t ld = N > 1 ? x.stride(0) : V;
    auto *tok = i32(a[1], N, "tok"), *parent = i32(a[2], N, "parent"), *cu = i32(a[3], B + 1, "cu");
    auto *best = i32(a[4], N, "best"), *rows = i32(a[5], N, "rows");
    auto *add_p = static_cast<int32_t *>(need(add, ScalarType::Int, B, "add"));
    auto *last = i32(a[7], B, "last");
    void *ws_p = need(ws, ScalarType::Byte, 0, "ws"), *stream = stream_of(a[9], x);
    const int64_t ws_bytes = ws.numel();
    return unlocked([&] {
        return abg_tree_accept(logits, ld, tok, parent, cu, best, rows, add_p, last, B, N, V, ws_p, ws_bytes, stream);
    });
}

template <int (*fn)(PyObject *const *), int kArgs>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    try {
        if (n != kArgs) throw Wrong("wrong number of arguments");
        return PyLong_FromLong(fn(args));
    } catch (const Wrong &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyMethodDef g_methods[] = {{"page_plan", nullptr, METH_FASTCALL, nullptr},   {"tree_plan", nullptr, METH_FASTCALL, nullptr},
                           {"kv_put", nullptr, METH_FASTCALL, nullptr},      {"tree_attn", nullptr, METH_FASTCALL, nullptr},
                           {"tree_accept", nullptr, METH_FASTCALL, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

template <int (*fn)(PyObject *const *), int kArgs>
PyCFunction entry() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&call<fn, kArgs>));
}

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
    g_methods[0].ml_meth = entry<page_plan, 15>();
    g_methods[1].ml_meth = entry<tree_plan, 6>();
    g_methods[2].ml_meth = entry<kv_put, 15>();
    g_methods[3].ml_meth = entry<tree_attn, 15>();
    g_methods[4].ml_meth = entry<tree_accept, 10>();
    return PyModule_Create(&g_module);
}
