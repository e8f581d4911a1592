// The torch functions around the paged cache (paged_plan, qk_norm_rope and its forms, kv4_append,
// kv4_gather, attn_decode_kv4): checks of their tensors, allocation of what they return, and the
// calls of libgqa's C entry points, whose addresses the package hands over once. In C++ because
// these calls take a few microseconds on the device: done in Python, the checks of a dozen
// tensors took 8 to 18 us a call on the host beside 4 to 7 us for the C call, launch included.
//
// A function returns what the package's function returns, or the status (an int) of a C call that
// refused. Wrong types raise TypeError, wrong shapes and devices ValueError.
#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../include/gqa.h"

namespace {

struct Refused {
    PyObject* type;
    std::string text;
};
[[noreturn]] void type_error(const std::string& text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

struct Functions {
    decltype(&gqa_paged_plan) paged_plan;
    decltype(&gqa_qk_norm_rope) norm_rope;
    decltype(&gqa_qk_norm_rope_append) append;
    decltype(&gqa_qk_norm_rope_bwd) bwd;
    decltype(&gqa_qk_norm_rope_bwd_workspace_bytes) bwd_bytes;
    decltype(&gqa_kv4_append) kv4_append;
    decltype(&gqa_kv4_gather) kv4_gather;
    decltype(&gqa_attn_decode_kv4) decode;
    decltype(&gqa_attn_decode_kv4_workspace_bytes) decode_bytes;
} gqa;

using Sizes = at::IntArrayRef;

std::string shape_text(Sizes s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// A tensor argument; its name for messages.
struct Arg {
    const at::Tensor* t;  // null: None
    const char* name;
    explicit operator bool() const { return t != nullptr; }
    const at::Tensor* operator->() const { return t; }
    template <class T = void>
    T* ptr() const { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
};
Arg tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return {&THPVariable_Unpack(o), name};
}
Arg tensor_or_none(PyObject* o, const char* name) { return o == Py_None ? Arg{nullptr, name} : tensor(o, name); }

int to_int(int64_t v, const char* name) {
    if (v > INT_MAX || v < INT_MIN) value_error(std::string(name) + " does not fit 32 bits");
    return (int)v;
}
int integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return to_int(v, name);
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

void has_shape(const Arg& a, Sizes shape) {
    if (a->sizes() != shape) value_error(std::string(a.name) + " must have the shape " + shape_text(shape) + ", not " + shape_text(a->sizes()));
}
void is_int32(const Arg& a) {
    if (a->scalar_type() != at::kInt || !a->is_contiguous()) type_error(std::string(a.name) + " must be a contiguous int32 tensor");
}
// A workspace's bytes are its elements': an expanded tensor has fewer behind it.
Arg workspace(PyObject* o) {
    const Arg a = tensor_or_none(o, "workspace");
    if (a && !a->is_contiguous()) value_error("workspace must be contiguous");
    return a;
}
// Layout of a bf16 operand [B, H, T, D], or [T, H, D] with three axes.
gqa_layout rows(const Arg& a, int dims) {
    if (a->scalar_type() != at::kBFloat16) type_error(std::string(a.name) + " must be a bf16 tensor");
    if (a->dim() != dims) value_error(std::string(a.name) + " must have " + std::to_string(dims) + " axes, not the shape " + shape_text(a->sizes()));
    const Sizes st = a->strides();
    if (st[dims - 1] != 1) value_error(std::string(a.name) + ": the last (D) axis must be contiguous");
    if (dims == 3) return {0, st[1], st[0]};
    return {st[0], st[1], st[2]};
}
// Layout of a 4-bit pool [pages, Hkv, page, D / 2 + 4].
gqa_kv4_layout pool4(const Arg& a, int64_t row) {
    if (a->scalar_type() != at::kByte) type_error(std::string(a.name) + " must be a uint8 tensor");
    if (a->dim() != 4 || a->size(3) != row)
        value_error(std::string(a.name) + " must be [pages, Hkv, page, " + std::to_string(row) + "], not " + shape_text(a->sizes()));
    if (a->stride(3) != 1 || a->stride(2) != row) value_error(std::string(a.name) + ": the rows of a page must be packed");
    return {a->stride(0), a->stride(1)};
}

// The device that all given tensors are on; it must be the current one.
int on_device(std::initializer_list<Arg> args) {
    int device = -1;
    for (const Arg& a : args) {
        if (!a) continue;
        if (!a->is_cuda()) type_error(std::string(a.name) + " must be a CUDA tensor");
        const int d = a->get_device();
        if (device == -1)
            device = d;
        else if (d != device)
            value_error(std::string(a.name) + " is on cuda:" + std::to_string(d) + ", the first operand on cuda:" + std::to_string(device));
    }
    if (device != c10::cuda::current_device())
        value_error("the operands are on cuda:" + std::to_string(device) + ", which is not the current device");
    return device;
}
void* stream_of(PyObject* stream, int device) {
    if (stream == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    void* p = PyLong_AsVoidPtr(stream);
    if (p == nullptr && PyErr_Occurred()) throw python_error();
    return p;
}

template <class F>
gqa_status without_gil(F f) {
    gqa_status st;
    Py_BEGIN_ALLOW_THREADS st = f();
    Py_END_ALLOW_THREADS return st;
}

PyObject* wrapped(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None); }
PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (r == nullptr) throw python_error();
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrapped(t));
    return r;
}

// Run f(args); a refusal, torch's errors and Python's become Python exceptions.
template <class F>
PyObject* call(Py_ssize_t have, Py_ssize_t want, F f) {
    HANDLE_TH_ERRORS
    try {
        if (have != want) type_error("expected " + std::to_string(want) + " arguments");
        // outputs and their views are plain tensors: nothing here is differentiated by torch
        at::AutoDispatchBelowADInplaceOrView below_autograd;
        return f();
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
PyObject* status(gqa_status st) { return PyLong_FromLong(st); }

// ---------------------------------------------------------------- plan
// seqlens, new_tokens, block_table, free_list, free_count, keep, out (5 tensors) or None, page_size,
// num_pages, max_tokens, stream
PyObject* py_paged_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 11, [&]() -> PyObject* {
        const Arg seqlens = tensor(a[0], "seqlens"), added = tensor(a[1], "new_tokens"), table = tensor(a[2], "block_table");
        const Arg list = tensor(a[3], "free_list"), count = tensor(a[4], "free_count"), keep = tensor_or_none(a[5], "keep");
        const int64_t S = seqlens->numel();
        for (const Arg& x : {seqlens, added, table, list, count}) is_int32(x);
        has_shape(seqlens, {S});
        has_shape(added, {S});
        if (keep) {
            is_int32(keep);
            has_shape(keep, {S});
        }
        if (table->dim() != 2 || table->size(0) != S || list->dim() != 1)
            value_error("block_table must be [S, max_pages] and free_list [capacity]");
        if (count->numel() != 1) value_error("free_count must hold one value");
        const int tokens = integer(a[9], "max_tokens");
        if (tokens <= 0) value_error("max_tokens must be positive");
        const int device = on_device({seqlens, added, table, list, count, keep});
        at::Tensor lens, cu, pos, slots, left;
        if (a[6] == Py_None) {
            // one allocation; positions and slots start on 16 bytes
            const int64_t at_lens = tokens, at_cu = at_lens + S, at_left = at_cu + S + 1, at_slots = (at_left + 1 + 3) / 4 * 4;
            const at::Tensor all = at::empty({at_slots + tokens}, seqlens->options());
            pos = all.narrow(0, 0, tokens);
            lens = all.narrow(0, at_lens, S);
            cu = all.narrow(0, at_cu, S + 1);
            left = all.narrow(0, at_left, 1);
            slots = all.narrow(0, at_slots, tokens);
        } else {
            static const char* const names[5] = {"seqlens_k", "cu_seqlens", "positions", "slots", "free_count"};
            const int64_t sizes[5] = {S, S + 1, tokens, tokens, 1};
            at::Tensor* const outs[5] = {&lens, &cu, &pos, &slots, &left};
            if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 5) type_error("out must be a PagedPlan");
            for (int i = 0; i < 5; ++i) {
                const Arg x = tensor(PyTuple_GET_ITEM(a[6], i), names[i]);
                is_int32(x);
                has_shape(x, {sizes[i]});
                on_device({seqlens, x});
                *outs[i] = *x.t;
            }
        }
        const int s = to_int(S, "seqlens"), max_pages = to_int(table->size(1), "max_pages"), capacity = to_int(list->numel(), "free_list");
        const int page = integer(a[7], "page_size"), pages = integer(a[8], "num_pages");
        void* const stream = stream_of(a[10], device);
        int* const p[5] = {lens.data_ptr<int>(), cu.data_ptr<int>(), pos.data_ptr<int>(), slots.data_ptr<int>(), left.data_ptr<int>()};
        const gqa_status st = without_gil([&] {
            return gqa.paged_plan(seqlens.ptr<int>(), keep.ptr<int>(), added.ptr<int>(), table.ptr<int>(), list.ptr<int>(),
                                  count.ptr<int>(), p[0], p[1], p[2], p[3], p[4], s, max_pages, page, pages, capacity, tokens, stream);
        });
        return st != GQA_OK ? status(st) : tuple_of({lens, cu, pos, slots, left});
    });
}

// ---------------------------------------------------------------- norm and rotation
// The seven arguments q_weight, k_weight, eps, cos, sin, positions, interleaved.
struct Rope {
    Arg q_weight, k_weight, cos, sin, positions;
    gqa_rope r{};
    Rope(PyObject* const* a, int64_t D, int64_t B, int64_t T)
        : q_weight(tensor_or_none(a[0], "q_weight")),
          k_weight(tensor_or_none(a[1], "k_weight")),
          cos(tensor_or_none(a[3], "cos")),
          sin(tensor_or_none(a[4], "sin")),
          positions(tensor_or_none(a[5], "positions")) {
        for (const Arg& w : {q_weight, k_weight})
            if (w && ((w->scalar_type() != at::kBFloat16 && w->scalar_type() != at::kFloat) || w->sizes() != Sizes{D} || !w->is_contiguous()))
                type_error(std::string(w.name) + " must be a contiguous bf16 or fp32 tensor [" + std::to_string(D) + "]");
        if (q_weight && k_weight && q_weight->scalar_type() != k_weight->scalar_type())
            type_error("q_weight and k_weight must have the same type");
        const Arg& w = q_weight ? q_weight : k_weight;
        r.q_weight = q_weight.ptr();
        r.k_weight = k_weight.ptr();
        r.weight_fp32 = w && w->scalar_type() == at::kFloat;
        r.eps = (float)number(a[2]);
        r.interleaved = truth(a[6]);
        if ((bool)cos != (bool)sin) value_error("cos and sin come together");
        if (!cos) {
            if (positions) value_error("positions need cos and sin");
            return;
        }
        for (const Arg& t : {cos, sin})
            if (t->scalar_type() != at::kFloat || t->dim() != 2 || t->sizes() != cos->sizes() || !t->is_contiguous())
                type_error("cos and sin must be contiguous fp32 tensors [positions, rot / 2]");
        r.cos = cos.ptr<float>();
        r.sin = sin.ptr<float>();
        r.n_positions = to_int(cos->size(0), "cos");
        r.rot = to_int(2 * cos->size(1), "cos");
        if (!positions) return;
        is_int32(positions);
        if (positions->sizes() == Sizes{B, T})
            r.positions_sb = T;
        else if (positions->sizes() != Sizes{T})
            value_error("positions must be [" + std::to_string(T) + "] or [" + std::to_string(B) + ", " + std::to_string(T) + "]");
        r.positions = positions.ptr<int>();
    }
};

// q [B, Hq, T, D] and k [B, Hkv, T, D].
struct QK {
    Arg q, k;
    gqa_layout lq, lk;
    int64_t B, Hq, Hkv, T, D;
    QK(PyObject* oq, PyObject* ok) : q(tensor(oq, "q")), k(tensor(ok, "k")), lq(rows(q, 4)), lk(rows(k, 4)) {
        B = q->size(0), Hq = q->size(1), T = q->size(2), D = q->size(3), Hkv = k->size(1);
        if (k->sizes() != Sizes{B, Hkv, T, D}) value_error("q and k must be [B, Hq, T, D] and [B, Hkv, T, D]");
    }
};
// An output like `like`: the given one, checked, or a contiguous new one.
struct Out {
    at::Tensor t;
    gqa_layout l;
    Out(const Arg& given, const Arg& like, int dims) {
        if (given) {
            l = rows(given, dims);
            has_shape(given, like->sizes());
            t = *given.t;
        } else {
            t = at::empty(like->sizes(), like->options());
            l = rows({&t, given.name}, dims);
        }
    }
};

// q, k, the seven, q_out, k_out, stream
PyObject* py_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 12, [&]() -> PyObject* {
        const QK x(a[0], a[1]);
        const Rope rope(a + 2, x.D, x.B, x.T);
        const Arg qo = tensor_or_none(a[9], "q_out"), ko = tensor_or_none(a[10], "k_out");
        const int device = on_device({x.q, x.k, qo, ko, rope.q_weight, rope.k_weight, rope.cos, rope.sin, rope.positions});
        const Out q(qo, x.q, 4), k(ko, x.k, 4);
        void* const stream = stream_of(a[11], device);
        const int B = to_int(x.B, "q"), T = to_int(x.T, "q"), Hq = to_int(x.Hq, "q"), Hkv = to_int(x.Hkv, "k"), D = to_int(x.D, "q");
        void *const pq = q.t.data_ptr(), *const pk = k.t.data_ptr();
        const gqa_status st = without_gil([&] {
            return gqa.norm_rope(x.q.ptr(), x.k.ptr(), pq, pk, B, T, Hq, Hkv, D, &x.lq, &x.lk, &q.l, &k.l, &rope.r, stream);
        });
        return st != GQA_OK ? status(st) : tuple_of({q.t, k.t});
    });
}

// dq_out, dk_out, q, k, the seven, dq, dk, workspace, stream
PyObject* py_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 15, [&]() -> PyObject* {
        const Arg gq = tensor(a[0], "dq_out"), gk = tensor(a[1], "dk_out");
        const QK x(a[2], a[3]);
        const gqa_layout lgq = rows(gq, 4), lgk = rows(gk, 4);
        has_shape(gq, x.q->sizes());
        has_shape(gk, x.k->sizes());
        const Rope rope(a + 4, x.D, x.B, x.T);
        const Arg oq = tensor_or_none(a[11], "dq"), ok = tensor_or_none(a[12], "dk"), ws = workspace(a[13]);
        const int device = on_device({gq, gk, x.q, x.k, oq, ok, ws, rope.q_weight, rope.k_weight, rope.cos, rope.sin, rope.positions});
        const Out dq(oq, x.q, 4), dk(ok, x.k, 4);
        const int B = to_int(x.B, "q"), T = to_int(x.T, "q"), Hq = to_int(x.Hq, "q"), Hkv = to_int(x.Hkv, "k"), D = to_int(x.D, "q");
        at::Tensor buf, dqw, dkw;
        void* ws_ptr = nullptr;
        size_t ws_bytes = 0;
        if (rope.q_weight || rope.k_weight) {
            // one allocation: the weights' gradients behind the workspace
            const int64_t need = ws ? 0 : (int64_t)gqa.bwd_bytes(B, T, Hq, Hkv, D) / 4;
            buf = at::empty({need + 2 * x.D}, x.q->options().dtype(at::kFloat));
            if (rope.q_weight) dqw = buf.narrow(0, need, x.D);
            if (rope.k_weight) dkw = buf.narrow(0, need + x.D, x.D);
            ws_ptr = ws ? ws.ptr() : buf.data_ptr();
            ws_bytes = ws ? ws->nbytes() : need * 4;
        }
        void* const stream = stream_of(a[14], device);
        void *const pq = dq.t.data_ptr(), *const pk = dk.t.data_ptr();
        float *const pqw = dqw.defined() ? dqw.data_ptr<float>() : nullptr, *const pkw = dkw.defined() ? dkw.data_ptr<float>() : nullptr;
        const gqa_status st = without_gil([&] {
            return gqa.bwd(gq.ptr(), gk.ptr(), x.q.ptr(), x.k.ptr(), pq, pk, pqw, pkw, B, T, Hq, Hkv, D, &lgq, &lgk, &x.lq, &x.lk,
                           &dq.l, &dk.l, &rope.r, ws_ptr, ws_bytes, stream);
        });
        return st != GQA_OK ? status(st) : tuple_of({dq.t, dk.t, dqw, dkw});
    });
}

// q, k, v, k_pool, v_pool, slots, the seven, pool_layout is NHD, q_out, stream
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 16, [&]() -> PyObject* {
        const Arg q = tensor(a[0], "q"), k = tensor(a[1], "k"), v = tensor(a[2], "v");
        const Arg kp = tensor(a[3], "k_pool"), vp = tensor(a[4], "v_pool"), slots = tensor(a[5], "slots");
        const gqa_layout lq = rows(q, 3), lk = rows(k, 3), lv = rows(v, 3);
        const int64_t n_tok = q->size(0), heads = k->size(1), dim = q->size(2);
        if (k->sizes() != Sizes{n_tok, heads, dim}) value_error("q and k must be [N, Hq, D] and [N, Hkv, D]");
        has_shape(v, k->sizes());
        is_int32(slots);
        has_shape(slots, {n_tok});
        gqa_layout lkp = rows(kp, 4), lvp = rows(vp, 4);
        has_shape(vp, kp->sizes());
        const bool nhd = truth(a[13]);
        if (nhd) {
            std::swap(lkp.sh, lkp.st);
            std::swap(lvp.sh, lvp.st);
        }
        if (kp->size(nhd ? 2 : 1) != heads || kp->size(3) != dim) value_error("the pools' heads and rows must be k's");
        const Rope rope(a + 6, dim, 1, n_tok);
        const Arg qo = tensor_or_none(a[14], "q_out");
        const int device = on_device({q, k, v, kp, vp, slots, qo, rope.q_weight, rope.k_weight, rope.cos, rope.sin, rope.positions});
        const Out out(qo, q, 3);
        void* const stream = stream_of(a[15], device);
        const int N = to_int(n_tok, "q"), Hq = to_int(q->size(1), "q"), Hkv = to_int(heads, "k"), D = to_int(dim, "q");
        const int page = to_int(kp->size(nhd ? 1 : 2), "k_pool"), pages = to_int(kp->size(0), "k_pool");
        void* const po = out.t.data_ptr();
        const gqa_status st = without_gil([&] {
            return gqa.append(q.ptr(), k.ptr(), v.ptr(), po, kp.ptr(), vp.ptr(), slots.ptr<int>(), N, Hq, Hkv, D, page, pages, &lq,
                              &lk, &lv, &out.l, &lkp, &lvp, &rope.r, stream);
        });
        return st != GQA_OK ? status(st) : wrapped(out.t);
    });
}

// ---------------------------------------------------------------- a cache in 4 bits
// k, v, k_pool, v_pool, slots, stream
PyObject* py_kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 6, [&]() -> PyObject* {
        const Arg k = tensor(a[0], "k"), v = tensor(a[1], "v"), kp = tensor(a[2], "k_pool"), vp = tensor(a[3], "v_pool");
        const Arg slots = tensor(a[4], "slots");
        const gqa_layout lk = rows(k, 3), lv = rows(v, 3);
        has_shape(v, k->sizes());
        is_int32(slots);
        has_shape(slots, {k->size(0)});
        const int64_t row = k->size(2) / 2 + 4;
        const gqa_kv4_layout lkp = pool4(kp, row), lvp = pool4(vp, row);
        has_shape(vp, kp->sizes());
        if (kp->size(1) != k->size(1)) value_error("the pools' heads must be k's");
        const int device = on_device({k, v, kp, vp, slots});
        void* const stream = stream_of(a[5], device);
        const int N = to_int(k->size(0), "k"), H = to_int(k->size(1), "k"), D = to_int(k->size(2), "k");
        const int page = to_int(kp->size(2), "k_pool"), pages = to_int(kp->size(0), "k_pool");
        return status(without_gil([&] {
            return gqa.kv4_append(k.ptr(), v.ptr(), kp.ptr(), vp.ptr(), slots.ptr<int>(), N, H, D, page, pages, &lk, &lv, &lkp, &lvp,
                                  stream);
        }));
    });
}

// k_pool, v_pool, slots, k, v, stream
PyObject* py_kv4_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 6, [&]() -> PyObject* {
        const Arg kp = tensor(a[0], "k_pool"), vp = tensor(a[1], "v_pool"), slots = tensor(a[2], "slots");
        if (kp->scalar_type() != at::kByte || kp->dim() != 4) type_error("k_pool must be a uint8 tensor [pages, Hkv, page, D / 2 + 4]");
        const int64_t row = kp->size(3), heads = kp->size(1), dim = 2 * (row - 4), n_tok = slots->numel();
        const gqa_kv4_layout lkp = pool4(kp, row), lvp = pool4(vp, row);
        has_shape(vp, kp->sizes());
        is_int32(slots);
        const Arg gk = tensor_or_none(a[3], "k"), gv = tensor_or_none(a[4], "v");
        const int device = on_device({kp, vp, slots, gk, gv});
        at::Tensor outs[2];
        gqa_layout l[2];
        for (int i = 0; i < 2; ++i) {
            const Arg& given = i ? gv : gk;
            if (given) {
                l[i] = rows(given, 3);
                has_shape(given, {n_tok, heads, dim});
                outs[i] = *given.t;
            } else {
                if (dim <= 0) value_error("k_pool must be [pages, Hkv, page, D / 2 + 4]");
                outs[i] = at::empty({n_tok, heads, dim}, kp->options().dtype(at::kBFloat16));
                l[i] = {0, dim, heads * dim};
            }
        }
        void* const stream = stream_of(a[5], device);
        const int N = to_int(n_tok, "slots"), H = to_int(heads, "k_pool"), D = to_int(dim, "k_pool");
        const int page = to_int(kp->size(2), "k_pool"), pages = to_int(kp->size(0), "k_pool");
        void *const pk = outs[0].data_ptr(), *const pv = outs[1].data_ptr();
        const gqa_status st = without_gil([&] {
            return gqa.kv4_gather(kp.ptr(), vp.ptr(), pk, pv, slots.ptr<int>(), N, H, D, page, pages, &lkp, &lvp, &l[0], &l[1], stream);
        });
        return st != GQA_OK ? status(st) : tuple_of({outs[0], outs[1]});
    });
}

// q, k_pool, v_pool, seqlens_k, block_table, max_seqlen_k or None, scale, window, out, workspace, stream;
// returns (out, workspace or None)
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 11, [&]() -> PyObject* {
        const Arg q = tensor(a[0], "q"), kp = tensor(a[1], "k_pool"), vp = tensor(a[2], "v_pool");
        const Arg lens = tensor(a[3], "seqlens_k"), table = tensor(a[4], "block_table");
        if (q->scalar_type() != at::kBFloat16 || !q->is_contiguous() || (q->dim() != 3 && q->dim() != 4))
            type_error("q must be a contiguous bf16 tensor [B, Hq, Tq, D] or [B, Hq, D]");
        const int64_t rows_q = q->dim() == 4 ? q->size(2) : 1, dim = q->size(-1), row = dim / 2 + 4;
        const gqa_kv4_layout lkp = pool4(kp, row), lvp = pool4(vp, row);
        has_shape(vp, kp->sizes());
        is_int32(lens);
        has_shape(lens, {q->size(0)});
        is_int32(table);
        if (table->dim() != 2 || table->size(0) != q->size(0)) value_error("block_table must be [B, max_pages]");
        const Arg given = tensor_or_none(a[8], "out"), ws = workspace(a[9]);
        const int device = on_device({q, kp, vp, lens, table, given, ws});
        at::Tensor out;
        if (given) {
            if (given->scalar_type() != at::kBFloat16 || given->sizes() != q->sizes() || !given->is_contiguous())
                value_error("out must be a contiguous bf16 tensor shaped like q");
            out = *given.t;
        } else {
            out = at::empty(q->sizes(), q->options());
        }
        const int B = to_int(q->size(0), "q"), Hq = to_int(q->size(1), "q"), Tq = to_int(rows_q, "q"), D = to_int(dim, "q");
        const int pages = to_int(kp->size(0), "k_pool"), Hkv = to_int(kp->size(1), "k_pool"), page = to_int(kp->size(2), "k_pool");
        const int max_pages = to_int(table->size(1), "block_table");
        const int longest = a[5] == Py_None ? to_int((int64_t)max_pages * page, "max_seqlen_k") : integer(a[5], "max_seqlen_k");
        const float scale = (float)number(a[6]);
        const int window = integer(a[7], "window");
        at::Tensor space;
        if (ws)
            space = *ws.t;
        else if (const size_t need = gqa.decode_bytes(B, Hq, Hkv, Tq, longest, D, window))
            space = at::empty({(int64_t)need}, kp->options());
        void* const stream = stream_of(a[10], device);
        void *const po = out.data_ptr(), *const pw = space.defined() ? space.data_ptr() : nullptr;
        const size_t bytes = space.defined() ? space.nbytes() : 0;
        const gqa_status st = without_gil([&] {
            return gqa.decode(q.ptr(), kp.ptr(), vp.ptr(), po, lens.ptr<int>(), table.ptr<int>(), page, pages, max_pages, B, Hq, Hkv,
                              Tq, longest, D, &lkp, &lvp, scale, window, pw, bytes, stream);
        });
        return st != GQA_OK ? status(st) : tuple_of({out, space});
    });
}

// The C entry points' addresses, in the order of Functions.
PyObject* py_set_functions(PyObject*, PyObject* const* a, Py_ssize_t n) {
    static_assert(sizeof(Functions) == 9 * sizeof(void*), "nine addresses");
    return call(n, 9, [&]() -> PyObject* {
        void* p[9];
        for (int i = 0; i < 9; ++i) {
            p[i] = PyLong_AsVoidPtr(a[i]);
            if (p[i] == nullptr) {
                if (PyErr_Occurred()) throw python_error();
                value_error("a null address");
            }
        }
        memcpy(&gqa, p, sizeof(gqa));
        Py_RETURN_NONE;
    });
}

#define GQA_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    GQA_METHOD("set_functions", py_set_functions), GQA_METHOD("paged_plan", py_paged_plan),
    GQA_METHOD("qk_norm_rope", py_norm_rope),      GQA_METHOD("qk_norm_rope_bwd", py_bwd),
    GQA_METHOD("qk_norm_rope_append", py_append),  GQA_METHOD("kv4_append", py_kv4_append),
    GQA_METHOD("kv4_gather", py_kv4_gather),       GQA_METHOD("attn_decode_kv4", py_decode),
    {nullptr, nullptr, 0, nullptr},
};
#ifndef GQA_BUILT_FOR
#define GQA_BUILT_FOR "built for an unknown torch"
#endif
// The module's documentation; the build looks it up in the file to see whether the module is of the
// installed versions.
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", GQA_BUILT_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
