// moba_calls.cpp -- the usual call of an operator in one step from Python: its operands
// looked over, its results and scratch made, and the C entry point called.
//
// Bound: the host, where tokens are few: the GPU has 3 to 17 us of work then.  Measured, us from
// call to call, against the same steps in Python: norms of 3 tokens 6 and 18, the gradient of 517
// 12 and 32, appending one token 9 and 25, one of each of 64 sequences 11 (the GPU's time) and 26, four
// forks 15 (the GPU's) and 29.
// Nothing is decided here: whatever is not the plain case (another device than the current
// one, operands that a check stops at, arguments of another kind, a refusal by the entry point)
// gives None, and ops.py goes through the same call step by step and says what is wrong.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "moba.h"

namespace {

using at::ScalarType;
using at::Tensor;

// A new tensor straight from the allocator (by the dispatcher 0.4 us more each).
Tensor make_new(at::IntArrayRef sizes, ScalarType type, int device) {
    return at::detail::empty_cuda(sizes, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)device), std::nullopt);
}
// (which does not fill it, as torch can be told to)
bool fills() {
    const at::Context &c = at::globalContext();
    return c.deterministicAlgorithms() && c.deterministicFillUninitializedMemory();
}

// The operands of one call.  `ok` turns false at the first that is not the plain case.
struct Operands {
    bool ok = true;
    int device = -1;

    // the call's device is that of its first tensor, and the current one
    explicit Operands(PyObject *first) {
        ok = THPVariable_Check(first);
        if (!ok) return;
        const Tensor t = THPVariable_Unpack(first);
        ok = t.is_cuda() && t.device().index() == c10::cuda::current_device() && !fills();
        device = t.device().index();
    }
    Tensor any(PyObject *o, ScalarType type) {
        if (!ok || !THPVariable_Check(o)) return fail();
        Tensor t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.device().index() != device || t.scalar_type() != type || t.layout() != at::kStrided)
            return fail();
        return t;
    }
    Tensor dense(PyObject *o, ScalarType type) {
        Tensor t = any(o, type);
        return ok && !t.is_contiguous() ? fail() : t;
    }
    // [T, H, D] bf16, a token's heads dense, and the elements between tokens
    Tensor heads(PyObject *o, long long *stride) {
        Tensor t = any(o, at::kBFloat16);
        if (!ok || t.dim() != 3) return fail();
        const long long T = t.size(0), H = t.size(1), D = t.size(2), w = H * D;
        if (T < 1 || w < 1 || t.stride(2) != 1 || t.stride(1) != D || (T > 1 && t.stride(0) < w)) return fail();
        *stride = T > 1 ? t.stride(0) : w;
        return t;
    }
    // norm weights [D], of one type; None where they may be missing
    Tensor weight(PyObject *o, long long D, int *bits) {
        if (!ok || !THPVariable_Check(o)) return fail();
        const ScalarType type = THPVariable_Unpack(o).scalar_type();
        const int mine = type == at::kFloat ? 32 : type == at::kBFloat16 ? 16 : 0;
        if (mine == 0 || (*bits && *bits != mine)) return fail();
        *bits = mine;
        Tensor t = dense(o, type);
        return ok && (t.dim() != 1 || t.size(0) != D) ? fail() : t;
    }
    int integer(PyObject *o) {
        if (!ok || !PyLong_CheckExact(o)) return no();
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(o, &over);
        return over || v < INT_MIN || v > INT_MAX ? no() : (int)v;
    }
    float number(PyObject *o) {
        if (!ok || !PyFloat_CheckExact(o)) return (float)no();
        return (float)PyFloat_AS_DOUBLE(o);
    }
    int flag(PyObject *o) {
        if (!ok || (o != Py_True && o != Py_False)) return no();
        return o == Py_True;
    }
    void need(bool what) { ok = ok && what; }

  private:
    Tensor fail() {
        ok = false;
        return {};
    }
    int no() {
        ok = false;
        return 0;
    }
};

// Results and scratch are made, and the call is enqueued, with the interpreter let go.
struct Released {
    PyThreadState *state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
};

// A result: the caller's tensor (whose checks are the operands'), or a new one.
struct Result {
    PyObject *given;
    Tensor t;
    Result(PyObject *o) : given(o == Py_None ? nullptr : o) {}
    bool made() const { return given == nullptr; }
    void make(at::IntArrayRef sizes, ScalarType type, int device) {
        if (made()) t = make_new(sizes, type, device);
    }
    PyObject *object() {
        if (made()) return THPVariable_Wrap(std::move(t));
        Py_INCREF(given);
        return given;
    }
};

void *stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
void *address(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

Tensor scratch(size_t bytes, int device) { return make_new({(int64_t)bytes}, at::kByte, device); }

// What is left of a call: None where the entry point refused it, its code where CUDA failed, or
// the results.
template <int N>
PyObject *answer(int rc, Result *const (&results)[N]) {
    if (rc == MOBA_ERR_CUDA) return PyLong_FromLong(rc);
    if (rc != MOBA_OK) Py_RETURN_NONE;
    if (N == 1) return results[0]->object();
    PyObject *tuple = PyTuple_New(N);
    if (!tuple) return nullptr;
    for (int i = 0; i < N; ++i) {
        PyObject *o = results[i] ? results[i]->object() : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(tuple);
            return nullptr;
        }
        PyTuple_SET_ITEM(tuple, i, o);
    }
    return tuple;
}

// q, k, q_weight, k_weight, positions, freqs, eps, interleaved, magnitude, q_out, k_out
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 11) Py_RETURN_NONE;
    Operands x(a[0]);
    const bool has_k = a[1] != Py_None;
    long long qs = 0, ks = 0, qos = 0, kos = 0;
    const Tensor q = x.heads(a[0], &qs), k = has_k ? x.heads(a[1], &ks) : Tensor();
    if (!x.ok) Py_RETURN_NONE;
    const long long T = q.size(0), D = q.size(2);
    int bits = 0;
    const Tensor qw = x.weight(a[2], D, &bits), kw = has_k ? x.weight(a[3], D, &bits) : Tensor();
    const Tensor pos = x.dense(a[4], at::kInt), freqs = x.dense(a[5], at::kDouble);
    const float eps = x.number(a[6]), magnitude = x.number(a[8]);
    const int interleaved = x.flag(a[7]);
    Result qo(a[9]), ko(a[10]);
    if (!qo.made()) qo.t = x.heads(a[9], &qos);
    if (has_k && !ko.made()) ko.t = x.heads(a[10], &kos);
    x.need(T <= INT_MAX && q.size(1) <= INT_MAX && (has_k || (ko.made() && a[3] == Py_None)));
    x.need(x.ok && pos.numel() == T && freqs.numel() <= 1024 && (!has_k || (k.size(0) == T && k.size(2) == D)));
    x.need(x.ok && (qo.made() || qo.t.sizes() == q.sizes()) && (!has_k || ko.made() || ko.t.sizes() == k.sizes()));
    if (!x.ok) Py_RETURN_NONE;
    int rc;
    {
        Released r;
        qo.make(q.sizes(), at::kBFloat16, x.device);
        if (has_k) ko.make(k.sizes(), at::kBFloat16, x.device);
        rc = moba_qk_norm_rope(address(q), address(k), address(qo.t), address(ko.t), address(qw), address(kw), bits, eps,
                               static_cast<const int32_t *>(address(pos)), static_cast<const double *>(address(freqs)),
                               (int)T, (int)q.size(1), has_k ? (int)k.size(1) : 0, (int)D, 2 * (int)freqs.numel(),
                               interleaved, magnitude, qs, ks, qos, kos, stream_of(x.device));
    }
    return answer(rc, {&qo, has_k ? &ko : nullptr});
    END_HANDLE_TH_ERRORS
}

// dq_out, dk_out, q, k, q_weight, k_weight, positions, freqs, eps, interleaved, magnitude, dq, dk,
// dq_weight, dk_weight, workspace
PyObject *qk_norm_rope_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 16) Py_RETURN_NONE;
    Operands x(a[2]);
    const bool has_k = a[3] != Py_None;
    x.need(has_k == (a[1] != Py_None) && (has_k || (a[5] == Py_None && a[12] == Py_None && a[14] == Py_None)));
    long long qs = 0, ks = 0, ys = 0, zs = 0, qos = 0, kos = 0;
    const Tensor q = x.heads(a[2], &qs), dy = x.heads(a[0], &ys);
    const Tensor k = has_k ? x.heads(a[3], &ks) : Tensor(), dz = has_k ? x.heads(a[1], &zs) : Tensor();
    if (!x.ok) Py_RETURN_NONE;
    const long long T = q.size(0), D = q.size(2);
    int bits = 0;
    const Tensor qw = x.weight(a[4], D, &bits), kw = has_k ? x.weight(a[5], D, &bits) : Tensor();
    const Tensor pos = x.dense(a[6], at::kInt), freqs = x.dense(a[7], at::kDouble);
    const float eps = x.number(a[8]), magnitude = x.number(a[10]);
    const int interleaved = x.flag(a[9]);
    Result qo(a[11]), ko(a[12]), wq(a[13]), wk(a[14]);
    int w32 = 32;
    if (!qo.made()) qo.t = x.heads(a[11], &qos);
    if (has_k && !ko.made()) ko.t = x.heads(a[12], &kos);
    if (!wq.made()) wq.t = x.weight(a[13], D, &w32);
    if (has_k && !wk.made()) wk.t = x.weight(a[14], D, &w32);
    const Tensor given = a[15] == Py_None ? Tensor() : x.dense(a[15], at::kByte);
    x.need(T <= INT_MAX && q.size(1) <= INT_MAX);
    x.need(x.ok && pos.numel() == T && freqs.numel() <= 1024 && dy.sizes() == q.sizes());
    x.need(x.ok && (!has_k || (k.size(0) == T && k.size(2) == D && dz.sizes() == k.sizes())));
    x.need(x.ok && (qo.made() || qo.t.sizes() == q.sizes()) && (!has_k || ko.made() || ko.t.sizes() == k.sizes()));
    if (!x.ok) Py_RETURN_NONE;
    const int Hq = (int)q.size(1), Hk = has_k ? (int)k.size(1) : 0;
    size_t need = 0;
    if (!given.defined()) {
        need = moba_qk_norm_rope_bwd_workspace_size((int)T, Hq, Hk, (int)D);
        if (need == 0) Py_RETURN_NONE;
    }
    int rc;
    {
        Released r;
        qo.make(q.sizes(), at::kBFloat16, x.device);
        wq.make({D}, at::kFloat, x.device);
        if (has_k) {
            ko.make(k.sizes(), at::kBFloat16, x.device);
            wk.make({D}, at::kFloat, x.device);
        }
        const Tensor ws = given.defined() ? given : scratch(need, x.device);
        rc = moba_qk_norm_rope_bwd(address(dy), address(dz), address(q), address(k), address(qw), address(kw),
                                   address(qo.t), address(ko.t), static_cast<float *>(address(wq.t)),
                                   static_cast<float *>(address(wk.t)), bits, eps,
                                   static_cast<const int32_t *>(address(pos)),
                                   static_cast<const double *>(address(freqs)), (int)T, Hq, Hk, (int)D,
                                   2 * (int)freqs.numel(), interleaved, magnitude, ys, zs, qs, ks, qos, kos, address(ws),
                                   (size_t)ws.numel(), stream_of(x.device));
    }
    return answer(rc, {&qo, has_k ? &ko : nullptr, &wq, has_k ? &wk : nullptr});
    END_HANDLE_TH_ERRORS
}

// The pools of one layer and the sequences' tables.
struct Paged {
    Tensor k, v, kbar, table, cu, lens;
    int P = 0, Hkv = 0, ps = 0, D = 0, n = 0, mp = 0;
    Paged(Operands &x, PyObject *kp, PyObject *vp, PyObject *bar, PyObject *t, PyObject *c, PyObject *l) {
        k = x.dense(kp, at::kBFloat16);
        v = x.dense(vp, at::kBFloat16);
        if (bar != Py_None) kbar = x.dense(bar, at::kFloat);
        table = x.dense(t, at::kInt);
        cu = x.dense(c, at::kInt);
        lens = x.dense(l, at::kInt);
        x.need(x.ok && k.dim() == 4 && v.sizes() == k.sizes() && table.dim() == 2 && k.numel() > 0);
        if (!x.ok) return;
        const long long s[6] = {k.size(0), k.size(1), k.size(2), k.size(3), lens.numel(), table.size(1)};
        for (long long i : s) x.need(i <= INT_MAX);
        P = (int)s[0], Hkv = (int)s[1], ps = (int)s[2], D = (int)s[3], n = (int)s[4], mp = (int)s[5];
        x.need(table.size(0) == n && cu.numel() == n + 1ll);
        if (kbar.defined()) x.need(kbar.dim() == 3 && kbar.size(0) == P && kbar.size(1) == Hkv && kbar.size(2) == D);
    }
    const int32_t *ints(const Tensor &t) const { return static_cast<const int32_t *>(address(t)); }
};

// q, k, v, k_pages, v_pages, kbar_pages, page_table, cu_new, cache_lens, max_new, block_size, freqs,
// positions, q_weight, k_weight, eps, interleaved, magnitude, q_out
PyObject *paged_append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 19) Py_RETURN_NONE;
    Operands x(a[3]);
    long long qs = 0, ks = 0, vs = 0, qos = 0;
    const Tensor q = x.heads(a[0], &qs), k = x.heads(a[1], &ks), v = x.heads(a[2], &vs);
    const Paged c(x, a[3], a[4], a[5], a[6], a[7], a[8]);
    if (!x.ok) Py_RETURN_NONE;
    const long long total = q.size(0);
    const int max_new = x.integer(a[9]), block = x.integer(a[10]);
    const Tensor freqs = x.dense(a[11], at::kDouble), pos = a[12] == Py_None ? Tensor() : x.dense(a[12], at::kInt);
    int bits = 0;
    const Tensor qw = a[13] == Py_None ? Tensor() : x.weight(a[13], c.D, &bits);
    const Tensor kw = a[14] == Py_None ? Tensor() : x.weight(a[14], c.D, &bits);
    const float eps = x.number(a[15]), magnitude = x.number(a[17]);
    const int interleaved = x.flag(a[16]);
    Result qo(a[18]);
    if (!qo.made()) qo.t = x.heads(a[18], &qos);
    x.need(total <= INT_MAX && q.size(1) <= INT_MAX && q.size(2) == c.D && k.sizes() == v.sizes());
    x.need(k.size(0) == total && k.size(1) == c.Hkv && k.size(2) == c.D);
    x.need(x.ok && freqs.numel() <= 1024 && (!pos.defined() || pos.numel() == total));
    x.need(x.ok && (qo.made() || qo.t.sizes() == q.sizes()));
    if (!x.ok) Py_RETURN_NONE;
    int rc;
    {
        Released r;
        qo.make(q.sizes(), at::kBFloat16, x.device);
        rc = moba_paged_append_rope(address(q), address(k), address(v), address(qo.t), address(c.k), address(c.v),
                                    static_cast<float *>(address(c.kbar)), c.ints(c.table), c.ints(c.cu),
                                    c.ints(c.lens), c.ints(pos), static_cast<const double *>(address(freqs)),
                                    address(qw), address(kw), bits, eps, c.n, (int)total, max_new, (int)q.size(1), c.Hkv,
                                    c.D, 2 * (int)freqs.numel(), interleaved, magnitude, qs, ks, vs, qos, c.P, c.ps,
                                    c.mp, block, nullptr, stream_of(x.device));
    }
    return answer(rc, {&qo});
    END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, page_table, cu_new, cache_lens, max_new, cu_groups, prefix_lens, out, lse, workspace
PyObject *paged_attn_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 12) Py_RETURN_NONE;
    Operands x(a[1]);
    const Paged c(x, a[1], a[2], Py_None, a[3], a[4], a[5]);
    const Tensor q = x.dense(a[0], at::kBFloat16);
    const int max_new = x.integer(a[6]);
    const Tensor cg = x.dense(a[7], at::kInt), pre = x.dense(a[8], at::kInt);
    Result out(a[9]), lse(a[10]);
    if (!out.made()) out.t = x.dense(a[9], at::kBFloat16);
    if (!lse.made()) lse.t = x.dense(a[10], at::kFloat);
    const Tensor given = a[11] == Py_None ? Tensor() : x.dense(a[11], at::kByte);
    x.need(x.ok && q.dim() == 3 && q.numel() > 0 && q.size(2) == c.D && q.size(0) <= INT_MAX && q.size(1) <= INT_MAX);
    x.need(x.ok && pre.numel() < INT_MAX && cg.numel() == pre.numel() + 1);
    if (!x.ok) Py_RETURN_NONE;
    const int total = (int)q.size(0), Hq = (int)q.size(1), groups = (int)pre.numel();
    x.need(out.made() || out.t.sizes() == q.sizes());
    x.need(lse.made() || (lse.t.dim() == 2 && lse.t.size(0) == total && lse.t.size(1) == Hq));
    if (!x.ok) Py_RETURN_NONE;
    size_t need = 0;
    if (!given.defined()) {
        need = moba_paged_attn_shared_workspace_size(c.n, groups, total, max_new, Hq, c.Hkv, c.D, c.ps, c.mp);
        if (need == 0) Py_RETURN_NONE;
    }
    int rc;
    {
        Released r;
        const Tensor ws = given.defined() ? given : scratch(need, x.device);
        out.make(q.sizes(), at::kBFloat16, x.device);
        lse.make({total, Hq}, at::kFloat, x.device);
        rc = moba_paged_attn_shared(address(q), address(c.k), address(c.v), c.ints(c.table), c.ints(c.cu),
                                    c.ints(c.lens), c.ints(cg), c.ints(pre), address(out.t),
                                    static_cast<float *>(address(lse.t)), c.n, groups, total, max_new, Hq, c.Hkv, c.D,
                                    c.P, c.ps, c.mp, address(ws), (size_t)ws.numel(), stream_of(x.device));
    }
    return answer(rc, {&out, &lse});
    END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(qk_norm_rope), FAST(qk_norm_rope_bwd), FAST(paged_append_rope), FAST(paged_attn_shared),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "moba_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_moba_calls() { return PyModule_Create(&module); }
