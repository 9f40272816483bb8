// binding.cpp -- the binding's short way for the softmax with a relative position bias and the 8-bit
// checkpoints: one call from Python that checks its tensors, allocates the results with torch and calls the C ABI
// (by addresses that the Python side hands over, so that this module is linked to torch alone).  A call it does not
// take -- a tensor of another kind, shape or device than the call needs, another device than the current one -- gives
// None, and the Python binding goes its own way, which names what is wrong.  Everything here runs with the GIL held.
// On the host of a GB300 the Python way of a call costs 14 to 27 us, most of it attribute lookups, conversions and
// allocations from Python; this one 6 to 10.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <tuple>
#include <vector>

#include "ln.h"

namespace {

constexpr int64_t kBlock = 32;  // columns of a checkpoint's block

struct Abi {
    decltype(&ln_softmax_rel_fwd_f32) rel_fwd_f32;
    decltype(&ln_softmax_rel_fwd_bf16) rel_fwd_bf16;
    decltype(&ln_softmax_rel_bwd_f32) rel_bwd_f32;
    decltype(&ln_softmax_rel_bwd_bf16) rel_bwd_bf16;
    decltype(&ln_softmax_rel_workspace_bytes_f32) rel_ws_f32;
    decltype(&ln_softmax_rel_workspace_bytes_bf16) rel_ws_bf16;
    decltype(&ln_ckpt8_store_f32) store_f32;
    decltype(&ln_ckpt8_store_bf16) store_bf16;
    decltype(&ln_ckpt8_load_f32) load_f32;
    decltype(&ln_ckpt8_load_bf16) load_bf16;
    decltype(&ln_bwd_ckpt8_f32) ln_f32;
    decltype(&ln_bwd_ckpt8_bf16) ln_bf16_;
    decltype(&ln_rms_bwd_ckpt8_f32) rms_f32;
    decltype(&ln_rms_bwd_ckpt8_bf16) rms_bf16;
    decltype(&ln_bwd_ckpt8_workspace_bytes) norm_ws;
};
const char* const kNames[] = {
    "ln_softmax_rel_fwd_f32", "ln_softmax_rel_fwd_bf16", "ln_softmax_rel_bwd_f32", "ln_softmax_rel_bwd_bf16",
    "ln_softmax_rel_workspace_bytes_f32", "ln_softmax_rel_workspace_bytes_bf16", "ln_ckpt8_store_f32",
    "ln_ckpt8_store_bf16", "ln_ckpt8_load_f32", "ln_ckpt8_load_bf16", "ln_bwd_ckpt8_f32", "ln_bwd_ckpt8_bf16",
    "ln_rms_bwd_ckpt8_f32", "ln_rms_bwd_ckpt8_bf16", "ln_bwd_ckpt8_workspace_bytes"};
constexpr size_t kCount = sizeof(kNames) / sizeof(kNames[0]);
static_assert(sizeof(Abi) == kCount * sizeof(void*), "one address for each name");
Abi abi;

// The edges of (buckets, max_distance, bidirectional), as the Python side has worked them out.
std::map<std::tuple<int64_t, int64_t, bool>, std::vector<int32_t>> edges_of;

// A plain CUDA tensor, or null.
const at::Tensor* tensor(PyObject* o) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.defined() && t.is_cuda() && t.layout() == at::kStrided ? &t : nullptr;
}

bool is(const at::Tensor* t, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
    return t && t->scalar_type() == type && t->sizes() == shape && t->device() == dev && t->is_contiguous();
}

bool io_type(const at::Tensor& t) { return t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16; }

bool current(const at::Device& dev) { return c10::cuda::current_device() == dev.index(); }

ln_stream_t stream_of(const at::Device& dev) {
    return reinterpret_cast<ln_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* failed(ln_status st) { return PyLong_FromLong((long)st); }

int64_t blocks_of(int64_t cols) { return (cols + kBlock - 1) / kBlock; }

// A call's ln_rel, and what its tensors have to be.  `x` must be a contiguous [B, H, Lq, Lk].
bool fill_rel(const at::Tensor& x, PyObject* table_, PyObject* span_, PyObject* both_, PyObject* scale_, PyObject* causal_,
              PyObject* lens_, PyObject* q_pos_, ln_rel* r, const at::Tensor** table) {
    const at::Device dev = x.device();
    *table = tensor(table_);
    const at::Tensor* t = *table;
    if (!t || t->dim() != 2 || t->size(1) != x.size(1) || !t->is_contiguous() || t->device() != dev ||
        (t->scalar_type() != at::kFloat && t->scalar_type() != x.scalar_type()))
        return false;
    if (!PyLong_Check(span_) || !PyBool_Check(both_) || !PyBool_Check(causal_)) return false;
    if (!PyFloat_Check(scale_) && !PyLong_Check(scale_)) return false;
    const int64_t span = PyLong_AsLongLong(span_);
    const double scale = PyFloat_AsDouble(scale_);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    const bool both = both_ == Py_True;
    const auto found = edges_of.find(std::make_tuple(t->size(0), span, both));
    if (found == edges_of.end()) return false;
    r->lens = r->q_pos = nullptr;
    if (lens_ != Py_None) {
        const at::Tensor* l = tensor(lens_);
        if (!is(l, {x.size(0)}, at::kInt, dev)) return false;
        r->lens = static_cast<const int32_t*>(l->data_ptr());
    }
    if (q_pos_ != Py_None) {
        const at::Tensor* q = tensor(q_pos_);
        if (!is(q, {x.size(0)}, at::kInt, dev)) return false;
        r->q_pos = static_cast<const int32_t*>(q->data_ptr());
    }
    r->B = x.size(0);
    r->H = x.size(1);
    r->Lq = x.size(2);
    r->Lk = x.size(3);
    r->table = t->data_ptr();
    r->edges = found->second.data();
    r->n_edges = (int32_t)found->second.size();
    r->table_f32 = t->scalar_type() == at::kFloat;
    r->bidirectional = both;
    r->causal = causal_ == Py_True;
    r->scale = (float)scale;
    return true;
}

// rel_fwd(x, table, max_distance, bidirectional, scale, causal, lens, q_pos, mask, ckpt) -> (y, q, k)
PyObject* rel_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* x = n == 10 ? tensor(a[0]) : nullptr;
    if (!x || x->dim() != 4 || !io_type(*x) || !x->is_contiguous() || !current(x->device())) return none();
    ln_rel r;
    const at::Tensor* table;
    if (!fill_rel(*x, a[1], a[2], a[3], a[4], a[5], a[6], a[7], &r, &table)) return none();
    const void* mask = nullptr;
    int64_t mask_rows = 1;
    if (a[8] != Py_None) {
        const at::Tensor* m = tensor(a[8]);
        if (!m || m->dim() != 2 || !is(m, {m->size(0), r.Lk}, x->scalar_type(), x->device())) return none();
        mask = m->data_ptr();
        mask_rows = m->size(0);
    }
    if (!PyBool_Check(a[9])) return none();
    const bool ckpt = a[9] == Py_True, f32 = x->scalar_type() == at::kFloat;
    at::Tensor y = at::empty(x->sizes(), x->options()), q, k;
    if (ckpt) {
        const int64_t rows = r.B * r.H * r.Lq, blocks = blocks_of(r.Lk);
        q = at::empty({rows, blocks * kBlock}, x->options().dtype(at::kChar));
        k = at::empty({rows, blocks}, x->options().dtype(at::kByte));
    }
    int8_t* qp = ckpt ? static_cast<int8_t*>(q.data_ptr()) : nullptr;
    uint8_t* kp = ckpt ? static_cast<uint8_t*>(k.data_ptr()) : nullptr;
    const ln_stream_t s = stream_of(x->device());
    const ln_status st =
        f32 ? abi.rel_fwd_f32(&r, static_cast<const float*>(x->data_ptr()), r.Lk, static_cast<const float*>(mask), mask_rows,
                              static_cast<float*>(y.data_ptr()), r.Lk, qp, kp, s)
            : abi.rel_fwd_bf16(&r, static_cast<const ln_bf16*>(x->data_ptr()), r.Lk, static_cast<const ln_bf16*>(mask),
                               mask_rows, static_cast<ln_bf16*>(y.data_ptr()), r.Lk, qp, kp, s);
    if (st != LN_OK) return failed(st);
    if (!ckpt) return Py_BuildValue("(NOO)", THPVariable_Wrap(y), Py_None, Py_None);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(y), THPVariable_Wrap(q), THPVariable_Wrap(k));
    END_HANDLE_TH_ERRORS
}

// Whether q and k are a checkpoint of [rows, cols].
bool is_ckpt(const at::Tensor* q, const at::Tensor* k, int64_t rows, int64_t cols, const at::Device& dev) {
    const int64_t blocks = blocks_of(cols);
    return is(q, {rows, blocks * kBlock}, at::kChar, dev) && is(k, {rows, blocks}, at::kByte, dev);
}

// rel_bwd(dy, y, k, cols, table, max_distance, bidirectional, scale, causal, lens, q_pos, want_table) ->
// (dx, dtable); y the probabilities with k and cols None, or a checkpoint's integers with its bytes and columns
PyObject* rel_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* dy = n == 12 ? tensor(a[0]) : nullptr;
    const at::Tensor* y = n == 12 ? tensor(a[1]) : nullptr;
    if (!dy || !y || dy->dim() != 4 || !io_type(*dy) || !dy->is_contiguous() || !current(dy->device())) return none();
    ln_rel r;
    const at::Tensor* table;
    if (!fill_rel(*dy, a[4], a[5], a[6], a[7], a[8], a[9], a[10], &r, &table)) return none();
    const void* probs = nullptr;
    const int8_t* qp = nullptr;
    const uint8_t* kp = nullptr;
    if (a[2] == Py_None) {
        if (!is(y, dy->sizes(), dy->scalar_type(), dy->device())) return none();
        probs = y->data_ptr();
    } else {
        const at::Tensor* k = tensor(a[2]);
        const int64_t cols = PyLong_Check(a[3]) ? PyLong_AsLongLong(a[3]) : -1;
        if (PyErr_Occurred()) PyErr_Clear();
        if (cols != r.Lk || !is_ckpt(y, k, r.B * r.H * r.Lq, cols, dy->device())) return none();
        qp = static_cast<const int8_t*>(y->data_ptr());
        kp = static_cast<const uint8_t*>(k->data_ptr());
    }
    if (!PyBool_Check(a[11])) return none();
    const bool sums = a[11] == Py_True, f32 = dy->scalar_type() == at::kFloat;
    at::Tensor dx = at::empty(dy->sizes(), dy->options()), dtable, ws;
    void *tp = nullptr, *wp = nullptr;
    size_t bytes = 0;
    if (sums) {
        bytes = f32 ? abi.rel_ws_f32(&r) : abi.rel_ws_bf16(&r);
        dtable = at::empty(table->sizes(), table->options());
        ws = at::empty({(int64_t)bytes + 1}, dy->options().dtype(at::kByte));
        tp = dtable.data_ptr();
        wp = ws.data_ptr();
    }
    const ln_stream_t s = stream_of(dy->device());
    const ln_status st =
        f32 ? abi.rel_bwd_f32(&r, static_cast<const float*>(dy->data_ptr()), r.Lk, static_cast<const float*>(probs), r.Lk,
                              qp, kp, static_cast<float*>(dx.data_ptr()), r.Lk, tp, wp, bytes, s)
            : abi.rel_bwd_bf16(&r, static_cast<const ln_bf16*>(dy->data_ptr()), r.Lk, static_cast<const ln_bf16*>(probs),
                               r.Lk, qp, kp, static_cast<ln_bf16*>(dx.data_ptr()), r.Lk, tp, wp, bytes, s);
    if (st != LN_OK) return failed(st);
    if (!sums) return Py_BuildValue("(NO)", THPVariable_Wrap(dx), Py_None);
    return Py_BuildValue("(NN)", THPVariable_Wrap(dx), THPVariable_Wrap(dtable));
    END_HANDLE_TH_ERRORS
}

// store(x) -> (q, k)
PyObject* store(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* x = n == 1 ? tensor(a[0]) : nullptr;
    if (!x || x->dim() != 2 || !io_type(*x) || !x->is_contiguous() || !current(x->device())) return none();
    const int64_t rows = x->size(0), cols = x->size(1), blocks = blocks_of(cols);
    at::Tensor q = at::empty({rows, blocks * kBlock}, x->options().dtype(at::kChar));
    at::Tensor k = at::empty({rows, blocks}, x->options().dtype(at::kByte));
    int8_t* qp = static_cast<int8_t*>(q.data_ptr());
    uint8_t* kp = static_cast<uint8_t*>(k.data_ptr());
    const ln_stream_t s = stream_of(x->device());
    const ln_status st = x->scalar_type() == at::kFloat
                             ? abi.store_f32(static_cast<const float*>(x->data_ptr()), cols, rows, cols, qp, kp, s)
                             : abi.store_bf16(static_cast<const ln_bf16*>(x->data_ptr()), cols, rows, cols, qp, kp, s);
    if (st != LN_OK) return failed(st);
    return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(k));
    END_HANDLE_TH_ERRORS
}

// load(q, k, cols, f32) -> x
PyObject* load(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* q = n == 4 ? tensor(a[0]) : nullptr;
    const at::Tensor* k = n == 4 ? tensor(a[1]) : nullptr;
    if (!q || !k || q->dim() != 2 || !PyLong_Check(a[2]) || !PyBool_Check(a[3]) || !current(q->device())) return none();
    const int64_t cols = PyLong_AsLongLong(a[2]), rows = q->size(0);
    if (PyErr_Occurred()) PyErr_Clear();
    if (cols < 1 || !is_ckpt(q, k, rows, cols, q->device())) return none();
    const bool f32 = a[3] == Py_True;
    at::Tensor x = at::empty({rows, cols}, q->options().dtype(f32 ? at::kFloat : at::kBFloat16));
    const int8_t* qp = static_cast<const int8_t*>(q->data_ptr());
    const uint8_t* kp = static_cast<const uint8_t*>(k->data_ptr());
    const ln_stream_t s = stream_of(q->device());
    const ln_status st = f32 ? abi.load_f32(qp, kp, rows, cols, static_cast<float*>(x.data_ptr()), cols, s)
                             : abi.load_bf16(qp, kp, rows, cols, static_cast<ln_bf16*>(x.data_ptr()), cols, s);
    if (st != LN_OK) return failed(st);
    return THPVariable_Wrap(x);
    END_HANDLE_TH_ERRORS
}

// norm_bwd(dy, q, k, cols, gamma, mean, rstd) -> (dx, dgamma, dbeta); mean None: RMSNorm, dbeta None
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* dy = n == 7 ? tensor(a[0]) : nullptr;
    if (!dy || dy->dim() != 2 || !io_type(*dy) || !dy->is_contiguous() || !current(dy->device())) return none();
    const at::Device dev = dy->device();
    const int64_t rows = dy->size(0), cols = dy->size(1);
    const at::Tensor *q = tensor(a[1]), *k = tensor(a[2]), *gamma = tensor(a[4]), *rstd = tensor(a[6]);
    const bool rms = a[5] == Py_None, f32 = dy->scalar_type() == at::kFloat;
    const at::Tensor* mean = rms ? nullptr : tensor(a[5]);
    const int64_t kept = PyLong_Check(a[3]) ? PyLong_AsLongLong(a[3]) : -1;
    if (PyErr_Occurred()) PyErr_Clear();
    if (kept != cols || !is_ckpt(q, k, rows, cols, dev) || !is(gamma, {cols}, dy->scalar_type(), dev) ||
        (!rms && !is(mean, {rows}, at::kFloat, dev)) || !is(rstd, {rows}, at::kFloat, dev))
        return none();
    const size_t bytes = abi.norm_ws(rows, cols);
    at::Tensor dx = at::empty(dy->sizes(), dy->options()), dgamma = at::empty({cols}, dy->options()), dbeta;
    if (!rms) dbeta = at::empty({cols}, dy->options());
    at::Tensor ws = at::empty({(int64_t)bytes + 1}, dy->options().dtype(at::kByte));
    const int8_t* qp = static_cast<const int8_t*>(q->data_ptr());
    const uint8_t* kp = static_cast<const uint8_t*>(k->data_ptr());
    const float* mp = rms ? nullptr : static_cast<const float*>(mean->data_ptr());
    const float* rp = static_cast<const float*>(rstd->data_ptr());
    void* wp = ws.data_ptr();
    const ln_stream_t s = stream_of(dev);
    ln_status st;
    auto run = [&](auto* tag, auto norm, auto rnorm) {
        using T = std::remove_pointer_t<decltype(tag)>;
        const T *d = static_cast<const T*>(dy->data_ptr()), *g = static_cast<const T*>(gamma->data_ptr());
        T *x = static_cast<T*>(dx.data_ptr()), *dg = static_cast<T*>(dgamma.data_ptr());
        return rms ? rnorm(d, qp, kp, g, rp, x, dg, rows, cols, wp, bytes, s)
                   : norm(d, qp, kp, g, mp, rp, x, dg, static_cast<T*>(dbeta.data_ptr()), rows, cols, wp, bytes, s);
    };
    st = f32 ? run((float*)nullptr, abi.ln_f32, abi.rms_f32) : run((ln_bf16*)nullptr, abi.ln_bf16_, abi.rms_bf16);
    if (st != LN_OK) return failed(st);
    if (rms) return Py_BuildValue("(NNO)", THPVariable_Wrap(dx), THPVariable_Wrap(dgamma), Py_None);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(dx), THPVariable_Wrap(dgamma), THPVariable_Wrap(dbeta));
    END_HANDLE_TH_ERRORS
}

// init({name: address}): the C ABI's entry points
PyObject* init(PyObject*, PyObject* d) {
    if (!PyDict_Check(d)) {
        PyErr_SetString(PyExc_TypeError, "a dict of addresses is needed");
        return nullptr;
    }
    void* at[kCount];
    for (size_t i = 0; i < kCount; ++i) {
        PyObject* v = PyDict_GetItemString(d, kNames[i]);
        at[i] = v ? PyLong_AsVoidPtr(v) : nullptr;
        if (PyErr_Occurred()) return nullptr;
        if (!at[i]) {
            PyErr_SetString(PyExc_KeyError, kNames[i]);
            return nullptr;
        }
    }
    memcpy(&abi, at, sizeof(abi));
    Py_RETURN_NONE;
}

// edges(buckets, max_distance, bidirectional, (edge, ...))
PyObject* edges(PyObject*, PyObject* args) {
    long long buckets, span;
    int both;
    PyObject* list;
    if (!PyArg_ParseTuple(args, "LLpO!", &buckets, &span, &both, &PyTuple_Type, &list)) return nullptr;
    std::vector<int32_t> v;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(list); ++i) v.push_back((int32_t)PyLong_AsLong(PyTuple_GET_ITEM(list, i)));
    if (PyErr_Occurred()) return nullptr;
    edges_of.emplace(std::make_tuple((int64_t)buckets, (int64_t)span, both != 0), std::move(v));
    Py_RETURN_NONE;
}

#define LN_FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LN_FAST(rel_fwd), LN_FAST(rel_bwd), LN_FAST(store), LN_FAST(load), LN_FAST(norm_bwd),
                         {"init", init, METH_O, nullptr}, {"edges", edges, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
