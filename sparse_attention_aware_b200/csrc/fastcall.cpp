// The binding's short way for the calls of a serving step.
//
// A decode step's kernels take 3 to 12 us; checking a call's tensors, making
// its outputs and filling its argument struct in Python takes as long again or
// longer (14 to 20 us).  These functions do the same for calls whose tensors
// are laid out as the library reads them, on the current device, with outputs
// made here: they return the outputs, or the library's status as a number, or
// None for any other call, which the Python code then checks, copies, places or
// refuses as documented.  Calls that are being captured into a graph are left to
// it too: it keeps the memory whose address the graph holds.  Nothing is kept
// between calls.
//
// Built as _fastcall.so against torch; the library's functions are handed over
// by address (init), so libsa is loaded in one place only.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sa.h"

namespace {

decltype(&sa_plan_append) f_plan;
decltype(&sa_rope_append) f_append;
decltype(&sa_rope_append_kv4) f_append4;
decltype(&sa_expand_kv4) f_expand;
decltype(&sa_sparse_decode_attn_kv4) f_decode;
decltype(&sa_kv4_decode_workspace_bytes) f_decode_bytes;

using at::ScalarType;

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool is(const at::Tensor *t, ScalarType type, at::IntArrayRef shape, int dev)
{
    return t && t->scalar_type() == type && t->sizes() == shape && t->is_cuda() && t->get_device() == dev &&
           t->is_contiguous();
}

void *ptr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

at::Tensor make(at::IntArrayRef shape, ScalarType type, int dev)
{
    return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
}

// the device of a call: that of its first tensor if it is the current one, else -1
int device_of(const at::Tensor *t)
{
    if (!t || !t->is_cuda()) return -1;
    const int dev = t->get_device();
    return dev == c10::cuda::current_device() ? dev : -1;
}

PyObject *none() { Py_RETURN_NONE; }

// Python's other threads run while one lives: an allocation or a launch may wait,
// for instance for room in the stream's queue
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// a number of 32 bits; others are left to the Python code's refusals
bool number(PyObject *o, int32_t *x)
{
    const long long v = PyLong_AsLongLong(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    *x = (int32_t)v;
    return v == *x;
}

// whether the stream (its handle as a Python number) is being captured, or cannot say
bool captured(PyObject *stream)
{
    cudaStreamCaptureStatus now = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(static_cast<cudaStream_t>(PyLong_AsVoidPtr(stream)), &now) != cudaSuccess) {
        cudaGetLastError();
        return true;
    }
    return now != cudaStreamCaptureStatusNone;
}

// A 4-bit cache
bool cache4(const at::Tensor *kv, const at::Tensor *pt, const at::Tensor *sl, int dev, sa_kv4_cache *c)
{
    if (!kv || !pt || !sl || kv->dim() != 4 || pt->dim() != 2) return false;
    const auto s = kv->sizes();
    if (s[3] <= 16 || !is(kv, at::kByte, s, dev) || !is(pt, at::kInt, pt->sizes(), dev) ||
        !is(sl, at::kInt, {pt->size(0)}, dev))
        return false;
    *c = {kv->data_ptr(), static_cast<const int32_t *>(pt->data_ptr()), static_cast<const int32_t *>(sl->data_ptr()),
          (int32_t)pt->size(0), (int32_t)s[1], (int32_t)s[3] - 16, (int32_t)s[2], (int32_t)pt->size(1), (int32_t)s[0]};
    return s[0] <= INT32_MAX && pt->size(1) <= INT32_MAX;
}

// plan(page_table, seq_lens, new_lens, free_pages, free_count, num_pages, page_size, max_tokens, seq_lens_out,
//      free_count_out, ws, ws_bytes, stream)
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 13 || captured(a[12])) return none();
    const at::Tensor *pt = tensor(a[0]), *sl = tensor(a[1]), *add = tensor(a[2]), *fp = tensor(a[3]), *fc = tensor(a[4]);
    const at::Tensor *slo = a[8] == Py_None ? sl : tensor(a[8]), *fco = a[9] == Py_None ? fc : tensor(a[9]);
    const int dev = device_of(pt);
    if (dev < 0 || pt->dim() != 2 || !fp || fp->dim() != 1) return none();
    const int64_t B = pt->size(0);
    sa_plan_args p{};
    if (!number(a[5], &p.num_pages) || !number(a[6], &p.page_size) || !number(a[7], &p.max_tokens)) return none();
    const int64_t tokens = p.max_tokens;
    if (!is(pt, at::kInt, pt->sizes(), dev) || !is(sl, at::kInt, {B}, dev) || !is(add, at::kInt, {B}, dev) ||
        !is(fp, at::kInt, fp->sizes(), dev) || !is(fc, at::kInt, {1}, dev) || !is(slo, at::kInt, {B}, dev) ||
        !is(fco, at::kInt, {1}, dev) || tokens < 0 || B > INT32_MAX || pt->size(1) > INT32_MAX ||
        fp->numel() > INT32_MAX)
        return none();
    at::Tensor cu, pos, slots, seq;
    p.page_table = static_cast<int32_t *>(ptr(pt));
    p.seq_lens = static_cast<int32_t *>(ptr(sl));
    p.new_lens = static_cast<int32_t *>(ptr(add));
    p.free_pages = static_cast<int32_t *>(ptr(fp));
    p.free_count = static_cast<int32_t *>(ptr(fc));
    p.seq_lens_out = static_cast<int32_t *>(ptr(slo));
    p.free_count_out = static_cast<int32_t *>(ptr(fco));
    p.batch = (int32_t)B;
    p.max_pages_per_seq = (int32_t)pt->size(1);
    p.num_free = (int32_t)fp->numel();
    void *ws = PyLong_AsVoidPtr(a[10]);
    const size_t wn = PyLong_AsSize_t(a[11]);
    const auto stream = static_cast<sa_stream_t>(PyLong_AsVoidPtr(a[12]));
    if (PyErr_Occurred()) return nullptr;
    sa_status st;
    {
        Unlocked threads;
        cu = make({B + 1}, at::kInt, dev), pos = make({tokens}, at::kInt, dev);
        slots = make({tokens}, at::kLong, dev), seq = make({tokens}, at::kInt, dev);
        p.cu_tokens = static_cast<int32_t *>(cu.data_ptr());
        p.positions = static_cast<int32_t *>(pos.data_ptr());
        p.slots = static_cast<int64_t *>(slots.data_ptr());
        p.seq_ids = static_cast<int32_t *>(seq.data_ptr());
        st = f_plan(&p, ws, wn, stream);
    }
    if (st != SA_OK) return PyLong_FromLong(st);
    return Py_BuildValue("NNNN", THPVariable_Wrap(cu), THPVariable_Wrap(pos), THPVariable_Wrap(slots),
                         THPVariable_Wrap(seq));
}

// bf16 [T][H][D] with contiguous heads; the elements between its tokens
bool rows(const at::Tensor *x, int64_t T, int64_t H, int64_t D, int dev, int64_t *stride)
{
    if (!x || x->scalar_type() != at::kBFloat16 || !x->is_cuda() || x->get_device() != dev ||
        x->sizes() != at::IntArrayRef({T, H, D}))
        return false;
    const auto s = x->strides();
    *stride = T > 1 ? s[0] : H * D;
    return s[2] == 1 && (H == 1 || s[1] == D) && *stride % 8 == 0 && (uintptr_t)x->data_ptr() % 16 == 0;
}

// append(k or kv, v or None, page_table, seq_lens, q, k, v, positions, slots, inv_freq, q_weight, k_weight, eps,
//        interleaved, ws, ws_bytes, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 17 || captured(a[16])) return none();
    const at::Tensor *pool = tensor(a[0]), *vpool = tensor(a[1]), *pt = tensor(a[2]), *sl = tensor(a[3]);
    const at::Tensor *q = tensor(a[4]), *k = tensor(a[5]), *v = tensor(a[6]), *pos = tensor(a[7]), *slots = tensor(a[8]);
    const at::Tensor *inv = tensor(a[9]), *qw = tensor(a[10]), *kw = tensor(a[11]);
    const int dev = device_of(q);
    if (dev < 0 || q->dim() != 3 || !pool || pool->dim() != 4 || !pt || pt->dim() != 2) return none();
    sa_kv4_cache c4{};
    sa_kv_cache c16{};
    const bool four = a[1] == Py_None;
    const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), Hkv = pool->size(1);
    if (T > INT32_MAX || Hq > INT32_MAX) return none();
    if (four) {
        if (!cache4(pool, pt, sl, dev, &c4) || c4.head_dim != D) return none();
    } else {
        const auto s = pool->sizes();
        if (s[3] != D || !is(pool, at::kBFloat16, s, dev) || !is(vpool, at::kBFloat16, s, dev) ||
            !is(pt, at::kInt, pt->sizes(), dev) || !is(sl, at::kInt, {pt->size(0)}, dev) || s[0] > INT32_MAX)
            return none();
        c16 = {pool->data_ptr(), vpool->data_ptr(), static_cast<const int32_t *>(pt->data_ptr()),
               static_cast<const int32_t *>(sl->data_ptr()), (int32_t)pt->size(0), (int32_t)s[1], (int32_t)D,
               (int32_t)s[2], (int32_t)pt->size(1), (int32_t)s[0]};
    }
    sa_append_args p{};
    if (!rows(q, T, Hq, D, dev, &p.q_stride) || !rows(k, T, Hkv, D, dev, &p.k_stride) ||
        !rows(v, T, Hkv, D, dev, &p.v_stride) || !is(pos, at::kInt, {T}, dev) || !is(slots, at::kLong, {T}, dev))
        return none();
    if (inv ? !is(inv, at::kFloat, {inv->numel()}, dev) : a[9] != Py_None) return none();
    const ScalarType wt = qw ? qw->scalar_type() : kw ? kw->scalar_type() : at::kBFloat16;
    if (wt != at::kBFloat16 && wt != at::kFloat) return none();
    if (qw ? !is(qw, wt, {D}, dev) : a[10] != Py_None) return none();
    if (kw ? !is(kw, wt, {D}, dev) : a[11] != Py_None) return none();
    at::Tensor out;
    p.q = ptr(q);
    p.k = ptr(k);
    p.v = ptr(v);
    p.q_out_stride = Hq * D;
    p.positions = static_cast<const int32_t *>(ptr(pos));
    p.slots = static_cast<const int64_t *>(ptr(slots));
    p.inv_freq = inv && inv->numel() ? static_cast<const float *>(ptr(inv)) : nullptr;
    p.q_weight = ptr(qw);
    p.k_weight = ptr(kw);
    p.weight_dtype = wt == at::kFloat ? SA_DTYPE_F32 : SA_DTYPE_BF16;
    p.eps = (float)PyFloat_AsDouble(a[12]);
    p.num_tokens = (int32_t)T;
    p.num_q_heads = (int32_t)Hq;
    p.rot_dim = inv ? (int32_t)(2 * inv->numel()) : 0;
    p.interleaved = PyObject_IsTrue(a[13]);
    void *ws = PyLong_AsVoidPtr(a[14]);
    const size_t wn = PyLong_AsSize_t(a[15]);
    sa_stream_t st = static_cast<sa_stream_t>(PyLong_AsVoidPtr(a[16]));
    if (PyErr_Occurred()) return nullptr;
    sa_status r;
    {
        Unlocked threads;
        out = make({T, Hq, D}, at::kBFloat16, dev);
        p.q_out = out.data_ptr();
        r = four ? f_append4(&c4, &p, ws, wn, st) : f_append(&c16, &p, ws, wn, st);
    }
    return r == SA_OK ? THPVariable_Wrap(out) : PyLong_FromLong(r);
}

// expand(kv, page_table, seq_lens, pages, ws, ws_bytes, stream)
PyObject *expand(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 7 || captured(a[6])) return none();
    const at::Tensor *kv = tensor(a[0]), *pages = tensor(a[3]);
    const int dev = device_of(kv);
    sa_kv4_cache c{};
    if (dev < 0 || !cache4(kv, tensor(a[1]), tensor(a[2]), dev, &c)) return none();
    if (!pages || !is(pages, at::kInt, {pages->numel()}, dev)) return none();
    const int64_t m = pages->numel();
    const int32_t *list = static_cast<const int32_t *>(ptr(pages));
    void *ws = PyLong_AsVoidPtr(a[4]);
    const size_t wn = PyLong_AsSize_t(a[5]);
    const auto stream = static_cast<sa_stream_t>(PyLong_AsVoidPtr(a[6]));
    if (PyErr_Occurred()) return nullptr;
    at::Tensor k, v;
    sa_status st;
    {
        Unlocked threads;
        k = make({m, c.num_kv_heads, c.page_size, c.head_dim}, at::kBFloat16, dev);
        v = make({m, c.num_kv_heads, c.page_size, c.head_dim}, at::kBFloat16, dev);
        st = f_expand(&c, list, (int32_t)m, k.data_ptr(), v.data_ptr(), ws, wn, stream);
    }
    if (st != SA_OK) return PyLong_FromLong(st);
    return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
}

// decode(kv, page_table, seq_lens, q, idx or blocks, counts, kind, scale, num_splits, want_lse, ws, ws_bytes, stream)
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 13 || captured(a[12])) return none();
    const at::Tensor *q = tensor(a[3]), *list = tensor(a[4]), *count = tensor(a[5]);
    const int dev = device_of(q);
    sa_kv4_cache c{};
    if (dev < 0 || q->dim() != 3 || !cache4(tensor(a[0]), tensor(a[1]), tensor(a[2]), dev, &c)) return none();
    const int64_t B = q->size(0), H = q->size(1), D = q->size(2);
    const bool f32 = q->scalar_type() == at::kFloat;
    if ((!f32 && q->scalar_type() != at::kBFloat16) || !q->is_contiguous() || B != c.batch || D != c.head_dim ||
        H > INT32_MAX || !list || list->dim() != 3)
        return none();
    sa_selection s{};
    s.kind = (sa_selection_kind)PyLong_AsLong(a[6]);
    const int64_t most = list->size(s.kind == SA_SEL_TOKENS ? 2 : 1);
    if (most > INT32_MAX) return none();
    if (s.kind == SA_SEL_TOKENS) {
        if (!is(list, at::kInt, {B, H, most}, dev) || !is(count, at::kInt, {B, H}, dev)) return none();
        s.idx = static_cast<const int32_t *>(ptr(list));
        s.count = static_cast<const int32_t *>(ptr(count));
        s.k_cap = (int32_t)most;
    } else {
        if (!is(list, at::kInt, {B, most, 4}, dev) || !is(count, at::kInt, {B}, dev)) return none();
        s.blocks = static_cast<const int32_t *>(ptr(list));
        s.block_counts = static_cast<const int32_t *>(ptr(count));
        s.max_blocks = (int32_t)most;
    }
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AsDouble(a[7]);
    int32_t splits = 0;
    if (!number(a[8], &splits)) return none();
    const int lse_too = PyObject_IsTrue(a[9]);
    void *ws = PyLong_AsVoidPtr(a[10]);
    const size_t have = PyLong_AsSize_t(a[11]);
    const auto stream = static_cast<sa_stream_t>(PyLong_AsVoidPtr(a[12]));
    if (PyErr_Occurred()) return nullptr;
    if (splits < 0 || splits > 64) return none();
    const size_t need = f_decode_bytes(&c, (int32_t)H, splits);
    if (need == 0 || need > have) return none();
    const void *queries = ptr(q);
    at::Tensor out, lse;
    sa_status st;
    {
        Unlocked threads;
        out = make({B, H, D}, at::kBFloat16, dev);
        if (lse_too) lse = make({B, H}, at::kFloat, dev);
        st = f_decode(&c, queries, f32 ? SA_DTYPE_F32 : SA_DTYPE_BF16, (int32_t)H, &s, (float)scale, splits,
                      out.data_ptr(), lse_too ? static_cast<float *>(lse.data_ptr()) : nullptr, ws, have, stream);
    }
    if (st != SA_OK) return PyLong_FromLong(st);
    if (!lse_too) Py_INCREF(Py_None);
    return Py_BuildValue("NN", THPVariable_Wrap(out), lse_too ? THPVariable_Wrap(lse) : Py_None);
}

// no C++ exception leaves a call (an allocation that fails comes again, as
// torch's own error, from the long way)
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    try {
        return F(self, a, n);
    } catch (const std::exception &) {
        PyErr_Clear();
        return none();
    }
}

// init(addresses of sa_plan_append, sa_rope_append, sa_rope_append_kv4, sa_expand_kv4,
//      sa_sparse_decode_attn_kv4, sa_kv4_decode_workspace_bytes)
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "six addresses");
        return nullptr;
    }
    f_plan = reinterpret_cast<decltype(f_plan)>(PyLong_AsVoidPtr(a[0]));
    f_append = reinterpret_cast<decltype(f_append)>(PyLong_AsVoidPtr(a[1]));
    f_append4 = reinterpret_cast<decltype(f_append4)>(PyLong_AsVoidPtr(a[2]));
    f_expand = reinterpret_cast<decltype(f_expand)>(PyLong_AsVoidPtr(a[3]));
    f_decode = reinterpret_cast<decltype(f_decode)>(PyLong_AsVoidPtr(a[4]));
    f_decode_bytes = reinterpret_cast<decltype(f_decode_bytes)>(PyLong_AsVoidPtr(a[5]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"init", FAST(init), nullptr},
                         {"plan", FAST(guarded<plan>), nullptr},
                         {"append", FAST(guarded<append>), nullptr},
                         {"expand", FAST(guarded<expand>), nullptr},
                         {"decode", FAST(guarded<decode>), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall()
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "made_for", SA_MADE_FOR) < 0) Py_CLEAR(m);
    return m;
}
