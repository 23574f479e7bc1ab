// marshal.cpp -- argument marshalling of the attention-side entry points, as a
// Python extension.  These calls take up to ten tensors for a few microseconds
// of GPU work: reading their types, sizes, strides and addresses through Python
// took 10 to 14 microseconds a call, and takes 2 to 3 here.  The checks are
// those of swiglu_mlp_amd/__init__.py for the other calls (ValueError before
// anything is launched); the work is the C ABI's, whose functions bind() is
// given, so that there is one copy of the library in the process.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "ck.h"
#include "views.hpp"

namespace {

decltype(&ck_qk_norm_rope) g_norm = nullptr;
decltype(&ck_cross_attn) g_attn = nullptr;
decltype(&ck_cross_attn_workspace_size) g_attn_size = nullptr;
PyObject* g_stream = nullptr;   // device index -> its current stream's address

const at::Tensor& tensor_arg(PyObject* o, const char* what)
{
    TORCH_CHECK_VALUE(THPVariable_Check(o), what, " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// nullptr for None
const at::Tensor* optional_arg(PyObject* o, const char* what)
{
    return o == Py_None ? nullptr : &tensor_arg(o, what);
}

// The dtype code and device of a call, from its queries.
int dtype_code(const at::Tensor& q)
{
    TORCH_CHECK_VALUE(q.is_cuda(), "q must be on a GPU, got ", q.device());
    TORCH_CHECK_VALUE(q.scalar_type() == at::kBFloat16 || q.scalar_type() == at::kHalf,
                      "q needs dtype bfloat16 or float16, got ", q.scalar_type());
    return q.scalar_type() == at::kHalf ? CK_DTYPE_FP16 : CK_DTYPE_BF16;
}

// A [batch, tokens, heads, d] tensor of q's type and device.
ck_heads heads_of(const at::Tensor& t, const char* what, const at::Tensor& q)
{
    TORCH_CHECK_VALUE(t.device() == q.device() && t.scalar_type() == q.scalar_type() && t.dim() == 4, what, " needs a ",
                      q.scalar_type(), " [batch, tokens, heads, d] tensor on ", q.device(), ", got ", t.scalar_type(),
                      " ", t.sizes(), " on ", t.device());
    // the stride of a dimension of one element is never used
    const int64_t sb = t.size(0) > 1 ? t.stride(0) : 0, st = t.size(1) > 1 ? t.stride(1) : 0,
                  sh = t.size(2) > 1 ? t.stride(2) : 0;
    void* p = t.data_ptr();
    TORCH_CHECK_VALUE(t.stride(3) == 1 && t.size(3) >= 8 && t.size(3) % 8 == 0 && (uintptr_t)p % 16 == 0 &&
                          (sb | st | sh) % 8 == 0,
                      what, " needs contiguous heads of a multiple of 8 channels, 16-byte aligned (strides in multiples "
                      "of 8 elements), got shape ", t.sizes(), ", strides ", t.strides());
    return ck_heads{p, sb, st, sh};
}

ck::View view_of(const at::Tensor& t)
{
    TORCH_CHECK(t.dim() <= ck::View::kDims, "a view of ", t.dim(), " dimensions");
    return ck::View::of(t.data_ptr(), (int64_t)t.element_size(), t.sizes().data(), t.strides().data(), (int)t.dim());
}

// What a call reads, once for all the comparisons with its outputs.
struct Reads {
    ck::View views[10];
    int n = 0;
    void add(std::initializer_list<const at::Tensor*> tensors)   // null: not given
    {
        for (const at::Tensor* t : tensors)
            if (t) views[n++] = view_of(*t);
    }
    bool apart_from(const ck::View& v) const
    {
        for (int i = 0; i < n; ++i)
            if (!ck::disjoint(v, views[i])) return false;
        return true;
    }
};

// An output shaped like `like` (whose ck_heads are `in`): a new contiguous
// tensor, or `out` checked.  `out` shares no element with `like` and `reads`, or
// it is `like` itself where `in_place` allows that (each head is read before it
// is written).
at::Tensor output(const at::Tensor* out, const at::Tensor& like, const ck_heads& in, const char* what,
                  std::initializer_list<const Reads*> reads, bool in_place, ck_heads* h)
{
    if (!out) {
        at::Tensor t = at::empty(like.sizes(), like.options());
        const int64_t d = like.size(3), row = like.size(2) * d;
        *h = ck_heads{t.data_ptr(), like.size(1) * row, row, d};
        return t;
    }
    *h = heads_of(*out, what, like);
    TORCH_CHECK_VALUE(out->sizes() == like.sizes(), what, " needs shape ", like.sizes(), ", got ", out->sizes());
    for (int i = 0; i < 4; ++i)
        TORCH_CHECK_VALUE(out->size(i) < 2 || out->stride(i) != 0, what, " must not be an expanded tensor");
    const ck::View v = view_of(*out);
    TORCH_CHECK_VALUE(v.distinct(), what, " must not hold an element twice, got strides ", out->strides());
    const bool same = h->data == in.data && h->batch_stride == in.batch_stride &&
                      h->token_stride == in.token_stride && h->head_stride == in.head_stride;
    bool ok = (in_place && same) || ck::disjoint(v, view_of(like));
    for (const Reads* r : reads) ok = ok && r->apart_from(v);
    TORCH_CHECK_VALUE(ok, what, " must not share memory with what the call reads");
    return *out;
}

void* stream_of(const at::Tensor& q, bool* failed)
{
    PyObject* index = PyLong_FromLong(q.get_device());
    PyObject* s = index ? PyObject_CallOneArg(g_stream, index) : nullptr;
    Py_XDECREF(index);
    void* p = s ? PyLong_AsVoidPtr(s) : nullptr;
    Py_XDECREF(s);
    *failed = PyErr_Occurred() != nullptr;
    return p;
}

struct Rope {
    const float *cos = nullptr, *sin = nullptr;
    int64_t rows = 0, half = 0;
};

Rope rope_of(const at::Tensor* cos, const at::Tensor* sin, const char* what, const at::Tensor& q)
{
    if (!cos && !sin) return Rope{};
    TORCH_CHECK_VALUE(cos && sin, what, "_rope is (cos, sin)");
    for (const at::Tensor* t : {cos, sin})
        TORCH_CHECK_VALUE(t->scalar_type() == at::kFloat && t->dim() == 2 && t->device() == q.device() &&
                              t->is_contiguous() && t->sizes() == cos->sizes(),
                          what, "_rope needs contiguous float32 [rows, half] cos and sin of one shape on ", q.device());
    return Rope{(const float*)cos->data_ptr(), (const float*)sin->data_ptr(), cos->size(0), cos->size(1)};
}

// One side of a call, but for its output.
ck_qk_side side_of(const at::Tensor& x, const ck_heads& in, const at::Tensor* weight, const Rope& rope,
                   const at::Tensor* pos, const char* what, const at::Tensor& q)
{
    ck_qk_side s{};
    s.x = in;
    s.batch = x.size(0), s.tokens = x.size(1), s.heads = x.size(2);
    if (weight) {
        TORCH_CHECK_VALUE(weight->scalar_type() == at::kFloat && weight->dim() == 1 && weight->size(0) == x.size(3) &&
                              weight->device() == q.device() && weight->is_contiguous(),
                          what, "_weight needs a contiguous float32 (", x.size(3), ",) tensor on ", q.device());
        s.weight = (const float*)weight->data_ptr();
    }
    s.cos = rope.cos, s.sin = rope.sin, s.table_rows = rope.rows;
    if (pos) {
        TORCH_CHECK_VALUE(rope.cos, what, "_pos without ", what, "_rope");
        TORCH_CHECK_VALUE(pos->scalar_type() == at::kInt && pos->device() == q.device() && pos->dim() == 2 &&
                              pos->size(0) == s.batch && pos->size(1) == s.tokens &&
                              (s.tokens < 2 || pos->stride(1) == 1),
                          what, "_pos needs an int32 (", s.batch, ", ", s.tokens, ") tensor with contiguous rows on ",
                          q.device());
        s.pos = (const int32_t*)pos->data_ptr();
        s.pos_stride = s.batch > 1 ? pos->stride(0) : 0;
    } else {
        TORCH_CHECK_VALUE(!rope.cos || s.tokens <= rope.rows, what, "_rope has ", rope.rows, " rows for ", s.tokens,
                          " tokens");
    }
    return s;
}

// qk_norm_rope(q, k, q_weight, k_weight, q_cos, q_sin, k_cos, k_sin, q_pos, k_pos, pairing, eps, q_out, k_out)
// -> y, (y, z), or the C status of a refused call
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK(n == 14 && g_norm, "qk_norm_rope: 14 arguments, after bind()");
    const at::Tensor& q = tensor_arg(a[0], "q");
    const int dtype = dtype_code(q);
    const c10::DeviceGuard guard(q.device());   // the launch is on its current stream
    const at::Tensor* k = optional_arg(a[1], "k");
    const at::Tensor *qw = optional_arg(a[2], "q_weight"), *kw = optional_arg(a[3], "k_weight");
    const at::Tensor *qp = optional_arg(a[8], "q_pos"), *kp = optional_arg(a[9], "k_pos");
    const at::Tensor *qo = optional_arg(a[12], "q_out"), *ko = optional_arg(a[13], "k_out");
    const at::Tensor *qc = optional_arg(a[4], "q_rope"), *qs = optional_arg(a[5], "q_rope");
    const at::Tensor *kc = optional_arg(a[6], "k_rope"), *ks = optional_arg(a[7], "k_rope");
    const Rope qr = rope_of(qc, qs, "q", q), kr = rope_of(kc, ks, "k", q);
    const int pairing = (int)PyLong_AsLong(a[10]);
    const float eps = (float)PyFloat_AsDouble(a[11]);
    if (PyErr_Occurred()) return nullptr;

    const ck_heads hq = heads_of(q, "q", q);
    const int64_t d = q.size(3), step = pairing == CK_PAIR_HALF ? 16 : 8;
    TORCH_CHECK_VALUE(d <= 256, "head size ", d, " is over 256");
    TORCH_CHECK_VALUE(!qr.cos || !kr.cos || qr.half == kr.half, "q_rope and k_rope turn different numbers of channels");
    const int64_t rot = 2 * (qr.cos ? qr.half : kr.half);
    TORCH_CHECK_VALUE(rot <= d && rot % step == 0, "the rotated channels must be a multiple of ", step, " up to ", d,
                      ", got ", rot);
    TORCH_CHECK_VALUE(k || (!kw && !kr.cos && !kp && !ko), "arguments for k without k");
    bool failed;
    void* stream = stream_of(q, &failed);
    if (failed) return nullptr;

    ck_qk_side sq = side_of(q, hq, qw, qr, qp, "q", q), sk{};
    if (k) {
        const ck_heads hk = heads_of(*k, "k", q);
        TORCH_CHECK_VALUE(k->size(3) == d, "q and k need one head size, got ", d, " and ", k->size(3));
        sk = side_of(*k, hk, kw, kr, kp, "k", q);
    }
    Reads small, own_q, own_k;
    if (qo || ko) {
        small.add({qw, qc, qs, qp, kw});
        if (kc != qc) small.add({kc});
        if (ks != qs) small.add({ks});
        if (kp != qp) small.add({kp});
        own_q.add({&q});
        own_k.add({k});
    }
    const at::Tensor y = output(qo, q, hq, "q_out", {&small, &own_k}, true, &sq.y);
    at::Tensor z;
    if (k) {
        z = output(ko, *k, sk.x, "k_out", {&small, &own_q}, true, &sk.y);
        TORCH_CHECK_VALUE(!qo || !ko || ck::disjoint(view_of(y), view_of(z)), "q_out and k_out must not share memory");
    }
    ck_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_norm(&sq, k ? &sk : nullptr, d, rot, pairing, dtype, eps, stream);
    Py_END_ALLOW_THREADS
    if (st != CK_OK) return PyLong_FromLong(st);
    if (!k) return THPVariable_Wrap(y);
    PyObject *py = THPVariable_Wrap(y), *pz = THPVariable_Wrap(z);
    PyObject* r = py && pz ? PyTuple_Pack(2, py, pz) : nullptr;
    Py_XDECREF(py);
    Py_XDECREF(pz);
    return r;
    END_HANDLE_TH_ERRORS
}

// cross_attn(q, k, v, scale, kv_len, key_mask, out, workspace) -> y, or the C status of a refused call
PyObject* cross_attn(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK(n == 8 && g_attn, "cross_attn: 8 arguments, after bind()");
    const at::Tensor& q = tensor_arg(a[0], "q");
    const int dtype = dtype_code(q);
    const c10::DeviceGuard guard(q.device());   // the launch is on its current stream
    const at::Tensor &k = tensor_arg(a[1], "k"), &v = tensor_arg(a[2], "v");
    const at::Tensor *len = optional_arg(a[4], "kv_len"), *mask = optional_arg(a[5], "key_mask");
    const at::Tensor *out = optional_arg(a[6], "out"), *ws = optional_arg(a[7], "workspace");
    const ck_heads hq = heads_of(q, "q", q), hk = heads_of(k, "k", q), hv = heads_of(v, "v", q);
    const int64_t b = q.size(0), tq = q.size(1), h = q.size(2), d = q.size(3);
    const int64_t kb = k.size(0), tk = k.size(1), kh = k.size(2);
    TORCH_CHECK_VALUE(v.sizes() == k.sizes(), "k and v need one shape, got ", k.sizes(), " and ", v.sizes());
    TORCH_CHECK_VALUE(k.size(3) == d && d <= 128, "q and k need one head size up to 128, got ", d, " and ", k.size(3));
    TORCH_CHECK_VALUE(!b || !tq || !h || (kb && b % kb == 0 && kh && h % kh == 0), "batch ", b, " and heads ", h,
                      " must be multiples of the encoder's ", kb, " and ", kh);
    const double scale = a[3] == Py_None ? 1.0 / std::sqrt((double)d) : PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) return nullptr;
    TORCH_CHECK_VALUE(scale > 0.0 && scale < 3.4e38, "scale must be positive and finite, got ", scale);
    TORCH_CHECK_VALUE(!len || (len->scalar_type() == at::kInt && len->dim() == 1 && len->size(0) == kb &&
                               len->device() == q.device() && len->is_contiguous()),
                      "kv_len needs a contiguous int32 (", kb, ",) tensor on ", q.device());
    TORCH_CHECK_VALUE(!mask || ((mask->scalar_type() == at::kBool || mask->scalar_type() == at::kByte) &&
                                mask->dim() == 2 && mask->size(0) == kb && mask->size(1) == tk &&
                                mask->device() == q.device() && (tk < 2 || mask->stride(1) == 1)),
                      "key_mask needs a bool or uint8 (", kb, ", ", tk, ") tensor with contiguous rows on ", q.device());
    bool failed;
    void* stream = stream_of(q, &failed);
    if (failed) return nullptr;

    const size_t need = g_attn_size(b, kb, tq, tk, h, kh, d);
    if (!need) ws = nullptr;
    TORCH_CHECK_VALUE(!ws || (ws->scalar_type() == at::kByte && ws->dim() == 1 && ws->is_contiguous() &&
                              ws->device() == q.device() && (size_t)ws->numel() >= need),
                      "workspace needs a contiguous uint8 tensor of ", need, " bytes on ", q.device());
    ck_heads hy;
    Reads reads;
    if (out || ws) reads.add({&k, &v, len, mask});
    const at::Tensor y = output(out, q, hq, "out", {&reads}, false, &hy);
    if (ws) {
        reads.add({&q, &y});
        TORCH_CHECK_VALUE(reads.apart_from(view_of(*ws)), "workspace must not share memory with the call's tensors");
    }
    at::Tensor room;
    if (need) room = ws ? *ws : at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    ck_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_attn(&hq, &hk, &hv, &hy, b, kb, tq, tk, h, kh, d, dtype, (float)scale,
                len ? (const int32_t*)len->data_ptr() : nullptr, mask ? (const uint8_t*)mask->data_ptr() : nullptr,
                mask && kb > 1 ? mask->stride(0) : 0, need ? room.data_ptr() : nullptr, need ? (size_t)room.numel() : 0,
                stream);
    Py_END_ALLOW_THREADS
    if (st != CK_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// bind(ck_qk_norm_rope, ck_cross_attn, ck_cross_attn_workspace_size, stream): the C functions' addresses and the
// callable that gives a device's current stream
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind: 4 arguments");
        return nullptr;
    }
    void* f[3];
    for (int i = 0; i < 3; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null function");
            return nullptr;
        }
    }
    g_norm = reinterpret_cast<decltype(g_norm)>(f[0]);
    g_attn = reinterpret_cast<decltype(g_attn)>(f[1]);
    g_attn_size = reinterpret_cast<decltype(g_attn_size)>(f[2]);
    Py_INCREF(a[3]);
    Py_XSETREF(g_stream, a[3]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"cross_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cross_attn)), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
