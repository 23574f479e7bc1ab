// marshal.cpp -- argument marshalling of the attention-side entry points, the MX
// FP4 linears and ck_block_norm, as a Python extension.  These calls take up to ten tensors for a few microseconds
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
decltype(&ck_mx4_weight_prep) g_mx4_prep = nullptr;
decltype(&ck_mx4_act_quant) g_mx4_quant = nullptr;
decltype(&ck_mx4_dequant) g_mx4_dequant = nullptr;
decltype(&ck_mx4_gemm_bf16) g_mx4_gemm = nullptr;
decltype(&ck_mx4_linear) g_mx4_linear = nullptr;
decltype(&ck_mx4_linear_workspace_size) g_mx4_linear_size = nullptr;
decltype(&ck_block_norm) g_block_norm = nullptr;
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

// ---- MX FP4 linears ----

int64_t pad(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// An activation or a weight [rows, columns] whose rows are contiguous; -> its row stride.
int64_t rows_of(const at::Tensor& x, at::ScalarType type, const char* what)
{
    TORCH_CHECK_VALUE(x.is_cuda(), what, " must be on a GPU, got ", x.device());
    TORCH_CHECK_VALUE(x.scalar_type() == type && x.dim() == 2, what, " needs a 2D ", type, " tensor, got ",
                      x.scalar_type(), " ", x.sizes());
    const int64_t ld = x.size(0) > 1 ? x.stride(0) : x.size(1);
    TORCH_CHECK_VALUE((x.size(1) < 2 || x.stride(1) == 1) && ld >= x.size(1) && ld % 8 == 0 &&
                          (uintptr_t)x.data_ptr() % 16 == 0,
                      what, " needs contiguous, 16-byte aligned rows, got shape ", x.sizes(), ", strides ", x.strides());
    return ld;
}

void check_group(int64_t k, int64_t group)
{
    TORCH_CHECK_VALUE(group >= 1 && group <= 256 && (group & (group - 1)) == 0,
                      "the rotation group must be a power of two up to 256, got ", group);
    TORCH_CHECK_VALUE(k >= 64 && k % 64 == 0 && k <= CK_MAX_K, "in_features must be a multiple of 64 up to ", CK_MAX_K,
                      ", got ", k);
    TORCH_CHECK_VALUE(k % group == 0, "in_features (", k, ") must be divisible by group_size ", group);
}

bool is_bytes(const at::Tensor& t, int64_t dims, c10::Device dev)
{
    return t.scalar_type() == at::kByte && t.dim() == dims && t.is_contiguous() && t.device() == dev;
}

// Codes and scales in the blocked layout: [rp / 32, kp / 64, 1024] and [rp / 32, kp / 256, 256] bytes.
void check_blocked(const at::Tensor& codes, const at::Tensor& scales, const char* what, c10::Device dev)
{
    TORCH_CHECK_VALUE(is_bytes(codes, 3, dev) && is_bytes(scales, 3, dev) && codes.size(2) == 1024 &&
                          scales.size(2) == 256 && codes.size(1) % 4 == 0 && scales.size(1) * 4 == codes.size(1) &&
                          scales.size(0) == codes.size(0),
                      what, " needs contiguous uint8 codes (rows / 32, k / 64, 1024) and scales (rows / 32, k / 256, 256) "
                      "on ", dev, ", got ", codes.sizes(), " and ", scales.sizes());
}

// out_features of a blocked weight: `n`, or all its rows.
int64_t features_of(PyObject* n, const at::Tensor& codes)
{
    const int64_t rows = codes.size(0) * 32;
    if (n == Py_None) return rows;
    const int64_t v = PyLong_AsLongLong(n);
    if (PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(v >= 0 && v % 16 == 0 && pad(v, 32) == rows, "n must be a multiple of 16 that the weight's ", rows,
                      " rows hold, got ", v);
    return v;
}

// The BF16 [m, n] output: new, or `out` checked; it may be the residual itself.
at::Tensor linear_out(const at::Tensor* out, int64_t m, int64_t n, const at::TensorOptions& like, const Reads& reads,
                      const at::Tensor* bias, const at::Tensor* residual)
{
    const c10::Device dev = like.device();
    TORCH_CHECK_VALUE(!bias || (bias->scalar_type() == at::kFloat && bias->dim() == 1 && bias->size(0) == n &&
                                bias->is_contiguous() && bias->device() == dev),
                      "bias needs a contiguous (", n, ",) float32 tensor on ", dev);
    for (const at::Tensor* t : {residual, out}) {
        if (!t) continue;
        TORCH_CHECK_VALUE(t->scalar_type() == at::kBFloat16 && t->dim() == 2 && t->size(0) == m && t->size(1) == n &&
                              t->is_contiguous() && t->device() == dev,
                          t == out ? "out" : "residual", " needs a contiguous (", m, ", ", n, ") bfloat16 tensor on ", dev);
    }
    if (!out) return at::empty({m, n}, like.dtype(at::kBFloat16));
    TORCH_CHECK_VALUE(reads.apart_from(view_of(*out)), "out must not share memory with what the call reads");
    TORCH_CHECK_VALUE(!residual || residual->data_ptr() == out->data_ptr() ||
                          ck::disjoint(view_of(*out), view_of(*residual)),
                      "residual must be out itself or not overlap it");
    return *out;
}

// A workspace of `need` bytes: new, or `ws` checked against `reads` and the output.
at::Tensor room_of(const at::Tensor* ws, size_t need, const at::TensorOptions& like, const Reads& reads,
                   const at::Tensor& y)
{
    if (!need) return at::Tensor();
    if (!ws) return at::empty({(int64_t)need}, like.dtype(at::kByte));
    TORCH_CHECK_VALUE(is_bytes(*ws, 1, like.device()) && (size_t)ws->numel() >= need && (uintptr_t)ws->data_ptr() % 256 == 0,
                      "workspace needs a contiguous, 256-byte aligned uint8 tensor of ", need, " bytes on ", like.device());
    const ck::View v = view_of(*ws);
    TORCH_CHECK_VALUE(reads.apart_from(v) && ck::disjoint(v, view_of(y)),
                      "workspace must not share memory with the call's tensors");
    return *ws;
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes(const at::Tensor& t) { return t.defined() ? (size_t)t.numel() : 0; }
template <typename T>
T* ptr_or_null(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

PyObject* pair(const at::Tensor& a, const at::Tensor& b)
{
    PyObject *pa = THPVariable_Wrap(a), *pb = THPVariable_Wrap(b);
    PyObject* r = pa && pb ? PyTuple_Pack(2, pa, pb) : nullptr;
    Py_XDECREF(pa);
    Py_XDECREF(pb);
    return r;
}

// mx4_quant(x, act, group, k, layout, weight) -> (codes, scales), or the C status of a refused call.  weight: x is an
// FP32 weight (contiguous), else a BF16 activation; k None: all of x's columns (half of them with SwiGLU).
PyObject* mx4_quant(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK(n == 6 && g_mx4_quant, "mx4_quant: 6 arguments, after bind()");
    const bool weight = a[5] == Py_True;
    const char* what = weight ? "weight" : "activation";
    const at::Tensor& x = tensor_arg(a[0], what);
    const int act = (int)PyLong_AsLong(a[1]), layout = (int)PyLong_AsLong(a[4]);
    const int64_t group = PyLong_AsLongLong(a[2]);
    if (PyErr_Occurred()) return nullptr;
    const int64_t ld = rows_of(x, weight ? at::kFloat : at::kBFloat16, what);
    const c10::DeviceGuard guard(x.device());
    const int64_t rows = x.size(0), parts = act == CK_ACT_SWIGLU ? 2 : 1;
    const int64_t k = a[3] == Py_None ? x.size(1) / parts : PyLong_AsLongLong(a[3]);
    if (PyErr_Occurred()) return nullptr;
    check_group(k, group);
    TORCH_CHECK_VALUE(x.size(1) >= parts * k && (!weight || ld == k), what, " needs ", parts * k,
                      " contiguous columns for in_features ", k, ", got ", x.size(1));
    TORCH_CHECK_VALUE(layout == CK_LAYOUT_ROWS || layout == CK_LAYOUT_BLOCKED, "4-bit codes use the rows or blocked layout");
    bool failed;
    void* stream = stream_of(x, &failed);
    if (failed) return nullptr;
    const bool blocked = layout == CK_LAYOUT_BLOCKED;
    const at::TensorOptions u8 = x.options().dtype(at::kByte);
    const int64_t rb = pad(rows, 32) / 32, kp = pad(k, 256);
    const at::Tensor codes = blocked ? at::empty({rb, kp / 64, 1024}, u8) : at::empty({rows, k / 2}, u8);
    const at::Tensor scales = blocked ? at::empty({rb, kp / 256, 256}, u8) : at::empty({rows, k / 32}, u8);
    auto *pc = (uint8_t*)codes.data_ptr(), *ps = (uint8_t*)scales.data_ptr();
    ck_status st;
    Py_BEGIN_ALLOW_THREADS
    st = weight ? g_mx4_prep((const float*)x.data_ptr(), rows, k, (int32_t)group, layout, pc, ps, stream)
                : g_mx4_quant((const uint16_t*)x.data_ptr(), ld, rows, k, act, (int32_t)group, layout, pc, ps, stream);
    Py_END_ALLOW_THREADS
    if (st != CK_OK) return PyLong_FromLong(st);
    return pair(codes, scales);
    END_HANDLE_TH_ERRORS
}

// mx4_dequant(codes, scales, rows, k) -> BF16 [rows, k], or the C status of a refused call.  rows and k None: all that
// the codes hold.
PyObject* mx4_dequant(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK(n == 4 && g_mx4_dequant, "mx4_dequant: 4 arguments, after bind()");
    const at::Tensor &codes = tensor_arg(a[0], "codes"), &scales = tensor_arg(a[1], "scales");
    TORCH_CHECK_VALUE(codes.is_cuda(), "codes must be on a GPU, got ", codes.device());
    const c10::DeviceGuard guard(codes.device());
    const bool blocked = codes.dim() == 3;
    if (blocked)
        check_blocked(codes, scales, "dequantization", codes.device());
    else
        TORCH_CHECK_VALUE(is_bytes(codes, 2, codes.device()) && is_bytes(scales, 2, codes.device()) &&
                              codes.size(0) == scales.size(0) && codes.size(1) == scales.size(1) * 16,
                          "dequantization needs contiguous uint8 codes (rows, k / 2) and scales (rows, k / 32), got ",
                          codes.sizes(), " and ", scales.sizes());
    const int64_t all_rows = blocked ? codes.size(0) * 32 : codes.size(0);
    const int64_t all_k = blocked ? codes.size(1) * 64 : codes.size(1) * 2;
    const int64_t rows = a[2] == Py_None ? all_rows : PyLong_AsLongLong(a[2]);
    const int64_t k = a[3] == Py_None ? all_k : PyLong_AsLongLong(a[3]);
    if (PyErr_Occurred()) return nullptr;
    check_group(k, 1);
    TORCH_CHECK_VALUE(blocked ? rows >= 0 && pad(rows, 32) == all_rows && pad(k, 256) == all_k
                              : rows == all_rows && k == all_k,
                      "the codes do not hold ", rows, " x ", k, " values: ", codes.sizes());
    bool failed;
    void* stream = stream_of(codes, &failed);
    if (failed) return nullptr;
    const at::Tensor y = at::empty({rows, k}, codes.options().dtype(at::kBFloat16));
    ck_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_mx4_dequant((const uint8_t*)codes.data_ptr(), (const uint8_t*)scales.data_ptr(), rows, k,
                       blocked ? CK_LAYOUT_BLOCKED : CK_LAYOUT_ROWS, (uint16_t*)y.data_ptr(), stream);
    Py_END_ALLOW_THREADS
    if (st != CK_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// mx4_gemm(x_codes, x_scales, w_codes, w_scales, m, n, bias, residual, out) -> y, or the C status of a refused call
PyObject* mx4_gemm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK(n == 9 && g_mx4_gemm, "mx4_gemm: 9 arguments, after bind()");
    const at::Tensor &xc = tensor_arg(a[0], "activation codes"), &xs = tensor_arg(a[1], "activation scales");
    const at::Tensor &wc = tensor_arg(a[2], "weight codes"), &ws = tensor_arg(a[3], "weight scales");
    const at::Tensor *bias = optional_arg(a[6], "bias"), *residual = optional_arg(a[7], "residual");
    const at::Tensor* out = optional_arg(a[8], "out");
    TORCH_CHECK_VALUE(xc.is_cuda(), "activation codes must be on a GPU, got ", xc.device());
    const c10::DeviceGuard guard(xc.device());
    check_blocked(xc, xs, "the activation", xc.device());
    check_blocked(wc, ws, "the weight", xc.device());
    const int64_t m = PyLong_AsLongLong(a[4]), nn = features_of(a[5], wc), k = xc.size(1) * 64;
    if (PyErr_Occurred()) return nullptr;
    TORCH_CHECK_VALUE(m >= 0 && pad(m, 32) == xc.size(0) * 32, "the activation's ", xc.size(0) * 32, " rows do not hold ", m);
    TORCH_CHECK_VALUE(wc.size(1) == xc.size(1), "in_features mismatch: activation ", k, ", weight ", wc.size(1) * 64);
    bool failed;
    void* stream = stream_of(xc, &failed);
    if (failed) return nullptr;
    Reads reads;
    if (out) reads.add({&xc, &xs, &wc, &ws, bias});
    const at::Tensor y = linear_out(out, m, nn, xc.options(), reads, bias, residual);
    ck_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_mx4_gemm((const uint8_t*)xc.data_ptr(), (const uint8_t*)xs.data_ptr(), (const uint8_t*)wc.data_ptr(),
                    (const uint8_t*)ws.data_ptr(), ptr_or_null<const float>(bias),
                    ptr_or_null<const uint16_t>(residual), m, nn, k, (uint16_t*)y.data_ptr(), stream);
    Py_END_ALLOW_THREADS
    if (st != CK_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// mx4_linear(x, w_codes, w_scales, n, group, act, bias, residual, out, workspace, k) -> y, or the C status of a refused
// call.  k: the weight's in_features, or None where only its padded ones are known.
PyObject* mx4_linear(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK(n == 11 && g_mx4_linear, "mx4_linear: 11 arguments, after bind()");
    const at::Tensor& x = tensor_arg(a[0], "activation");
    const at::Tensor &wc = tensor_arg(a[1], "weight codes"), &ws = tensor_arg(a[2], "weight scales");
    const at::Tensor *bias = optional_arg(a[6], "bias"), *residual = optional_arg(a[7], "residual");
    const at::Tensor *out = optional_arg(a[8], "out"), *work = optional_arg(a[9], "workspace");
    const int64_t ld = rows_of(x, at::kBFloat16, "activation");
    const c10::DeviceGuard guard(x.device());
    check_blocked(wc, ws, "the weight", x.device());
    const int64_t m = x.size(0), nn = features_of(a[3], wc), group = PyLong_AsLongLong(a[4]);
    const int act = (int)PyLong_AsLong(a[5]);
    const bool known = a[10] != Py_None;
    const int64_t weight_k = known ? PyLong_AsLongLong(a[10]) : 0;
    if (PyErr_Occurred()) return nullptr;
    const int64_t k = act == CK_ACT_SWIGLU ? x.size(1) / 2 : x.size(1);
    TORCH_CHECK_VALUE(act != CK_ACT_SWIGLU || x.size(1) % 2 == 0, "gate and up need one width, got ", x.size(1), " columns");
    check_group(k, group);
    TORCH_CHECK_VALUE(!known || k == weight_k, "in_features mismatch: activation ", k, ", weight ", weight_k);
    TORCH_CHECK_VALUE(pad(k, 256) == wc.size(1) * 64, "in_features mismatch: activation ", k, ", weight ", wc.size(1) * 64,
                      " (padded to a multiple of 256)");
    bool failed;
    void* stream = stream_of(x, &failed);
    if (failed) return nullptr;
    Reads reads;
    if (out || work) reads.add({&x, &wc, &ws, bias});
    const at::Tensor y = linear_out(out, m, nn, x.options(), reads, bias, residual);
    if (work) reads.add({residual});
    const at::Tensor room = room_of(work, g_mx4_linear_size(m, k, nn), x.options(), reads, y);
    ck_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_mx4_linear((const uint16_t*)x.data_ptr(), ld, act, (const uint8_t*)wc.data_ptr(),
                      (const uint8_t*)ws.data_ptr(), ptr_or_null<const float>(bias),
                      ptr_or_null<const uint16_t>(residual), m, nn, k, (int32_t)group, (uint16_t*)y.data_ptr(), ptr(room),
                      bytes(room), stream);
    Py_END_ALLOW_THREADS
    if (st != CK_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// ---- between two sub-blocks ----

// Rows [batch, tokens, width] or [tokens, width] like x.
ck_rows norm_rows(const at::Tensor& t, const char* what, const at::Tensor& x)
{
    TORCH_CHECK_VALUE(t.device() == x.device() && t.scalar_type() == x.scalar_type() && t.sizes() == x.sizes(), what,
                      " needs a ", x.scalar_type(), " ", x.sizes(), " tensor on ", x.device(), ", got ", t.scalar_type(),
                      " ", t.sizes(), " on ", t.device());
    const bool three = t.dim() == 3;
    const int64_t sb = three && t.size(0) > 1 ? t.stride(0) : 0, st = t.size(-2) > 1 ? t.stride(-2) : 0;
    void* p = t.data_ptr();
    TORCH_CHECK_VALUE(t.stride(-1) == 1 && (sb | st) % 8 == 0 && sb >= 0 && (uintptr_t)p % 16 == 0, what,
                      " needs contiguous, 16-byte aligned rows (strides in multiples of 8 elements), got strides ",
                      t.strides());
    return ck_rows{p, sb, st};
}

// A modulation [width], [batch, width] (with x [batch, tokens, width]) or x's shape, the dimensions before the width of
// any size 1; of x's type or FP32.
ck_rows modulation(const at::Tensor* m, const char* what, const at::Tensor& x, int* dtype)
{
    if (!m) return ck_rows{};
    const int64_t w = x.size(-1);
    const bool f32 = m->scalar_type() == at::kFloat;
    TORCH_CHECK_VALUE(m->device() == x.device() && (f32 || m->scalar_type() == x.scalar_type()), what, " needs a ",
                      x.scalar_type(), " or float32 tensor on ", x.device(), ", got ", m->scalar_type(), " on ",
                      m->device());
    const int mine = f32 ? CK_DTYPE_FP32 : x.scalar_type() == at::kHalf ? CK_DTYPE_FP16 : CK_DTYPE_BF16;
    TORCH_CHECK_VALUE(*dtype < 0 || *dtype == mine, "gate, scale and shift need one type");
    *dtype = mine;
    ck_rows r{m->data_ptr(), 0, 0};
    const int64_t d = m->dim();
    bool fits = d >= 1 && d <= x.dim() && m->size(d - 1) == w;
    if (fits && d == x.dim()) {
        for (int64_t i = 0; i < d - 1; ++i) fits = fits && (m->size(i) == x.size(i) || m->size(i) == 1);
        if (fits) {
            r.batch_stride = d == 3 && m->size(0) > 1 ? m->stride(0) : 0;
            r.token_stride = m->size(d - 2) > 1 ? m->stride(d - 2) : 0;
        }
    } else if (fits && d == 2) {
        fits = m->size(0) == x.size(0);
        r.batch_stride = m->size(0) > 1 ? m->stride(0) : 0;
    }
    TORCH_CHECK_VALUE(fits, what, " needs shape (", w, ",)", x.dim() == 3 ? ", (batch, width)" : "", " or ", x.sizes(),
                      " with any of the sizes before the width 1, got ", m->sizes());
    const int64_t step = f32 ? 4 : 8;
    TORCH_CHECK_VALUE(m->stride(-1) == 1 && r.batch_stride >= 0 && (r.batch_stride | r.token_stride) % step == 0 &&
                          (uintptr_t)r.data % 16 == 0,
                      what, " needs contiguous, 16-byte aligned channels, got strides ", m->strides());
    return r;
}

const float* gain(const at::Tensor* t, const char* what, const at::Tensor& x)
{
    if (!t) return nullptr;
    TORCH_CHECK_VALUE(t->scalar_type() == at::kFloat && t->dim() == 1 && t->size(0) == x.size(-1) && t->is_contiguous() &&
                          t->device() == x.device() && (uintptr_t)t->data_ptr() % 16 == 0,
                      what, " needs a contiguous, 16-byte aligned float32 (", x.size(-1), ",) tensor on ", x.device());
    return static_cast<const float*>(t->data_ptr());
}

// An output of ck_block_norm: new and contiguous, or `out` checked: x or the branch itself, or apart from all that is read.
at::Tensor norm_out(const at::Tensor* out, const char* what, const at::Tensor& x, const ck_rows& rx,
                    const at::Tensor* branch, const ck_rows& rb, const Reads& reads, ck_rows* h)
{
    if (!out) {
        at::Tensor t = at::empty(x.sizes(), x.options());
        *h = ck_rows{t.data_ptr(), x.size(-2) * x.size(-1), x.size(-1)};
        return t;
    }
    *h = norm_rows(*out, what, x);
    const ck::View v = view_of(*out);
    for (int i = 0; i < x.dim(); ++i)
        TORCH_CHECK_VALUE(out->size(i) < 2 || out->stride(i) != 0, what, " must not be an expanded tensor");
    TORCH_CHECK_VALUE(v.distinct(), what, " must not hold an element twice, got strides ", out->strides());
    auto same = [&](const ck_rows& r) {
        return h->data == r.data && h->batch_stride == r.batch_stride && h->token_stride == r.token_stride;
    };
    const bool ok = (same(rx) || ck::disjoint(v, view_of(x))) &&
                    (!branch || same(rb) || ck::disjoint(v, view_of(*branch))) && reads.apart_from(v);
    TORCH_CHECK_VALUE(ok, what, " must be x or branch itself or share no memory with what the call reads");
    return *out;
}

// block_norm(x, branch, gate, residual_scale, branch_scale, branch_kind, branch_weight, branch_bias, kind, weight, bias,
// scale, shift, eps, x_out, out) -> out, x_out or (x_out, out), or the C status of a refused call
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK(n == 16 && g_block_norm, "block_norm: 16 arguments, after bind()");
    const at::Tensor& x = tensor_arg(a[0], "x");
    TORCH_CHECK_VALUE(x.is_cuda(), "x must be on a GPU, got ", x.device());
    TORCH_CHECK_VALUE(x.scalar_type() == at::kBFloat16 || x.scalar_type() == at::kHalf,
                      "x needs dtype bfloat16 or float16, got ", x.scalar_type());
    TORCH_CHECK_VALUE((x.dim() == 2 || x.dim() == 3) && x.size(-1) >= 8 && x.size(-1) % 8 == 0 &&
                          x.size(-1) <= CK_MAX_NORM_WIDTH,
                      "x needs shape ([batch,] tokens, width) with a width in multiples of 8 up to ", CK_MAX_NORM_WIDTH,
                      ", got ", x.sizes());
    const c10::DeviceGuard guard(x.device());
    const at::Tensor *branch = optional_arg(a[1], "branch"), *gate = optional_arg(a[2], "gate");
    const at::Tensor *bw = optional_arg(a[6], "branch_weight"), *bb = optional_arg(a[7], "branch_bias");
    const at::Tensor *w = optional_arg(a[9], "weight"), *b = optional_arg(a[10], "bias");
    const at::Tensor *scale = optional_arg(a[11], "scale"), *shift = optional_arg(a[12], "shift");
    const at::Tensor *xo = optional_arg(a[14], "x_out"), *ho = optional_arg(a[15], "out");
    ck_block_norm_args k{};
    k.residual_scale = (float)PyFloat_AsDouble(a[3]), k.branch_scale = (float)PyFloat_AsDouble(a[4]);
    k.branch_norm.kind = (int)PyLong_AsLong(a[5]), k.norm.kind = (int)PyLong_AsLong(a[8]);
    k.eps = (float)PyFloat_AsDouble(a[13]);
    if (PyErr_Occurred()) return nullptr;
    const bool normed = k.norm.kind != CK_NORM_NONE;
    TORCH_CHECK_VALUE(branch || (!gate && !xo && !bw && !bb && k.branch_norm.kind == CK_NORM_NONE),
                      "arguments for the branch without a branch");
    TORCH_CHECK_VALUE(normed || (!w && !b && !scale && !shift && !ho), "arguments for the norm without a norm");
    TORCH_CHECK_VALUE(normed || branch, "nothing to do: neither a branch nor a norm");
    TORCH_CHECK_VALUE(k.branch_norm.kind != CK_NORM_NONE || (!bw && !bb), "branch_weight or branch_bias without branch_norm");
    k.x = norm_rows(x, "x", x);
    if (branch) k.branch = norm_rows(*branch, "branch", x);
    k.batch = x.dim() == 3 ? x.size(0) : 1, k.tokens = x.size(-2), k.width = x.size(-1);
    k.branch_norm.weight = gain(bw, "branch_weight", x), k.branch_norm.bias = gain(bb, "branch_bias", x);
    k.norm.weight = gain(w, "weight", x), k.norm.bias = gain(b, "bias", x);
    k.dtype = x.scalar_type() == at::kHalf ? CK_DTYPE_FP16 : CK_DTYPE_BF16;
    int mod = -1;
    k.gate = modulation(gate, "gate", x, &mod);
    k.scale = modulation(scale, "scale", x, &mod);
    k.shift = modulation(shift, "shift", x, &mod);
    k.mod_dtype = mod < 0 ? k.dtype : mod;
    bool failed;
    void* stream = stream_of(x, &failed);
    if (failed) return nullptr;
    Reads reads;
    if (xo || ho) reads.add({gate, bw, bb, w, b, scale, shift});
    at::Tensor r, h;
    if (branch) r = norm_out(xo, "x_out", x, k.x, branch, k.branch, reads, &k.x_out);
    if (normed) h = norm_out(ho, "out", x, k.x, branch, k.branch, reads, &k.out);
    TORCH_CHECK_VALUE(!xo || !ho || ck::disjoint(view_of(r), view_of(h)), "x_out and out must not share memory");
    ck_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_block_norm(&k, stream);
    Py_END_ALLOW_THREADS
    if (st != CK_OK) return PyLong_FromLong(st);
    if (!branch) return THPVariable_Wrap(h);
    if (!normed) return THPVariable_Wrap(r);
    return pair(r, h);
    END_HANDLE_TH_ERRORS
}

// bind(functions..., stream): the addresses of the C functions of `slots` below and the callable that gives a device's
// current stream
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    void** const slots[] = {
        (void**)&g_norm, (void**)&g_attn, (void**)&g_attn_size, (void**)&g_mx4_prep, (void**)&g_mx4_quant,
        (void**)&g_mx4_dequant, (void**)&g_mx4_gemm, (void**)&g_mx4_linear, (void**)&g_mx4_linear_size,
        (void**)&g_block_norm};
    constexpr int kSlots = sizeof(slots) / sizeof(slots[0]);
    if (n != kSlots + 1) {
        PyErr_Format(PyExc_TypeError, "bind: %d arguments", kSlots + 1);
        return nullptr;
    }
    void* f[kSlots];
    for (int i = 0; i < kSlots; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null function");
            return nullptr;
        }
    }
    for (int i = 0; i < kSlots; ++i) *slots[i] = f[i];
    Py_INCREF(a[kSlots]);
    Py_XSETREF(g_stream, a[kSlots]);
    Py_RETURN_NONE;
}

#define CK_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CK_METHOD(qk_norm_rope), CK_METHOD(cross_attn), CK_METHOD(mx4_quant), CK_METHOD(mx4_dequant),
                         CK_METHOD(mx4_gemm),     CK_METHOD(mx4_linear), CK_METHOD(block_norm), CK_METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
