// api_block.hip -- the C ABI (include/ck.h) of the MX FP4 linears and of
// ck_block_norm: host-side argument checks, workspace carving and dispatch, as
// in api.hip.
#include "api_checks.hpp"
#include "ck.h"
#include "ck_internal.hpp"
#include "mx4.hpp"

using namespace ck::api;

namespace {

constexpr int64_t kMaxValues = 1LL << 34;     // of an operand, padded: launches below 2^32 threads
constexpr int64_t kMaxOutputs = 1LL << 35;    // m * n
constexpr int64_t kMaxFeatures = 1LL << 21;   // a tile's 256 rows of y in 31-bit offsets

size_t codes_bytes(int64_t rows, int64_t k) { return (size_t)(ck::mx4::pad_rows(rows) * ck::mx4::pad_cols(k) / 2); }
size_t scales_bytes(int64_t rows, int64_t k) { return (size_t)(ck::mx4::pad_rows(rows) * ck::mx4::pad_cols(k) / 32); }

// Sizes of an operand [rows, k].
ck_status check_operand(int64_t rows, int64_t k, int32_t group)
{
    CK_TRY(check_k(k, group));
    if (rows < 0) return CK_ESHAPE;
    if (rows > kMaxIndex || ck::mx4::pad_rows(rows) * ck::mx4::pad_cols(k) >= kMaxValues) return CK_EUNSUPPORTED;
    return CK_OK;
}

ck_status check_rows_or_blocked(int32_t layout)
{
    return layout == CK_LAYOUT_ROWS || layout == CK_LAYOUT_BLOCKED ? CK_OK : CK_EINVAL;
}

// Sizes of a product.
ck_status check_product(int64_t m, int64_t n, int64_t k, int32_t group)
{
    CK_TRY(check_operand(m, k, group));
    CK_TRY(check_operand(n, k, group));
    if (n % 16 != 0) return CK_ESHAPE;
    if (n >= kMaxFeatures || (m > 0 && n >= kMaxOutputs / m)) return CK_EUNSUPPORTED;
    return CK_OK;
}

// Bias is read as float4, the residual as 16-byte groups.
ck_status check_epilogue(const float* bias, const uint16_t* residual, const uint16_t* y)
{
    if (!y || !aligned16(y)) return CK_EINVAL;
    if (bias && !aligned16(bias)) return CK_EINVAL;
    if (residual && !aligned16(residual)) return CK_EINVAL;
    return CK_OK;
}

bool good_workspace(const void* ws, size_t bytes, size_t need)
{
    return need == 0 || (ws && bytes >= need && ((uintptr_t)ws % kAlign) == 0);
}

}  // namespace

extern "C" {

int64_t ck_mx4_rows(int64_t rows) { return rows <= 0 ? 0 : ck::mx4::pad_rows(rows); }
int64_t ck_mx4_cols(int64_t k) { return k <= 0 ? 0 : ck::mx4::pad_cols(k); }

ck_status ck_mx4_weight_prep(const float* w, int64_t n, int64_t k, int32_t group, int32_t layout, uint8_t* codes,
                             uint8_t* scales, void* stream)
{
    CK_TRY(check_rows_or_blocked(layout));
    CK_TRY(check_operand(n, k, group));
    if (n == 0) return CK_OK;
    if (!w || !codes || !scales || !aligned16(w) || !aligned16(codes) || !aligned16(scales)) return CK_EINVAL;
    return from_hip(ck::launch_mx4_quant(2, w, k, n, k, group, layout == CK_LAYOUT_BLOCKED, codes, scales,
                                         (hipStream_t)stream));
}

ck_status ck_mx4_weight_pack(const uint8_t* codes, const uint8_t* scales, int64_t n, int64_t k, uint8_t* codes_blk,
                             uint8_t* scales_blk, void* stream)
{
    CK_TRY(check_operand(n, k, 1));
    if (n == 0) return CK_OK;
    if (!codes || !scales || !codes_blk || !scales_blk || !aligned16(codes) || !aligned16(codes_blk) ||
        !aligned16(scales_blk))
        return CK_EINVAL;
    return from_hip(ck::launch_mx4_pack(codes, scales, n, k, codes_blk, scales_blk, (hipStream_t)stream));
}

ck_status ck_mx4_act_quant(const uint16_t* x, int64_t ldx, int64_t m, int64_t k, int32_t act, int32_t group,
                           int32_t layout, uint8_t* codes, uint8_t* scales, void* stream)
{
    CK_TRY(check_rows_or_blocked(layout));
    CK_TRY(check_operand(m, k, group));
    CK_TRY(check_act(act, ldx, k));
    if (m == 0) return CK_OK;
    if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales)) return CK_EINVAL;
    return from_hip(ck::launch_mx4_quant(act == CK_ACT_SWIGLU ? 1 : 0, x, ldx, m, k, group,
                                         layout == CK_LAYOUT_BLOCKED, codes, scales, (hipStream_t)stream));
}

ck_status ck_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t k, int32_t layout,
                         uint16_t* y, void* stream)
{
    CK_TRY(check_rows_or_blocked(layout));
    CK_TRY(check_operand(rows, k, 1));
    if (rows == 0) return CK_OK;
    if (!codes || !scales || !y || !aligned16(codes) || !aligned16(y)) return CK_EINVAL;
    return from_hip(ck::launch_mx4_dequant(codes, scales, rows, k, layout == CK_LAYOUT_BLOCKED, y,
                                           (hipStream_t)stream));
}

ck_status ck_mx4_gemm_bf16(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                           const uint8_t* w_scales, const float* bias, const uint16_t* residual, int64_t m, int64_t n,
                           int64_t k, uint16_t* y, void* stream)
{
    CK_TRY(check_product(m, n, k, 1));
    if (m == 0 || n == 0) return CK_OK;
    if (!x_codes || !x_scales || !w_codes || !w_scales || !aligned16(x_codes) || !aligned16(x_scales) ||
        !aligned16(w_codes) || !aligned16(w_scales))
        return CK_EINVAL;
    CK_TRY(check_epilogue(bias, residual, y));
    return from_hip(ck::launch_mx4_gemm(x_codes, x_scales, w_codes, w_scales, m, n, k, y,
                                        ck::EpiExtra{bias, residual}, (hipStream_t)stream));
}

// The activation's codes, then its scales; nothing where the quantizer is inside the
// product.
size_t ck_mx4_linear_workspace_size(int64_t m, int64_t k, int64_t n)
{
    if (m <= 0 || n <= 0 || check_product(m, n, k, 1) != CK_OK || ck::mx4_fused(m, k)) return 0;
    return round_up(codes_bytes(m, k)) + round_up(scales_bytes(m, k));
}

ck_status ck_mx4_linear(const uint16_t* x, int64_t ldx, int32_t act, const uint8_t* w_codes, const uint8_t* w_scales,
                        const float* bias, const uint16_t* residual, int64_t m, int64_t n, int64_t k, int32_t group,
                        uint16_t* y, void* workspace, size_t workspace_bytes, void* stream)
{
    CK_TRY(check_product(m, n, k, group));
    CK_TRY(check_act(act, ldx, k));
    if (m == 0 || n == 0) return CK_OK;
    if (!x || !w_codes || !w_scales || !aligned16(x) || !aligned16(w_codes) || !aligned16(w_scales)) return CK_EINVAL;
    CK_TRY(check_epilogue(bias, residual, y));
    if (!good_workspace(workspace, workspace_bytes, ck_mx4_linear_workspace_size(m, k, n))) return CK_EWORKSPACE;
    hipStream_t st = (hipStream_t)stream;
    if (ck::mx4_fused(m, k))   // the quantizer inside the product: one launch, no workspace
        return from_hip(ck::launch_mx4_fused(act == CK_ACT_SWIGLU ? 1 : 0, x, ldx, w_codes, w_scales, m, n, k, group, y,
                                             ck::EpiExtra{bias, residual}, st));
    uint8_t* xc = static_cast<uint8_t*>(workspace);
    uint8_t* xs = xc + round_up(codes_bytes(m, k));
    CK_TRY(from_hip(ck::launch_mx4_quant(act == CK_ACT_SWIGLU ? 1 : 0, x, ldx, m, k, group, true, xc, xs, st)));
    return from_hip(ck::launch_mx4_gemm(xc, xs, w_codes, w_scales, m, n, k, y, ck::EpiExtra{bias, residual}, st));
}

// ---- between two sub-blocks ----

static ck_status check_rows(const ck_rows& r, int64_t step)
{
    if (!aligned16(r.data)) return CK_EINVAL;
    for (const int64_t st : {r.batch_stride, r.token_stride})
        if (st < 0 || st >= (1LL << 40) || st % step != 0) return CK_ESHAPE;
    return CK_OK;
}

static ck_status check_norm(const ck_norm& n)
{
    if (n.kind != CK_NORM_NONE && n.kind != CK_NORM_RMS && n.kind != CK_NORM_LAYER) return CK_EINVAL;
    if (n.kind == CK_NORM_NONE && (n.weight || n.bias)) return CK_EINVAL;
    if (!aligned16(n.weight) || !aligned16(n.bias)) return CK_EINVAL;
    return CK_OK;
}

static bool finite(float v) { return v >= -3.4028235e38f && v <= 3.4028235e38f; }

ck_status ck_block_norm(const ck_block_norm_args* a, void* stream)
{
    if (!a) return CK_EINVAL;
    if (a->dtype != CK_DTYPE_BF16 && a->dtype != CK_DTYPE_FP16) return CK_EINVAL;
    if (a->mod_dtype != a->dtype && a->mod_dtype != CK_DTYPE_FP32) return CK_EINVAL;
    if (!(a->eps >= 0x1p-126f) || !finite(a->eps) || !finite(a->residual_scale) || !finite(a->branch_scale))
        return CK_EINVAL;
    if (a->batch < 0 || a->tokens < 0 || a->width < 8 || a->width % 8 != 0) return CK_ESHAPE;
    if (a->width > CK_MAX_NORM_WIDTH) return CK_EUNSUPPORTED;
    constexpr int64_t kMaxRows = 1 << 24;
    const int64_t rows = product_below(a->batch, a->tokens, 1, kMaxRows);
    if (rows >= kMaxRows) return CK_EUNSUPPORTED;
    CK_TRY(check_norm(a->norm));
    CK_TRY(check_norm(a->branch_norm));
    if (!a->branch.data && (a->branch_norm.kind != CK_NORM_NONE || a->gate.data || a->x_out.data)) return CK_EINVAL;
    if (a->norm.kind == CK_NORM_NONE && (a->out.data || a->scale.data || a->shift.data)) return CK_EINVAL;
    const int64_t mod_step = a->mod_dtype == CK_DTYPE_FP32 ? 4 : 8;
    for (const ck_rows* r : {&a->x, &a->branch, &a->x_out, &a->out}) CK_TRY(check_rows(*r, 8));
    for (const ck_rows* r : {&a->gate, &a->scale, &a->shift}) CK_TRY(check_rows(*r, mod_step));
    if (rows == 0) return CK_OK;
    if (!a->x.data || (!a->x_out.data && !a->out.data)) return CK_EINVAL;
    ck::BlockNormArgs k{};
    k.x = static_cast<const uint16_t*>(a->x.data), k.branch = static_cast<const uint16_t*>(a->branch.data);
    k.x_out = static_cast<uint16_t*>(a->x_out.data), k.out = static_cast<uint16_t*>(a->out.data);
    k.x_sb = a->x.batch_stride, k.x_st = a->x.token_stride;
    k.b_sb = a->branch.batch_stride, k.b_st = a->branch.token_stride;
    k.xo_sb = a->x_out.batch_stride, k.xo_st = a->x_out.token_stride;
    k.o_sb = a->out.batch_stride, k.o_st = a->out.token_stride;
    k.batch = a->batch, k.tokens = a->tokens, k.width = a->width;
    k.gate = {a->gate.data, a->gate.batch_stride, a->gate.token_stride};
    k.scale = {a->scale.data, a->scale.batch_stride, a->scale.token_stride};
    k.shift = {a->shift.data, a->shift.batch_stride, a->shift.token_stride};
    k.bw = a->branch_norm.weight, k.bb = a->branch_norm.bias, k.branch_kind = a->branch_norm.kind;
    k.w = a->norm.weight, k.b = a->norm.bias, k.kind = a->norm.kind;
    k.mod32 = a->mod_dtype == CK_DTYPE_FP32, k.fp16 = a->dtype == CK_DTYPE_FP16;
    k.residual_scale = a->residual_scale, k.branch_scale = a->branch_scale, k.eps = a->eps;
    return from_hip(ck::launch_block_norm(k, (hipStream_t)stream));
}

}  // extern "C"
