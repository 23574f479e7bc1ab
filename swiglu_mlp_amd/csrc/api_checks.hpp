// api_checks.hpp -- argument checks that the entry points' files (api.hip,
// api_block.hip) share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ck.h"

#define CK_TRY(expr)                     \
    do {                                 \
        const ck_status st_ = (expr);    \
        if (st_ != CK_OK) return st_;    \
    } while (0)

namespace ck {
namespace api {

constexpr size_t kAlign = 256;

inline size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool pow2_group(int32_t g) { return g >= 1 && g <= 256 && (g & (g - 1)) == 0; }

// Checks shared by every call that takes an in_features dimension.
inline ck_status check_k(int64_t k, int32_t group)
{
    if (!pow2_group(group)) return CK_EUNSUPPORTED;
    if (k < 1) return CK_ESHAPE;
    if (k > CK_MAX_K) return CK_EUNSUPPORTED;
    if (k % 64 != 0 || k % group != 0) return CK_ESHAPE;
    return CK_OK;
}

inline ck_status check_act(int32_t act, int64_t ldx, int64_t k)
{
    if (act != CK_ACT_NONE && act != CK_ACT_SWIGLU) return CK_EINVAL;
    const int64_t need = act == CK_ACT_SWIGLU ? 2 * k : k;
    if (ldx < need || ldx % 8 != 0) return CK_ESHAPE;
    return CK_OK;
}

inline ck_status from_hip(hipError_t e) { return e == hipSuccess ? CK_OK : CK_EHIP; }

// a * b * c of non-negative sizes, or limit if it is not below it.
inline int64_t product_below(int64_t a, int64_t b, int64_t c, int64_t limit)
{
    if (a == 0 || b == 0 || c == 0) return 0;
    if (a >= limit || b >= limit || c >= limit || a * b >= limit) return limit;
    return a * b * c < limit ? a * b * c : limit;
}

constexpr int64_t kMaxIndex = 0x7fffffffLL;   // a dimension alone

}  // namespace api
}  // namespace ck
