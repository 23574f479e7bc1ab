// mx4.hpp -- microscaled 4-bit operands (include/ck.h, "MX FP4 linears"): where
// codes and scales lie, and the device steps that the quantizer and the few-row
// product share.
#pragma once
#include "ck_device.hpp"
#include "heads.hpp"

namespace ck {
namespace mx4 {

// Blocked layout of an operand [rows, k]: rows padded to 32, k to 256.
//   codes:  1 KB block (r / 32, k / 64) at ((r / 32) * (kp / 64) + k / 64) * 1024,
//           inside it ((k % 64) / 32) * 512 + (r % 32) * 16 + (k % 32) / 2, the
//           even k in the low nibble: one operand of the 32 x 32 x 64 product in
//           lane order (lane 32 h + r holds row r, the 32 values of half h);
//   scales: 256 bytes (r / 32, k / 256) at ((r / 32) * (kp / 256) + k / 256) * 256,
//           inside it (32 h + r % 32) * 4 + (k % 256) / 64: the four scales of a
//           lane in one register, picked by the product's scale select.
constexpr int kRows = 32;
constexpr int kCols = 256;
inline int64_t pad_rows(int64_t rows) { return (rows + kRows - 1) / kRows * kRows; }
inline int64_t pad_cols(int64_t k) { return (k + kCols - 1) / kCols * kCols; }

// E8M0 scale byte of a block whose largest magnitude is a: floor(log2 a) - 2,
// biased by 127 and not below 0; 255 (NaN) where a is infinite or NaN.
__device__ __forceinline__ uint32_t scale_byte(float a)
{
    const uint32_t e = (__float_as_uint(a) >> 23) & 0xffu;
    return e == 255u ? 255u : max(e, 2u) - 2u;
}

// 2^(byte - 127), byte < 255 (2^-127 is a subnormal).
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(max(byte << 23, 0x00400000u)); }

// silu(g) * u for the quantizer, within (8 + 1.25 max(-g, 0)) 2^-24 of itself from g =
// -87 on, far below half a step of a 4-bit value.  In units of 2^-24: the hardware's
// exponential and reciprocal (1 ulp) 2 each, the sum and the products by g and u 1
// each; the constant log2(e) 0.23 and the product with it 1, both times |g| as errors
// of an exponent (for positive g their share e^-g / (1 + e^-g), below 0.28 / g).
// Below -87, where silu is under 2^-119, the reciprocal is subnormal and then, e^-g
// past FP32, zero: -0.  g = -inf gives NaN (-inf * 0).
__device__ __forceinline__ float silu_mul(float g, float u)
{
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -0x1.715476p+0f)) * u;
}

// Eight values as codes (to the nearest, ties to even, at most 6 in magnitude)
// of scale s: one v_cvt_scalef32_pk_fp4_f32 a pair.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float s)
{
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
    return q;
}

__device__ __forceinline__ float max_abs(float a, float b, float c)   // NaN if one is
{
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b)),
                                         __builtin_fabsf(c));
}

// One lane's 32 consecutive values of a row -> its 16 bytes of codes and its
// scale byte.  Rotates groups of 2^LOG_G values first (lane kb of the row holds
// values 32 kb .. 32 kb + 31; lanes kb ^ 1, ^ 2, ^ 4 are its neighbours in the
// wave): strides up to 16 inside the lane, the others by lane exchange in the
// sign-folded form of fwht_cross_lane_signed (the lane then holds sigma times
// its values; the codes' sign bits are flipped back).
template <int LOG_G>
__device__ __forceinline__ uint4 quantize32(float (&v)[4][8], int lane, uint32_t* byte)
{
    uint32_t flip = 0;
    if constexpr (LOG_G > 0) {
        constexpr int IN = LOG_G < 5 ? LOG_G : 5;
#pragma unroll
        for (int j = 0; j < 4; ++j) fwht_in_lane<(1 << (IN < 3 ? IN : 3))>(v[j]);
#pragma unroll
        for (int h = 1; h < 4 && 8 * h < (1 << IN); h <<= 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j & h) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = v[j][i], q = v[j + h][i];
                    v[j][i] = p + q;
                    v[j + h][i] = p - q;
                }
            }
        }
        if constexpr (LOG_G >= 6) {
            const float t = (lane & 1) ? -1.0f : 1.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) fmac_dpp8<0xB1>(v[j], t);
            flip = (lane & 1) ? 0x88888888u : 0u;
        }
        if constexpr (LOG_G >= 7) {
            const float t = (lane & 2) ? -1.0f : 1.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) fmac_dpp8<0x4E>(v[j], t);
            flip ^= (lane & 2) ? 0x88888888u : 0u;
        }
        if constexpr (LOG_G >= 8) {
            const float t = (lane & 4) ? -1.0f : 1.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = __builtin_fmaf(v[j][i], t, swizzle_xor<4>(v[j][i]));
        }
        // 1 / sqrt(g): a power of two for even LOG_G, else one rounding of 2^-24
        // (before the scale is chosen, so a value and its block's largest see the same one)
        constexpr float c = (LOG_G & 1 ? 0x1.6a09e6p-1f : 1.0f) / (float)(1 << (LOG_G / 2));
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * c;
    }
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 8; i += 2) a = max_abs(v[j][i], v[j][i + 1], a);
    *byte = scale_byte(a);
    const float s = scale_value(min(*byte, 254u));
    return make_uint4(codes8(v[0], s) ^ flip, codes8(v[1], s) ^ flip, codes8(v[2], s) ^ flip, codes8(v[3], s) ^ flip);
}

// 32 values from element `at` on.  KIND 0: BF16 x; 1: BF16 [gate | up] (up k
// further), silu(gate) * up; 2: FP32.
template <int KIND>
__device__ __forceinline__ void load32(const void* __restrict__ src, int64_t at, int64_t k, float (&v)[4][8])
{
    if constexpr (KIND == 2) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<float4*>(v[j]) = p[2 * j];
            *reinterpret_cast<float4*>(v[j] + 4) = p[2 * j + 1];
        }
    } else {
        const uint16_t* x = static_cast<const uint16_t*>(src) + at;
        uint4 a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = reinterpret_cast<const uint4*>(x)[j];
        if constexpr (KIND == 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = reinterpret_cast<const uint4*>(x + k)[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            unpack8<bf16>(a[j], v[j]);
            if constexpr (KIND == 1) {
                float u[8];
                unpack8<bf16>(b[j], u);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = silu_mul(v[j][i], u[i]);
            }
        }
    }
}

}  // namespace mx4
}  // namespace ck
