// mx4_quant.hip -- quantization to microscaled 4-bit floating point, the
// relayout of serialized weights, and the way back (include/ck.h, "MX FP4
// linears").
//
// Every block of 32 consecutive k has a scale of its own, so unlike the INT8
// quantizer nothing is reduced over a row: a lane takes one block (32 values),
// and only the rotation's strides from 32 up cross lanes, within the eight lanes
// of 256 values.  A wave takes 8 rows x 256 values and a workgroup 32 x 256: in
// the blocked layout that is 4 KB of codes and 256 bytes of scales, both
// contiguous, written in pieces of 128 bytes or more.  With SwiGLU, whose rows are
// two streams, it is 4 x 512 and 16 x 512: reads of 1 KB keep memory busier there
// (200 million values in rows of 5120, 8192, 12288 and 28672: 170, 155, 161 and 162 us
// for 187, 157, 172 and 174; rows of 11008 are the other way, 171 for 160), not in one
// stream (98304 x 4096 171 us for 162).  A lane's four 16-byte loads of a row meet in
// the same cache lines; marked nontemporal they fetch each line four times (281 us for
// 176).
//
// Bound by HBM: 49152 x 4096 BF16 rotated by 128, 510 MB, 80 us (6.4 TB/s); 16384 x
// 12288 with SwiGLU, 912 MB, 168 us (5.4; without its arithmetic 8 us less); FP32
// 12288 x 4096, 228 MB, 46 us (5.0); back to BF16, 127 MB, 19.5 us (6.5); 16 rows
// 2.2 to 4 us, a launch.
#include "ck_internal.hpp"
#include "mx4.hpp"

namespace ck {
namespace mx4 {

template <int KIND>
constexpr uint32_t kQuantRows = KIND == 1 ? 16 : 32;   // of a workgroup

// units: of 256 values of a row; wide: workgroups along a row.
template <int KIND, int LOG_G, bool BLOCKED>
__global__ __launch_bounds__(256) void mx4_quant_kernel(const void* __restrict__ src, int64_t ld, int64_t m, int64_t k,
                                                        uint32_t units, uint32_t wide, uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales)
{
    constexpr uint32_t ROWS = kQuantRows<KIND>, LANES = 256 / ROWS;   // lanes of a row
    const uint32_t rg = blockIdx.x / wide;
    const uint32_t unit = (blockIdx.x - rg * wide) * (LANES / 8) + threadIdx.x % LANES / 8;
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)rg * ROWS + threadIdx.x / LANES;
    const uint32_t kb = unit * 8 + (lane & 7);   // the row's block of 32
    const bool live = row < m && (int64_t)kb * 32 < k;
    float v[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    // lanes past k or m hold zeros and stay for the exchanges; a group never
    // reaches past k (it divides it)
    if (live) load32<KIND>(src, row * ld + (int64_t)kb * 32, k, v);
    uint32_t byte;
    uint4 q = quantize32<LOG_G>(v, lane, &byte);
    if constexpr (BLOCKED) {
        // the four scales of a (row, half) in its first lane: lanes + 2, + 4, + 6
        uint32_t w = byte | (uint32_t)__builtin_amdgcn_update_dpp(0, (int)byte, 0x4E, 0xf, 0xf, false) << 8;
        w |= (uint32_t)__builtin_amdgcn_ds_swizzle((int)w, (4 << 10) | 0x1f) << 16;
        if (unit >= units) return;   // (the grid ends with the padding rows)
        if (!live) q = make_uint4(0, 0, 0, 0);   // padding is zero, and so is its scale byte; not the rotation's -0
        const uint32_t r = (uint32_t)row & 31, h = lane & 1, j = (lane >> 1) & 3;
        const int64_t chunk = (row >> 5) * units + unit;
        *reinterpret_cast<uint4*>(codes + chunk * 4096 + j * 1024 + h * 512 + r * 16) = q;
        if (j == 0) *reinterpret_cast<uint32_t*>(scales + chunk * 256 + (h * 32 + r) * 4) = w;
    } else if (live) {
        *reinterpret_cast<uint4*>(codes + row * (k / 2) + kb * 16) = q;
        scales[row * (k / 32) + kb] = (uint8_t)byte;
    }
}

// Row-major codes [n, k / 2] and scales [n, k / 32] -> blocked; rows and columns
// of padding are zero.  One lane a block of 32, as above.
__global__ __launch_bounds__(256) void mx4_pack_kernel(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, int64_t n, int64_t k,
                                                       uint32_t units, uint8_t* __restrict__ out,
                                                       uint8_t* __restrict__ out_scales)
{
    const uint32_t rb = blockIdx.x / units, unit = blockIdx.x - rb * units;
    const uint32_t r = threadIdx.x >> 3, h = threadIdx.x & 1, j = (threadIdx.x >> 1) & 3;
    const int64_t row = (int64_t)rb * 32 + r;
    const uint32_t kb = unit * 8 + (threadIdx.x & 7);
    uint4 q = make_uint4(0, 0, 0, 0);
    uint8_t s = 0;
    if (row < n && (int64_t)kb * 32 < k) {
        q = *reinterpret_cast<const uint4*>(codes + row * (k / 2) + kb * 16);
        s = scales[row * (k / 32) + kb];
    }
    const int64_t chunk = (int64_t)rb * units + unit;
    *reinterpret_cast<uint4*>(out + chunk * 4096 + j * 1024 + h * 512 + r * 16) = q;
    out_scales[chunk * 256 + (h * 32 + r) * 4 + j] = s;
}

// Codes and scales -> BF16 [m, k] (exact; past BF16's range infinite).  A lane
// takes 8 values: 4 bytes of codes, 16 of values.
template <bool BLOCKED>
__global__ __launch_bounds__(256) void mx4_dequant_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, int64_t m, int64_t k,
                                                          uint32_t units, uint16_t* __restrict__ out)
{
    const uint32_t rg = blockIdx.x / units, unit = blockIdx.x - rg * units;   // 8 rows, 256 values
    const uint32_t t = threadIdx.x & 31;
    const int64_t row = (int64_t)rg * 8 + (threadIdx.x >> 5);
    const int64_t at = (int64_t)unit * 256 + t * 8;
    if (row >= m || at >= k) return;
    const uint32_t kb = t >> 2;   // block of 32 in the unit
    uint32_t q, byte;
    if constexpr (BLOCKED) {
        const int64_t chunk = (row >> 5) * units + unit;
        const uint32_t r = (uint32_t)row & 31, h = kb & 1, j = kb >> 1;
        q = *reinterpret_cast<const uint32_t*>(codes + chunk * 4096 + j * 1024 + h * 512 + r * 16 + (t & 3) * 4);
        byte = scales[chunk * 256 + (h * 32 + r) * 4 + j];
    } else {
        q = *reinterpret_cast<const uint32_t*>(codes + row * (k / 2) + at / 2);
        byte = scales[row * (k / 32) + unit * 8 + kb];
    }
    const float s = scale_value(min(byte, 254u));
    uint4 o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
    if (byte == 255u) o = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    *reinterpret_cast<uint4*>(out + row * k + at) = o;
}

}  // namespace mx4

namespace {

template <int KIND, int LOG_G>
hipError_t launch_quant(const void* src, int64_t ld, int64_t m, int64_t k, bool blocked, uint8_t* codes,
                        uint8_t* scales, hipStream_t st)
{
    const uint32_t units = (uint32_t)(mx4::pad_cols(k) / 256);
    constexpr uint32_t rows = mx4::kQuantRows<KIND>, row_units = 32 / rows;
    const uint32_t wide = (units + row_units - 1) / row_units;
    const int64_t all = blocked ? mx4::pad_rows(m) : m;
    const dim3 grid((uint32_t)((all + rows - 1) / rows) * wide);
    if (blocked)
        mx4::mx4_quant_kernel<KIND, LOG_G, true><<<grid, dim3(256), 0, st>>>(src, ld, m, k, units, wide, codes, scales);
    else
        mx4::mx4_quant_kernel<KIND, LOG_G, false><<<grid, dim3(256), 0, st>>>(src, ld, m, k, units, wide, codes, scales);
    return hipGetLastError();
}

template <int KIND>
hipError_t pick_group(const void* src, int64_t ld, int64_t m, int64_t k, int g, bool blocked, uint8_t* codes,
                      uint8_t* scales, hipStream_t st)
{
    switch (g) {
        case 1: return launch_quant<KIND, 0>(src, ld, m, k, blocked, codes, scales, st);
        case 2: return launch_quant<KIND, 1>(src, ld, m, k, blocked, codes, scales, st);
        case 4: return launch_quant<KIND, 2>(src, ld, m, k, blocked, codes, scales, st);
        case 8: return launch_quant<KIND, 3>(src, ld, m, k, blocked, codes, scales, st);
        case 16: return launch_quant<KIND, 4>(src, ld, m, k, blocked, codes, scales, st);
        case 32: return launch_quant<KIND, 5>(src, ld, m, k, blocked, codes, scales, st);
        case 64: return launch_quant<KIND, 6>(src, ld, m, k, blocked, codes, scales, st);
        case 128: return launch_quant<KIND, 7>(src, ld, m, k, blocked, codes, scales, st);
        default: return launch_quant<KIND, 8>(src, ld, m, k, blocked, codes, scales, st);
    }
}

}  // namespace

hipError_t launch_mx4_quant(int kind, const void* src, int64_t ld, int64_t m, int64_t k, int g, bool blocked,
                            uint8_t* codes, uint8_t* scales, hipStream_t st)
{
    switch (kind) {
        case 0: return pick_group<0>(src, ld, m, k, g, blocked, codes, scales, st);
        case 1: return pick_group<1>(src, ld, m, k, g, blocked, codes, scales, st);
        default: return pick_group<2>(src, ld, m, k, g, blocked, codes, scales, st);
    }
}

hipError_t launch_mx4_pack(const uint8_t* codes, const uint8_t* scales, int64_t n, int64_t k, uint8_t* out,
                           uint8_t* out_scales, hipStream_t st)
{
    const uint32_t units = (uint32_t)(mx4::pad_cols(k) / 256);
    mx4::mx4_pack_kernel<<<dim3((uint32_t)(mx4::pad_rows(n) / 32) * units), dim3(256), 0, st>>>(codes, scales, n, k,
                                                                                              units, out, out_scales);
    return hipGetLastError();
}

hipError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t m, int64_t k, bool blocked,
                              uint16_t* out, hipStream_t st)
{
    const uint32_t units = (uint32_t)(mx4::pad_cols(k) / 256);
    const dim3 grid((uint32_t)((m + 7) / 8) * units);
    if (blocked)
        mx4::mx4_dequant_kernel<true><<<grid, dim3(256), 0, st>>>(codes, scales, m, k, units, out);
    else
        mx4::mx4_dequant_kernel<false><<<grid, dim3(256), 0, st>>>(codes, scales, m, k, units, out);
    return hipGetLastError();
}

}  // namespace ck
