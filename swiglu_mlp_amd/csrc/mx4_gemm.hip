// mx4_gemm.hip -- the product of microscaled 4-bit operands (include/ck.h, "MX
// FP4 linears"): y[m, n] = bf16(sum_k x[m, k] w[n, k] (+ bias[n]) (+ residual[m, n])),
// both operands in the blocked layout.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 x 64 by 64 x 32 values of 4
// bits, each lane's 32 with a scale of its own, and adds in FP32.  W is its A
// operand and x its B operand, so a lane ends with four consecutive n of one m.
#include "ck_internal.hpp"
#include "mx4.hpp"

namespace ck {
namespace mx4 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// One 32 x 32 tile of y per wave, operands straight from memory.
__global__ __launch_bounds__(256) void mx4_gemm_kernel(const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                                                       const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
                                                       int64_t M, int64_t N, uint32_t units, uint32_t tiles_m,
                                                       uint32_t tiles, uint16_t* __restrict__ y, EpiExtra ex)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const uint32_t tile = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (tile >= tiles) return;
    const uint32_t tn = tile / tiles_m, tm = tile - tn * tiles_m;
    const int lane = threadIdx.x & 63;
    v16f acc = {};
    for (uint32_t u = 0; u < units; ++u) {
        const int64_t cw = (int64_t)tn * units + u, cx = (int64_t)tm * units + u;
        const int sw = *reinterpret_cast<const int*>(ws + cw * 256 + lane * 4);
        const int sx = *reinterpret_cast<const int*>(xs + cx * 256 + lane * 4);
        v8i a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const v4i p = *reinterpret_cast<const v4i*>(wc + cw * 4096 + j * 1024 + lane * 16);
            const v4i q = *reinterpret_cast<const v4i*>(xc + cx * 4096 + j * 1024 + lane * 16);
            a[j] = v8i{p[0], p[1], p[2], p[3], 0, 0, 0, 0};
            b[j] = v8i{q[0], q[1], q[2], q[3], 0, 0, 0, 0};
        }
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[0], b[0], acc, 4, 4, 0, sw, 0, sx);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[1], b[1], acc, 4, 4, 1, sw, 1, sx);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[2], b[2], acc, 4, 4, 2, sw, 2, sx);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[3], b[3], acc, 4, 4, 3, sw, 3, sx);
    }
    const int64_t m = (int64_t)tm * 32 + (lane & 31);
    if (m >= M) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t n = (int64_t)tn * 32 + 8 * q + 4 * (lane >> 5);
        if (n >= N) break;
        float v[4] = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
        if (ex.bias)
            for (int i = 0; i < 4; ++i) v[i] += ex.bias[n + i];
        if (ex.res) {
            const uint2 r = *reinterpret_cast<const uint2*>(ex.res + m * N + n);
            v[0] += bf16_lo(r.x), v[1] += bf16_hi(r.x), v[2] += bf16_lo(r.y), v[3] += bf16_hi(r.y);
        }
        *reinterpret_cast<uint2*>(y + m * N + n) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
#endif
}

}  // namespace mx4

size_t mx4_gemm_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mx4_gemm(const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* ws, int64_t m,
                           int64_t n, int64_t k, uint16_t* y, EpiExtra ex, void*, hipStream_t st)
{
    const uint32_t units = (uint32_t)(mx4::pad_cols(k) / 256);
    const uint32_t tm = (uint32_t)(mx4::pad_rows(m) / 32), tn = (uint32_t)(mx4::pad_rows(n) / 32), tiles = tm * tn;
    mx4::mx4_gemm_kernel<<<dim3((tiles + 3) / 4), dim3(256), 0, st>>>(xc, xs, wc, ws, m, n, units, tm, tiles, y, ex);
    return hipGetLastError();
}

}  // namespace ck
