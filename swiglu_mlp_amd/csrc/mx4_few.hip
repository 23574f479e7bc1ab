// mx4_few.hip -- the product of microscaled 4-bit operands (include/ck.h, "MX FP4
// linears") where it is small: few rows of x, the weight streamed once, or few
// tiles.  Both operands go straight into the matrix cores' registers.
//
// With few rows nothing but the weight's bytes counts, and the time of a call
// that moves 25 MB is latency, as it is with few tiles: so a workgroup takes 16 NA
// rows of the weight and 16 MF rows of x, and its 8 waves share k, every wave with
// its first loads on their way before it does anything else.
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 16 weight rows (its A operand) and 16 rows
// of x (B) over 128 values; in the blocked layout a lane's 16 bytes of either lie in
// runs of 256 bytes.  The waves' sums meet in LDS, in a fixed order.  No barrier and
// no LDS before that: next to the tiles of mx4_gemm.hip a call starts and ends 2 us
// sooner (333 x 2112 -> 1040 4.3 us in 32 x 32 pieces, 6.8 on a 64 x 128 tile of
// that kernel), but its smaller pieces read the operands more often, and 4 x 4
// fragments are as many as the registers hold (256 x 4096 -> 4096 7.0 us, 8.9).
//
// FUSED: while the weight's loads are in flight the workgroup quantizes the rows
// of x itself, into LDS, so the call is one launch; every workgroup repeats that,
// so only while it is one block of 32 values a thread (rows * k <= 16384): one token
// 4096 -> 12288, 26.7 MB of weight, 7.0 us (16 tokens, quantized before: 4.2 + 6.8).
#include "ck_internal.hpp"
#include "mx4.hpp"

namespace ck {
namespace mx4 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kFusedValues = 32 * kThreads;   // of x: one block of 32 a thread

struct FewArgs {
    const uint8_t *xc, *xs;     // blocked codes and scales of x, or
    const uint16_t* x;          // (FUSED) its BF16 rows
    int64_t ldx;
    const uint8_t *wc, *ws;
    uint16_t* y;
    EpiExtra ex;
    int M, N, k, log_g;
    int pairs;                  // kp / 256
    int units, m_tiles;         // of 16 NA weight rows, of 16 MF rows of x
    int xb, wb;                 // 32-row blocks
};

template <int T>
__device__ __forceinline__ v4f product16(v4i a, v4i b, v4f c, int sa, int sb)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                            v8i{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, 2 * T, sa,
                                                            2 * T, sb);
}

__device__ __forceinline__ uint4 quantize32_by(int log_g, float (&v)[4][8], int lane, uint32_t* byte)
{
    switch (log_g) {   // uniform
        case 0: return quantize32<0>(v, lane, byte);
        case 1: return quantize32<1>(v, lane, byte);
        case 2: return quantize32<2>(v, lane, byte);
        case 3: return quantize32<3>(v, lane, byte);
        case 4: return quantize32<4>(v, lane, byte);
        case 5: return quantize32<5>(v, lane, byte);
        case 6: return quantize32<6>(v, lane, byte);
        case 7: return quantize32<7>(v, lane, byte);
        default: return quantize32<8>(v, lane, byte);
    }
}

// NA x MF fragments of 16 x 16 a workgroup.  ACT (FUSED): 0 x, 1 silu(gate) * up.
// Two workgroups a CU (at most 128 registers), but for 4 x 4 fragments.  (With x from
// memory 2 x 1 fragments spill 12 registers there: 16 x 4096 -> 24576 10.2 us.)
template <int NA, int MF, bool FUSED, int ACT>
__global__ __launch_bounds__(kThreads, NA * MF > 4 ? 2 : 4) void mx4_few_kernel(FewArgs g)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int UB = (FUSED ? NA : NA + MF) <= 3 ? 2 : 1;   // pairs of a batch
    constexpr int F = NA * MF;
    constexpr int CODES = FUSED ? kFusedValues / 2 : 0, SCALES = FUSED ? kFusedValues / 32 : 0;
    constexpr int RED = kWaves * F * 1024;
    __shared__ __attribute__((aligned(16))) char smem[RED > CODES + SCALES ? RED : CODES + SCALES];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // One XCD (workgroup % 8) takes consecutive tiles, and a unit's lie together, so
    // that its L2 holds the unit's weight rows.
    const int each = gridDim.x >> 3, tile = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
    const int unit = tile / g.m_tiles;
    if (unit >= g.units) return;
    const int row0 = (tile - unit * g.m_tiles) * (16 * MF);   // of x
    const int r = lane & 15, kg = lane >> 4;
    const int kb = 4 * g.pairs;

    // this lane's first bytes of each fragment's rows: codes of 128 values in two
    // blocks of 64, two halves each; scales in one register for 256 values
    auto codes_at = [&](int rb, int odd) {
        return (int64_t)rb * kb * 1024 + (kg >> 1) * 1024 + (kg & 1) * 512 + (odd * 16 + r) * 16;
    };
    auto scales_at = [&](int rb, int odd) { return (int64_t)rb * g.pairs * 256 + ((kg & 1) * 32 + odd * 16 + r) * 4; };
    const uint8_t *wc[NA], *ws[NA], *xc[MF], *xs[MF];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const int row16 = unit * NA + i, rb = min(row16 >> 1, g.wb - 1);   // past the end: rows that are not stored
        wc[i] = g.wc + codes_at(rb, row16 & 1);
        ws[i] = g.ws + scales_at(rb, row16 & 1);
    }
    if constexpr (!FUSED) {
#pragma unroll
        for (int j = 0; j < MF; ++j) {
            const int rb = min((row0 >> 5) + (j >> 1), g.xb - 1);
            xc[j] = g.xc + codes_at(rb, j & 1);
            xs[j] = g.xs + scales_at(rb, j & 1);
        }
    }
    v4i a[2][UB][2][NA], x[2][UB][2][MF];
    int sa[2][UB][NA], sx[2][UB][MF];
    // batch n of this wave: pairs wave + kWaves (UB n + u); past the last one nothing is loaded
    auto load = [&](int n, int side) {
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const int p = wave + kWaves * (UB * n + u);
            if (p >= g.pairs) break;
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                a[side][u][0][i] = *reinterpret_cast<const v4i*>(wc[i] + (int64_t)p * 4096);
                a[side][u][1][i] = *reinterpret_cast<const v4i*>(wc[i] + (int64_t)p * 4096 + 2048);
                sa[side][u][i] = *reinterpret_cast<const int*>(ws[i] + (int64_t)p * 256);
            }
            if constexpr (!FUSED) {
#pragma unroll
                for (int j = 0; j < MF; ++j) {
                    x[side][u][0][j] = *reinterpret_cast<const v4i*>(xc[j] + (int64_t)p * 4096);
                    x[side][u][1][j] = *reinterpret_cast<const v4i*>(xc[j] + (int64_t)p * 4096 + 2048);
                    sx[side][u][j] = *reinterpret_cast<const int*>(xs[j] + (int64_t)p * 256);
                }
            }
        }
    };

    float v[4][8];
    bool live = false;
    int row = 0, blk = 0;
    const int blocks = g.k >> 5;          // of a row
    if constexpr (FUSED) {
        // x first (the quantizer waits for it), then the weight
        const int per = (blocks + 7) & ~7;   // teams of 8 lanes hold 256 values of one row
        row = tid / per, blk = tid - row * per;
        live = row < g.M && blk < blocks;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
        if (live) load32<ACT>(g.x, row * g.ldx + blk * 32, g.k, v);
    }
    load(0, 0);
    if constexpr (FUSED) {
        uint32_t byte;
        const uint4 q = quantize32_by(g.log_g, v, lane, &byte);
        if (live) {
            *reinterpret_cast<uint4*>(smem + (row * blocks + blk) * 16) = q;
            smem[CODES + row * blocks + blk] = (char)byte;
        }
        __syncthreads();
    }

    v4f acc[NA][MF];
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < MF; ++j) acc[i][j] = v4f{};
    auto compute = [&](int n, int side) {
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const int p = wave + kWaves * (UB * n + u);
            if (p >= g.pairs) break;
            int ta[NA], tx[MF];
            v4i bx[2][MF];
#pragma unroll
            for (int i = 0; i < NA; ++i) ta[i] = (int)((uint32_t)sa[side][u][i] >> (8 * (kg >> 1)));
#pragma unroll
            for (int j = 0; j < MF; ++j) {
                if constexpr (FUSED) {
                    // rows past M and blocks past k: zero codes
                    uint32_t s[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int b = p * 8 + 4 * t + kg;
                        const bool ok = r < g.M && b < blocks;
                        const int place = ok ? r * blocks + b : 0;
                        const v4i c = *reinterpret_cast<const v4i*>(smem + place * 16);
                        const uint32_t e = (uint8_t)smem[CODES + place];
                        bx[t][j] = ok ? c : v4i{};
                        s[t] = ok ? e : 127u;
                    }
                    tx[j] = (int)(s[0] | s[1] << 16);
                } else {
                    bx[0][j] = x[side][u][0][j];
                    bx[1][j] = x[side][u][1][j];
                    tx[j] = (int)((uint32_t)sx[side][u][j] >> (8 * (kg >> 1)));
                }
            }
#pragma unroll
            for (int i = 0; i < NA; ++i)
#pragma unroll
                for (int j = 0; j < MF; ++j) {
                    acc[i][j] = product16<0>(a[side][u][0][i], bx[0][j], acc[i][j], ta[i], tx[j]);
                    acc[i][j] = product16<1>(a[side][u][1][i], bx[1][j], acc[i][j], ta[i], tx[j]);
                }
        }
    };
    const int batches = (g.pairs - wave + kWaves * UB - 1) / (kWaves * UB);
    for (int n = 0; n < batches; n += 2) {
        load(n + 1, 1);
        compute(n, 0);
        load(n + 2, 0);
        compute(n + 1, 1);
    }

    // the waves' sums, in order: D holds column l % 16 (row m of x) and rows 4 (l / 16) + 0..3 (n)
    if constexpr (FUSED) __syncthreads();   // the codes are read no more
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < MF; ++j)
            *reinterpret_cast<v4f*>(smem + ((wave * F + i * MF + j) * 64 + lane) * 16) = acc[i][j];
    __syncthreads();
    for (int t = tid; t < F * 64; t += kThreads) {
        const int f = t >> 6, l = t & 63;
        const int m = row0 + (f % MF) * 16 + (l & 15), n = (unit * NA + f / MF) * 16 + 4 * (l >> 4);
        if (m >= g.M || n >= g.N) continue;
        v4f s = *reinterpret_cast<const v4f*>(smem + t * 16);
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s = s + *reinterpret_cast<const v4f*>(smem + (w * F * 64 + t) * 16);
        float y0 = s[0], y1 = s[1], y2 = s[2], y3 = s[3];
        epi_extra4(y0, y1, y2, y3, g.ex, m, n, g.N);
        *reinterpret_cast<uint2*>(g.y + (int64_t)m * g.N + n) = make_uint2(pack_bf16x2(y0, y1), pack_bf16x2(y2, y3));
    }
#endif  // __HIP_DEVICE_COMPILE__
}

template <int NA, int MF, bool FUSED, int ACT>
hipError_t launch_few(FewArgs g, hipStream_t st)
{
    g.units = (g.N + 16 * NA - 1) / (16 * NA);
    g.m_tiles = (g.M + 16 * MF - 1) / (16 * MF);
    const dim3 grid((g.units * g.m_tiles + 7) / 8 * 8);
    mx4_few_kernel<NA, MF, FUSED, ACT><<<grid, dim3(kThreads), 0, st>>>(g);
    return hipGetLastError();
}

}  // namespace mx4

// rows: of x a workgroup, 16, 32 or 64.
hipError_t launch_mx4_few(const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* ws, int64_t m, int64_t n,
                          int64_t k, int rows, uint16_t* y, EpiExtra ex, hipStream_t st)
{
    mx4::FewArgs g{};
    g.xc = xc, g.xs = xs, g.wc = wc, g.ws = ws, g.y = y, g.ex = ex;
    g.M = (int)m, g.N = (int)n, g.k = (int)k, g.pairs = (int)(mx4::pad_cols(k) / 256);
    g.xb = (int)(mx4::pad_rows(m) / 32), g.wb = (int)(mx4::pad_rows(n) / 32);
    if (rows == 64) return mx4::launch_few<4, 4, false, 0>(g, st);
    if (rows == 32) return mx4::launch_few<2, 2, false, 0>(g, st);
    // 32 rows of the weight a workgroup where they still give every CU one
    return n >= 32 * num_cus() ? mx4::launch_few<2, 1, false, 0>(g, st) : mx4::launch_few<1, 1, false, 0>(g, st);
}

bool mx4_fused(int64_t m, int64_t k)
{
    return m <= 16 && m * ((k + 255) / 256 * 256) <= mx4::kFusedValues;
}

hipError_t launch_mx4_fused(int act, const uint16_t* x, int64_t ldx, const uint8_t* wc, const uint8_t* ws, int64_t m,
                            int64_t n, int64_t k, int g_size, uint16_t* y, EpiExtra ex, hipStream_t st)
{
    mx4::FewArgs g{};
    g.x = x, g.ldx = ldx, g.wc = wc, g.ws = ws, g.y = y, g.ex = ex;
    g.M = (int)m, g.N = (int)n, g.k = (int)k, g.pairs = (int)(mx4::pad_cols(k) / 256);
    g.wb = (int)(mx4::pad_rows(n) / 32);
    while ((1 << g.log_g) < g_size) ++g.log_g;
    if (n >= 32 * num_cus())
        return act ? mx4::launch_few<2, 1, true, 1>(g, st) : mx4::launch_few<2, 1, true, 0>(g, st);
    return act ? mx4::launch_few<1, 1, true, 1>(g, st) : mx4::launch_few<1, 1, true, 0>(g, st);
}

}  // namespace ck
