// qknorm.hip -- the RMS norm of query and key heads with the position rotation
// in the same pass (include/ck.h, ck_qk_norm_rope).
//
// For one token and head, x of d channels:
//   z_i = x_i * rsqrt(sum_i x_i^2 / d + eps) * w_i
//   (y_a, y_b) = (z_a cos - z_b sin, z_b cos + z_a sin)   for each pair (a, b)
// in FP32 with one rounding at the end (a rounding between the norm and the
// rotation would double the output's error for nothing: both are in registers).
//
// The kernel is bound by HBM: 2 bytes read and 2 written per element, about 10
// VALU operations (4 x 16384 tokens of 32 + 8 heads of 128, 1.34 GB: 226 us, 5.9
// TB/s; 16 tokens of those: 3.0 to 3.4 us).  Layout: a team of 8, 16 or 32 lanes holds one head (8
// channels, one 16-byte load, per lane), so a wave's load covers consecutive
// heads of a token, whole cache lines.  A team takes up to U heads of one
// token: the norm weights and the token's cos / sin values are read once for
// all of them (as 32-bit tables they are four times a head's own bytes with the
// half pairing), and all U loads are in flight before the first is used.
#include "ck_internal.hpp"
#include "heads.hpp"
#include "qk_lanes.hpp"

namespace ck {
namespace qkn {

// One side (the queries or the keys) of a call.  Strides in elements.
struct Side {
    const uint16_t* x;
    uint16_t* y;
    const float* w;
    const float* cos;
    const float* sin;
    const int32_t* pos;
    int64_t x_sb, x_st, x_sh, y_sb, y_st, y_sh, pos_sb;
    uint32_t items;      // (token, head group) teams: batch * tokens * hg
    uint32_t heads, hg;  // head h = u * hg + (item % hg), u < U
    uint32_t table;      // rows of cos and sin
    FastDiv by_hg, by_tokens;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool NT>
__device__ __forceinline__ uint4 load16(const uint16_t* p)
{
    if constexpr (NT) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
    return *reinterpret_cast<const uint4*>(p);
}
template <bool NT>
__device__ __forceinline__ void store16(uint16_t* p, uint4 v)
{
    if constexpr (NT)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(p));
    else
        *reinterpret_cast<uint4*>(p) = v;
}

template <int TEAM>
__device__ __forceinline__ float team_sum(float v)
{
    v = v + dpp_xor<1>(v);
    v = v + dpp_xor<2>(v);
    v = v + swizzle_xor<4>(v);
    if constexpr (TEAM >= 16) v = v + swizzle_xor<8>(v);
    if constexpr (TEAM >= 32) v = v + swizzle_xor<16>(v);
    return v;
}

// NT: nontemporal loads and stores of the heads, for calls past the Infinity
// Cache.  Measured with / without: 4 x 16384 tokens of 32 + 8 heads of 128 (1.3
// GB) 230 / 257 us, 16384 tokens of 24 + 24 heads 68 / 79 us; 4096 tokens of
// those (101 MB) 20.4 / 19.6 us.
template <typename T, int TEAM, bool HALF, int U, bool NT>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(Side sq, Side sk, uint32_t q_blocks, uint32_t d,
                                                           uint32_t rot, float eps)
{
    const bool is_k = blockIdx.x >= q_blocks;   // workgroup-uniform
    const Side& s = is_k ? sk : sq;
    const uint32_t block = blockIdx.x - (is_k ? q_blocks : 0u);
    const uint32_t lane = threadIdx.x & (TEAM - 1);
    const uint32_t item = block * (256u / TEAM) + threadIdx.x / TEAM;
    // lanes with nothing to do stay for the exchanges between lanes below
    const Lane ln = lane_of(lane, d, rot, HALF);
    const bool live = item < s.items && ln.live;
    const uint32_t it = item < s.items ? item : 0u;
    const uint32_t bt = s.by_hg.div(it);
    const uint32_t h0 = it - bt * s.hg;
    const uint32_t b = s.by_tokens.div(bt);
    const uint32_t t = bt - b * s.by_tokens.d;
    const uint32_t c = ln.c;   // first channel of this lane

    const uint16_t* x = s.x + (int64_t)b * s.x_sb + (int64_t)t * s.x_st + c;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t h = u * s.hg + h0;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (live && h < s.heads) raw[u] = load16<NT>(x + (int64_t)h * s.x_sh);
    }

    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    if (s.w) {
        *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(s.w + c);
        *reinterpret_cast<float4*>(w + 4) = *reinterpret_cast<const float4*>(s.w + c + 4);
    }

    // The rotation as y = z * cs + partner * sn.  interleaved: 4 pairs in the
    // lane; half: the partner of channel c + i is rot / 2 channels away, in
    // lane + or - rot / 16 of the team.  Channels past rot skip it (times 1 plus
    // their neighbour times 0 would spread an infinity).
    const bool rope = s.cos != nullptr;   // workgroup-uniform
    const bool turns = rope && ln.turns;
    float cs[HALF ? 8 : 4], sn[HALF ? 8 : 4], pw[8];
    float bad = 0.0f;
    if (rope) {
        uint32_t p = t;
        if (s.pos) {   // a position outside the table writes NaN, and reads row 0
            p = (uint32_t)s.pos[(int64_t)b * s.pos_sb + t];
            if (p >= s.table) {
                p = 0;
                bad = __uint_as_float(0x7fc00000u);
            }
        }
        const int64_t at = (int64_t)p * (rot / 2) + ln.table;
        if constexpr (HALF) {
            if (turns) {
                const float* ct = s.cos + at;
                const float* st = s.sin + at;
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    *reinterpret_cast<float4*>(cs + i) = *reinterpret_cast<const float4*>(ct + i);
                    *reinterpret_cast<float4*>(sn + i) = *reinterpret_cast<const float4*>(st + i);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) pw[i] = ln.upper ? 1.0f : -1.0f;
            if (s.w) {
                const float* ow = s.w + ln.other_c;
#pragma unroll
                for (int i = 0; i < 8; ++i) pw[i] = pw[i] * ow[i];
            }
        } else if (turns) {
            *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(s.cos + at);
            *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(s.sin + at);
        }
    }

    uint16_t* y = s.y + (int64_t)b * s.y_sb + (int64_t)t * s.y_st + c;
    const float inv_d = 1.0f / (float)d;
    // the partner lane's address for the exchange (a byte address in the wave)
    const int from = (int)(((threadIdx.x & 63u) - lane + ln.other) * 4u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t h = u * s.hg + h0;
        float v[8];
        unpack8<T>(raw[u], v);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
        const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(team_sum<TEAM>(ss), inv_d, eps)) + bad;
        float o[8];
        if constexpr (HALF) {
            float pv[8];
            if (rope) {   // the partner's channels, still as 16-bit values: 4 exchanges, not 8
                uint4 pr;
                pr.x = __builtin_amdgcn_ds_bpermute(from, raw[u].x);
                pr.y = __builtin_amdgcn_ds_bpermute(from, raw[u].y);
                pr.z = __builtin_amdgcn_ds_bpermute(from, raw[u].z);
                pr.w = __builtin_amdgcn_ds_bpermute(from, raw[u].w);
                unpack8<T>(pr, pv);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = v[i] * r * w[i];
                if (turns) o[i] = __builtin_fmaf(pv[i] * r * pw[i], sn[i], o[i] * cs[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = v[i] * r * w[i];
            if (turns) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = o[2 * i], z = o[2 * i + 1];
                    o[2 * i] = __builtin_fmaf(-z, sn[i], a * cs[i]);
                    o[2 * i + 1] = __builtin_fmaf(a, sn[i], z * cs[i]);
                }
            }
        }
        if (live && h < s.heads) store16<NT>(y + (int64_t)h * s.y_sh, pack8<T>(o));
    }
}

}  // namespace qkn

namespace {

qkn::Side make_side(const QkSideArgs& a, int u)
{
    qkn::Side s{};
    s.x = a.x;
    s.y = a.y;
    s.w = a.w;
    s.cos = a.cos;
    s.sin = a.sin;
    s.pos = a.pos;
    s.x_sb = a.x_sb, s.x_st = a.x_st, s.x_sh = a.x_sh;
    s.y_sb = a.y_sb, s.y_st = a.y_st, s.y_sh = a.y_sh;
    s.pos_sb = a.pos_sb;
    s.heads = (uint32_t)a.heads;
    s.hg = (uint32_t)((a.heads + u - 1) / u);
    s.items = (uint32_t)(a.batch * a.tokens * s.hg);
    s.table = (uint32_t)a.table;
    s.by_hg = FastDiv(s.hg ? s.hg : 1);
    s.by_tokens = FastDiv((uint32_t)(a.tokens ? a.tokens : 1));
    return s;
}

template <typename T, int TEAM, bool HALF, int U, bool NT>
hipError_t launch(const QkSideArgs& q, const QkSideArgs& k, int64_t d, int64_t rot, float eps, hipStream_t st)
{
    constexpr uint32_t per_block = 256 / TEAM;
    const qkn::Side sq = make_side(q, U), sk = make_side(k, U);
    const uint32_t qb = (sq.items + per_block - 1) / per_block, kb = (sk.items + per_block - 1) / per_block;
    if (qb + kb == 0) return hipSuccess;
    qkn::qk_norm_rope_kernel<T, TEAM, HALF, U, NT>
        <<<dim3(qb + kb), dim3(256), 0, st>>>(sq, sk, qb, (uint32_t)d, (uint32_t)rot, eps);
    return hipGetLastError();
}

template <typename T, int TEAM, bool HALF>
hipError_t pick_u(const QkSideArgs& q, const QkSideArgs& k, int64_t d, int64_t rot, float eps, hipStream_t st)
{
    const int64_t rows = q.batch * q.tokens * q.heads + k.batch * k.tokens * k.heads;
    // U heads a team once that still gives every CU 8 waves (4096 tokens of 24 + 24
    // heads of 128: 19.6 us, one head a team 22.0; 512 tokens of 32 + 8: 5.0 and
    // 4.8; 16 tokens: 3.8 and 3.0)
    if (rows * TEAM < 4 * 64 * 8 * (int64_t)num_cus()) return launch<T, TEAM, HALF, 1, false>(q, k, d, rot, eps, st);
    if (rows * d * 4 < kInfinityCacheBytes) return launch<T, TEAM, HALF, 4, false>(q, k, d, rot, eps, st);
    return launch<T, TEAM, HALF, 4, true>(q, k, d, rot, eps, st);
}

template <typename T>
hipError_t pick(const QkSideArgs& q, const QkSideArgs& k, int64_t d, int64_t rot, bool half, float eps,
                hipStream_t st)
{
    if (d <= 64)
        return half ? pick_u<T, 8, true>(q, k, d, rot, eps, st) : pick_u<T, 8, false>(q, k, d, rot, eps, st);
    if (d <= 128)
        return half ? pick_u<T, 16, true>(q, k, d, rot, eps, st) : pick_u<T, 16, false>(q, k, d, rot, eps, st);
    return half ? pick_u<T, 32, true>(q, k, d, rot, eps, st) : pick_u<T, 32, false>(q, k, d, rot, eps, st);
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkSideArgs& q, const QkSideArgs& k, int64_t d, int64_t rot, bool half,
                               bool fp16, float eps, hipStream_t st)
{
    return fp16 ? pick<f16>(q, k, d, rot, half, eps, st) : pick<bf16>(q, k, d, rot, half, eps, st);
}

}  // namespace ck
