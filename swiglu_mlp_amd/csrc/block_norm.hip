// block_norm.hip -- what joins two sub-blocks of a transformer block in one
// pass (include/ck.h, ck_block_norm):
//   r = residual_scale x + branch_scale gate N_b(branch)      -> x_out
//   h = N(r) (1 + scale) + shift                              -> out
// N_b and N an RMS norm (v rsqrt(mean v^2 + eps) w), a layer norm ((v - mean)
// rsqrt(mean (v - mean)^2 + eps) w + b) or nothing.
//
// A row lives in registers between its loads and its stores, so x and branch are
// read once and r and h written once: 8 bytes a value, which is what bounds it.
// All steps are FP32 and h is computed from the unrounded r; the variance is that
// of the centred values (a second sum over registers), not a difference of sums.
//
// 65536 rows of 4096 with two RMS norms, 2.1 GB: 387 us (5.5 TB/s); 8192 rows with
// three modulations a sequence, 268 MB, 51 us (5.3); 16 rows 2.7 to 4 us, a launch.
#include "ck_internal.hpp"
#include "heads.hpp"

namespace ck {
namespace bnorm {

// A modulation: 16-bit or FP32 values [batch, tokens, width], null for none.
struct Mod {
    const void* p;
    int64_t sb, st;
};

struct Params {
    const uint16_t* x;
    const uint16_t* branch;
    uint16_t* x_out;
    uint16_t* out;
    int64_t x_sb, x_st, b_sb, b_st, xo_sb, xo_st, o_sb, o_st;
    uint32_t rows, width;
    FastDiv by_tokens;
    Mod gate, scale, shift;
    const float *bw, *bb, *w, *b;   // branch norm's and norm's weight and bias
    int branch_kind, kind;          // CK_NORM_*
    bool mod32;
    float residual_scale, branch_scale, eps, inv_width;
};

template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* lds, int slot)
{
    v = v + dpp_xor<1>(v);
    v = v + dpp_xor<2>(v);
    v = v + swizzle_xor<4>(v);
    v = v + swizzle_xor<8>(v);
    v = v + swizzle_xor<16>(v);
    v = v + __shfl_xor(v, 32, 64);
    if constexpr (TEAM > 64) {
        constexpr int WAVES = TEAM / 64;
        float* p = lds + slot * WAVES;   // a slot for each sum of a row: no second barrier
        if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
        __syncthreads();
        v = p[0];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) v = v + p[i];
    }
    return v;
}

__device__ __forceinline__ void load_f32(const float* p, float (&v)[8])
{
    *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p);
    *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(p + 4);
}

// A modulation's values of each chunk.  16-bit ones of short rows (U <= 2) are
// loaded with the row itself (begin), all others where they are used: FP32 ones
// and long rows would cost registers, and waves in flight with them.
template <typename T, int U>
struct ModValues {
    static constexpr bool kEarly = U <= 2;
    uint4 raw[kEarly ? U : 1];

    __device__ __forceinline__ static int64_t at(const Mod& m, int64_t b, int64_t t) { return b * m.sb + t * m.st; }
    __device__ __forceinline__ void begin(const Mod& m, bool f32, int64_t b, int64_t t, const uint32_t (&c)[U])
    {
        if constexpr (kEarly) {
            if (m.p && !f32) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    raw[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(m.p) + at(m, b, t) + c[u]);
            }
        }
    }
    __device__ __forceinline__ void get(const Mod& m, bool f32, int64_t b, int64_t t, int u, uint32_t c, float (&v)[8]) const
    {
        if (f32)
            load_f32(static_cast<const float*>(m.p) + at(m, b, t) + c, v);
        else if constexpr (kEarly)
            unpack8<T>(raw[u], v);
        else
            unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(m.p) + at(m, b, t) + c), v);
    }
};

// v -> N(v) over the row; dead chunks hold zeros and stay zeros in the sums.
template <int TEAM, int U>
__device__ __forceinline__ void normalise(float (&v)[U][8], const bool (&live)[U], const uint32_t (&c)[U], int kind,
                                          const float* w, const float* b, const Params& p, float* lds, int slot)
{
    if (kind == 0) return;
    constexpr bool kEarly = U <= 2;   // weights on their way during the sums, where registers allow it
    float g[kEarly ? U : 1][8], o[kEarly ? U : 1][8];
    if constexpr (kEarly) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (w) load_f32(w + c[u], g[u]);
            if (b) load_f32(b + c[u], o[u]);
        }
    }
    if (kind == 2) {
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) s = s + v[u][i];
        const float mean = team_sum<TEAM>(s, lds, slot) * p.inv_width;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = live[u] ? v[u][i] - mean : 0.0f;
    }
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[u][i], v[u][i], ss);
    const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(team_sum<TEAM>(ss, lds, slot + 1), p.inv_width, p.eps));
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = kEarly ? u : 0;
        if constexpr (!kEarly) {
            if (w) load_f32(w + c[u], g[0]);
            if (b) load_f32(b + c[u], o[0]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[u][i] = v[u][i] * r;
            if (w) v[u][i] = v[u][i] * g[at][i];
            if (b) v[u][i] = v[u][i] + o[at][i];
        }
    }
}

// TEAM threads a row (a wave, or the workgroup), U chunks of 8 values a thread.
// NT: nontemporal loads and stores of the rows.
template <typename T, int TEAM, int U, bool NT>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void block_norm_kernel(Params p)
{
    constexpr int THREADS = TEAM < 256 ? 256 : TEAM;
    __shared__ float lds[TEAM > 64 ? 4 * (TEAM / 64) : 1];
    const uint32_t row = blockIdx.x * (THREADS / TEAM) + threadIdx.x / TEAM;
    if (row >= p.rows) return;   // whole waves: a workgroup of one row has none of these
    const uint32_t lane = threadIdx.x & (TEAM - 1);
    const uint32_t bi = p.by_tokens.div(row);
    const int64_t b = bi, t = row - bi * p.by_tokens.d;

    bool live[U];
    uint32_t c[U];
    uint4 rx[U], rb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t at = (u * TEAM + lane) * 8;
        live[u] = at < p.width;
        c[u] = live[u] ? at : 0;
        rx[u] = rb[u] = make_uint4(0, 0, 0, 0);
        if (live[u]) {
            rx[u] = load16<NT>(p.x + b * p.x_sb + t * p.x_st + at);
            if (p.branch) rb[u] = load16<NT>(p.branch + b * p.b_sb + t * p.b_st + at);
        }
    }
    ModValues<T, U> gate, scale, shift;
    gate.begin(p.gate, p.mod32, b, t, c);
    scale.begin(p.scale, p.mod32, b, t, c);
    shift.begin(p.shift, p.mod32, b, t, c);
    float v[U][8];
    if (p.branch) {
#pragma unroll
        for (int u = 0; u < U; ++u) unpack8<T>(rb[u], v[u]);
        normalise<TEAM, U>(v, live, c, p.branch_kind, p.bw, p.bb, p, lds, 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float g[8], x[8];
            unpack8<T>(rx[u], x);
            if (p.gate.p) {
                gate.get(p.gate, p.mod32, b, t, u, c[u], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] * g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[u][i] = __builtin_fmaf(p.branch_scale, v[u][i], p.residual_scale * x[i]);
                if (!live[u]) v[u][i] = 0.0f;
            }
            if (p.x_out && live[u]) store16<NT>(p.x_out + b * p.xo_sb + t * p.xo_st + c[u], pack8<T>(v[u]));
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            unpack8<T>(rx[u], v[u]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] * p.residual_scale;
        }
    }
    if (!p.out) return;
    normalise<TEAM, U>(v, live, c, p.kind, p.w, p.b, p, lds, 2);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float g[8];
        if (p.scale.p) {
            scale.get(p.scale, p.mod32, b, t, u, c[u], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = __builtin_fmaf(v[u][i], g[i], v[u][i]);
        }
        if (p.shift.p) {
            shift.get(p.shift, p.mod32, b, t, u, c[u], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] + g[i];
        }
        if (live[u]) store16<NT>(p.out + b * p.o_sb + t * p.o_st + c[u], pack8<T>(v[u]));
    }
}

}  // namespace bnorm

namespace {

template <typename T, int TEAM, int U, bool NT>
hipError_t launch(const bnorm::Params& p, hipStream_t st)
{
    constexpr uint32_t nt = TEAM < 256 ? 256 : TEAM, per = nt / TEAM;
    bnorm::block_norm_kernel<T, TEAM, U, NT><<<dim3((p.rows + per - 1) / per), dim3(nt), 0, st>>>(p);
    return hipGetLastError();
}

// A workgroup a row, so that the row's bytes are in flight at once from many lanes;
// a wave a row (no barriers between the sums, less to wait for) where many rows are
// narrow.  Measured, wave and workgroup: 16384 rows of 1160 39 and 43 us, 4096 of
// them 11.4 and 12.2, 1024 5.8 and 5.9, 16 4.9 and 3.7; 16384 rows of 2048 51 and 46;
// 4096 rows of 4096 34 and 28 (248 registers a lane).  Past 8192 channels a workgroup
// needs 255 or 256 registers a lane, and a SIMD holds two waves (FP16) or one (BF16):
// 16384 rows of 12288 380 us (4.2 TB/s) and 505 (3.2), of 16384 475 (4.5) and 638
// (3.4), where rows of 8192 take 195 and 201 (5.4).
template <typename T, bool NT>
hipError_t pick_team(const bnorm::Params& p, hipStream_t st)
{
    if (p.width <= 512) return launch<T, 64, 1, NT>(p, st);
    if (p.width <= 1536 && p.rows >= 16u * (uint32_t)num_cus())
        return p.width <= 1024 ? launch<T, 64, 2, NT>(p, st) : launch<T, 64, 3, NT>(p, st);
    if (p.width <= 2048) return launch<T, 256, 1, NT>(p, st);
    if (p.width <= 4096) return launch<T, 256, 2, NT>(p, st);
    if (p.width <= 8192) return launch<T, 256, 4, NT>(p, st);
    return launch<T, 256, 8, NT>(p, st);
}

// Rows past the Infinity Cache go by nontemporal loads and stores: 65536 rows of
// 4096 387 us for 403, 32768 of 8192 388 for 405; 4096 of 4096 (134 MB) 29 for 28.
template <typename T>
hipError_t pick(const bnorm::Params& p, hipStream_t st)
{
    const int64_t bytes = (int64_t)p.rows * p.width * 8;
    return bytes < kInfinityCacheBytes ? pick_team<T, false>(p, st) : pick_team<T, true>(p, st);
}

bnorm::Mod mod_of(const ModArgs& m) { return bnorm::Mod{m.p, m.sb, m.st}; }

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t st)
{
    bnorm::Params p{};
    p.x = a.x, p.branch = a.branch, p.x_out = a.x_out, p.out = a.out;
    p.x_sb = a.x_sb, p.x_st = a.x_st, p.b_sb = a.b_sb, p.b_st = a.b_st;
    p.xo_sb = a.xo_sb, p.xo_st = a.xo_st, p.o_sb = a.o_sb, p.o_st = a.o_st;
    p.rows = (uint32_t)(a.batch * a.tokens), p.width = (uint32_t)a.width;
    p.by_tokens = FastDiv((uint32_t)a.tokens);
    p.gate = mod_of(a.gate), p.scale = mod_of(a.scale), p.shift = mod_of(a.shift);
    p.bw = a.bw, p.bb = a.bb, p.w = a.w, p.b = a.b;
    p.branch_kind = a.branch_kind, p.kind = a.kind, p.mod32 = a.mod32;
    p.residual_scale = a.residual_scale, p.branch_scale = a.branch_scale, p.eps = a.eps;
    p.inv_width = 1.0f / (float)a.width;
    return a.fp16 ? pick<f16>(p, st) : pick<bf16>(p, st);
}

}  // namespace ck
