// attn.hip -- attention of query rows over encoder keys and values of another
// length (include/ck.h, ck_cross_attn) on the 16-bit matrix cores of gfx950.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale (q_r . k_j) - m_r)
// over the allowed keys j, in one pass over the keys with the running maximum
// m_r and sum of the softmax in FP32.
//
// Rows.  All query rows that read the same keys (the sequences sharing one
// encoder sequence, their tokens, and the query heads of one key head) are one
// list of rows, so grouped heads and shared encoder states read K and V once.
//
// Tile.  A wave holds 32 rows and walks over tiles of 64 keys.  It computes
// S^T = K Q^T with v_mfma_f32_32x32x16 (K as the A operand): a lane then holds
// 32 scores of ONE row (lane % 32), so the row maximum is an in-lane maximum
// and one exchange with lane ^ 32, and the rescale factor is one register.
// The accumulator's key order, (i % 4) + 8 (i / 4) + 4 (lane / 32), is used as
// it is for the B operand P^T of O^T = V^T P^T: the products of a 16-key step
// may be taken in any key order that both operands share, so lane half h takes
// keys 4 h .. 4 h + 3 and 8 + 4 h .. 8 + 4 h + 3, and P never leaves its
// registers.  V^T in that order comes from row-major V in LDS by transposing
// reads (ds_read_b64_tr_b16: four keys of one channel per lane).
//
// K and V tiles go from HBM straight to LDS (buffer_load ... lds, 16 bytes a
// lane), double buffered: tile t + 1 loads while tile t is computed, with one
// barrier a tile.  A lane may choose its source but not its place, so the
// 16-byte chunks of a row are permuted on the source side (k_swz, v_swz) such
// that the reads of both operands touch every LDS bank once.
//
// Keys that are not allowed are never read: their lanes load from past the
// buffer, which gives zeros, so infinities and NaN there cannot reach a
// product, and their scores are set to -inf.
#include "ck_internal.hpp"
#include "heads.hpp"

namespace ck {
namespace attn {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;   // keys per tile

struct Params {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* o;
    int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh, v_sb, v_st, v_sh, o_sb, o_st, o_sh;
    const int32_t* kv_len;
    const uint8_t* mask;
    int64_t mask_sb;
    uint32_t tk, d, share, heads_kv, rows, m_tiles;
    float c;                        // scale * log2(e)
    FastDiv by_g, by_tq, by_hkv, by_tiles;
};

#if defined(__HIP_DEVICE_COMPILE__)

__device__ __forceinline__ void wait_vm0() { __builtin_amdgcn_s_waitcnt(0x0F70); }   // vmcnt(0) only

// s_barrier without a fence; the empty asm statements keep memory accesses on
// their side of it.
__device__ __forceinline__ void workgroup_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 16 bytes per lane from a buffer to LDS: lane l's land at byte lds + 16 l.
// Inline assembly, so that the compiler does not wait for it before unrelated
// LDS reads; the caller waits (wait_vm0) before the data's first use.
__device__ __forceinline__ void lds_dma_b128(v4i rsrc, uint32_t voff, uint32_t lds)
{
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, 0 offen lds"
        :
        : "v"(voff), "s"(rsrc), "s"(lds)
        : "memory");
}

__device__ __forceinline__ v4i make_rsrc(const void* base)
{
    const uint64_t a = (uint64_t)base;
    return v4i{(int)(uint32_t)a, (int)(uint32_t)((a >> 32) & 0xffffu), 0x7fffffff, 0x00020000};
}

// Place of 16-byte chunk c of row r inside the row, for the K tile (read as 16
// rows of one chunk at a time) and the V tile (read as 4 rows x 64 bytes).
// CH chunks a row; a row pitch of 16 CH bytes already spreads rows over the
// banks for CH = 12, half for CH = 8 and not at all for CH = 16.
template <int CH>
__device__ __forceinline__ uint32_t k_swz(uint32_t r, uint32_t c)
{
    if constexpr (CH == 16) return c ^ (r & 15u);
    if constexpr (CH == 8) return c ^ ((r >> 1) & 7u);
    return c ^ ((r >> 2) & 3u);
}
template <int CH>
__device__ __forceinline__ uint32_t v_swz(uint32_t r, uint32_t c)
{
    if constexpr (CH == 16) return c ^ ((r & 3u) << 2);
    if constexpr (CH == 8) return c ^ (((r >> 1) & 1u) << 2);
    return c;
}

template <typename T>
__device__ __forceinline__ v16f mfma(v4u a, v4u b, v16f c)
{
    if constexpr (__is_same(T, f16))
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c,
                                                       0, 0, 0);
}

// The value of lane ^ 32 combined with the lane's own.
__device__ __forceinline__ float half_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

#endif

// DP: channels padded to 64, 96 or 128 (the chunks past d load zeros).
// NW: waves per workgroup, 32 rows each.
template <typename T, int DP, int NW>
__global__ __launch_bounds__(NW * 64, 2) void tile_kernel(Params p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int CH = DP / 8;                       // 16-byte chunks per row
    constexpr int TILE_B = kTile * DP * 2;           // bytes of one K or V tile
    constexpr int NI = TILE_B / 1024;                // loads (1 KB) per K or V tile
    constexpr int PER = 2 * NI / NW;                 // ... of the pair, per wave
    static_assert(2 * NI % NW == 0, "loads split evenly over the waves");
    constexpr int KS = DP / 16;                      // 16-channel steps of S
    constexpr int DB = DP / 32;                      // 32-channel blocks of O
    // FP16 probabilities are scaled by 2^6, so small ones keep their bits: with
    // the deferred maximum below they reach at most 2^14.
    constexpr float kLift = __is_same(T, f16) ? 6.0f : 0.0f;
    constexpr float kDefer = 8.0f;
    __shared__ __attribute__((aligned(1024))) char smem[2 * 2 * TILE_B];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t half = lane >> 5, col = lane & 31;

    // workgroup -> (encoder sequence, key head, row tile)
    const uint32_t bh = p.by_tiles.div(blockIdx.x);
    const uint32_t mt = blockIdx.x - bh * p.m_tiles;
    const uint32_t eb = p.by_hkv.div(bh);
    const uint32_t hk = bh - eb * p.heads_kv;

    // this lane's row -> (sequence, token, head)
    const uint32_t row = (mt * NW + wave) * 32 + col;
    const uint32_t rr = row < p.rows ? row : p.rows - 1;
    const uint32_t rt = p.by_g.div(rr);
    const uint32_t head = hk * p.by_g.d + (rr - rt * p.by_g.d);
    const uint32_t si = p.by_tq.div(rt);
    const uint32_t tok = rt - si * p.by_tq.d;
    const int64_t seq = (int64_t)eb * p.share + si;

    v4u q[KS];
    {
        const uint16_t* qp = p.q + seq * p.q_sb + (int64_t)tok * p.q_st + (int64_t)head * p.q_sh;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const uint32_t c = 16 * s + 8 * half;
            q[s] = v4u{0, 0, 0, 0};
            if (c < p.d) q[s] = *reinterpret_cast<const v4u*>(qp + c);
        }
    }

    uint32_t len = p.tk;
    if (p.kv_len) {
        const int32_t l = p.kv_len[eb];
        len = l < 0 ? 0u : min((uint32_t)l, p.tk);
    }
    const uint32_t tiles = (len + kTile - 1) / kTile;
    const uint8_t* mask = p.mask ? p.mask + (int64_t)eb * p.mask_sb : nullptr;

    // this wave's loads: load j of the 2 NI (K's, then V's) fills bytes 1024 j .. of a buffer
    const char* k_base = reinterpret_cast<const char*>(p.k + (int64_t)eb * p.k_sb + (int64_t)hk * p.k_sh);
    const char* v_base = reinterpret_cast<const char*>(p.v + (int64_t)eb * p.v_sb + (int64_t)hk * p.v_sh);
    const uint32_t k_pitch = (uint32_t)(p.k_st * 2), v_pitch = (uint32_t)(p.v_st * 2);
    uint32_t src_row[PER], src_off[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = wave * PER + i;
        const bool is_v = j >= NI;
        const uint32_t slot = (uint32_t)(is_v ? j - NI : j) * 64 + lane;
        const uint32_t r = slot / CH, place = slot % CH;
        const uint32_t c = is_v ? v_swz<CH>(r, place) : k_swz<CH>(r, place);   // both are involutions
        src_row[i] = r;
        src_off[i] = 8 * c < p.d ? r * (is_v ? v_pitch : k_pitch) + 16 * c : kBufferOutside;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;

    auto tile_bits = [&](uint32_t t, uint32_t mbyte) -> uint64_t {   // allowed keys of tile t
        const uint32_t left = len - t * kTile;
        uint64_t bits = left >= 64 ? ~0ull : (1ull << left) - 1;
        if (mask) bits &= __ballot(mbyte != 0);
        return bits;
    };
    auto mask_byte = [&](uint32_t t) -> uint32_t {
        const uint32_t j = t * kTile + lane;
        return mask && j < len ? mask[j] : 0u;
    };
    auto load_tile = [&](uint32_t t, uint64_t bits) {
        const v4i rk = make_rsrc(k_base + (uint64_t)t * kTile * k_pitch);
        const v4i rv = make_rsrc(v_base + (uint64_t)t * kTile * v_pitch);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = wave * PER + i;
            uint32_t off = src_off[i];
            if (bits != ~0ull && !((bits >> src_row[i]) & 1)) off = kBufferOutside;
            lds_dma_b128(j >= NI ? rv : rk, off, lds0 + (t & 1) * 2 * TILE_B + j * 1024);
        }
    };

    v16f o[DB];
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;
    bool any = false;   // whether any key was allowed (the same for all rows)

    uint64_t bits = 0;
    uint32_t next_byte = 0;
    if (tiles) {
        bits = tile_bits(0, mask_byte(0));
        load_tile(0, bits);
        next_byte = mask_byte(1);
    }

    const uint32_t k_row = col * CH;                       // K fragment: row col (+ 32), chunk 2 s + half
    const uint32_t g16 = lane >> 4, j16 = lane & 15;       // V fragment: see the transposing read above
    const uint32_t v_key = 4 * (g16 >> 1) + (j16 >> 2);
    const uint32_t v_chunk = 2 * (g16 & 1) + ((j16 & 3) >> 1);

    for (uint32_t t = 0; t < tiles; ++t) {
        wait_vm0();
        workgroup_barrier();   // tile t is in LDS, and every wave is done with the other buffer
        uint64_t next_bits = 0;
        if (t + 1 < tiles) {
            next_bits = tile_bits(t + 1, next_byte);
            load_tile(t + 1, next_bits);
            if (t + 2 < tiles) next_byte = mask_byte(t + 2);
        }
        const char* kb = smem + (t & 1) * 2 * TILE_B;
        const char* vb = kb + TILE_B;

        v16f s[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[n][i] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint32_t at = (k_row + n * 32 * CH + k_swz<CH>(col, 2 * ks + half)) * 16;
                s[n] = mfma<T>(*reinterpret_cast<const v4u*>(kb + at), q[ks], s[n]);
            }
        }
        any |= bits != 0;
        if (bits != ~0ull) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint32_t w = (uint32_t)(bits >> (32 * n)) >> (4 * half);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!((w >> ((i & 3) + 8 * (i >> 2))) & 1u)) s[n][i] = -__builtin_inff();
            }
        }
        // The maximum in use may lag behind the true one by up to 2^kDefer in
        // the probabilities: FP32 sums and 16-bit floats lose nothing by it, and
        // most tiles skip the rescale of the accumulators.
        float mx = s[0][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[0][i]);
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[1][i]);
        mx = half_max(mx);
        if (__any((mx - m) * p.c > kDefer)) {
            const float mn = fmaxf(m, mx);
            const float alpha = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f((m - mn) * p.c);
            m = mn;
            l = l * alpha;
#pragma unroll
            for (int b = 0; b < DB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][i] *= alpha;
        }
        const float shift = (m == -__builtin_inff() ? 0.0f : -m * p.c) + kLift;
        v4u pf[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float e[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][i], p.c, shift));
            float sum[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = (e[i] + e[i + 4]) + (e[i + 8] + e[i + 12]);
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
            for (int g = 0; g < 2; ++g)
                pf[2 * n + g] = v4u{pack2<T>(e[8 * g], e[8 * g + 1]), pack2<T>(e[8 * g + 2], e[8 * g + 3]),
                                    pack2<T>(e[8 * g + 4], e[8 * g + 5]), pack2<T>(e[8 * g + 6], e[8 * g + 7])};
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
            for (int b = 0; b < DB; ++b) {
                typedef __attribute__((address_space(3))) v4s lds_v4s;
                const uint32_t at = ((v_key + 16 * g) * CH + v_swz<CH>(v_key, 4 * b + v_chunk)) * 16 + 8 * (j16 & 1);
                const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(vb + at));
                const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(vb + at + 8 * CH * 16));
                const v8s a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                o[b] = mfma<T>(__builtin_bit_cast(v4u, a), pf[g], o[b]);
            }
        }
        bits = next_bits;
    }

    // o[b][i] is channel 32 b + (i % 4) + 8 (i / 4) + 4 half of row col: pairs
    // of 4-channel groups are exchanged between the halves for 16-byte stores.
    const float total = half_sum(l);
    const float inv = any ? 1.0f / total : 0.0f;   // no allowed key: o is zero
    if (row < p.rows) {
        uint16_t* op = p.o + seq * p.o_sb + (int64_t)tok * p.o_st + (int64_t)head * p.o_sh;
#pragma unroll
        for (int b = 0; b < DB; ++b) {
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
                const uint32_t x0 = pack2<T>(o[b][i] * inv, o[b][i + 1] * inv);
                const uint32_t x1 = pack2<T>(o[b][i + 2] * inv, o[b][i + 3] * inv);
                const uint32_t y0 = pack2<T>(o[b][i + 4] * inv, o[b][i + 5] * inv);
                const uint32_t y1 = pack2<T>(o[b][i + 6] * inv, o[b][i + 7] * inv);
                const auto r0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
                const auto r1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
                const uint32_t c = 32 * b + 2 * i + 8 * half;
                if (c < p.d) *reinterpret_cast<v4u*>(op + c) = v4u{r0[0], r1[0], r0[1], r1[1]};
            }
        }
    }
#endif
}

}  // namespace attn

namespace {

template <typename T, int DP, int NW>
hipError_t launch(attn::Params p, uint32_t bh, hipStream_t st)
{
    p.m_tiles = (p.rows + 32 * NW - 1) / (32 * NW);
    p.by_tiles = FastDiv(p.m_tiles);
    attn::tile_kernel<T, DP, NW><<<dim3(bh * p.m_tiles), dim3(NW * 64), 0, st>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t pick(const attn::Params& p, uint32_t bh, hipStream_t st)
{
    if (p.d <= 64) return launch<T, 64, 4>(p, bh, st);
    if (p.d <= 96) return launch<T, 96, 4>(p, bh, st);
    return launch<T, 128, 4>(p, bh, st);
}

}  // namespace

size_t cross_attn_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_cross_attn(const AttnArgs& a, hipStream_t st)
{
    attn::Params p{};
    p.q = a.q, p.k = a.k, p.v = a.v, p.o = a.o;
    p.q_sb = a.q_sb, p.q_st = a.q_st, p.q_sh = a.q_sh;
    p.k_sb = a.k_sb, p.k_st = a.k_st, p.k_sh = a.k_sh;
    p.v_sb = a.v_sb, p.v_st = a.v_st, p.v_sh = a.v_sh;
    p.o_sb = a.o_sb, p.o_st = a.o_st, p.o_sh = a.o_sh;
    p.kv_len = a.kv_len;
    p.mask = a.mask;
    p.mask_sb = a.mask_sb;
    p.tk = (uint32_t)a.tk;
    p.d = (uint32_t)a.d;
    p.share = (uint32_t)(a.batch / a.kv_batch);
    p.heads_kv = (uint32_t)a.kv_heads;
    const int64_t g = a.heads / a.kv_heads;
    p.rows = (uint32_t)(p.share * a.tq * g);
    p.c = a.scale * 1.44269504088896340736f;
    p.by_g = FastDiv((uint32_t)g);
    p.by_tq = FastDiv((uint32_t)a.tq);
    p.by_hkv = FastDiv((uint32_t)a.kv_heads);
    const uint32_t bh = (uint32_t)(a.kv_batch * a.kv_heads);
    return a.fp16 ? pick<f16>(p, bh, st) : pick<bf16>(p, bh, st);
}

}  // namespace ck
