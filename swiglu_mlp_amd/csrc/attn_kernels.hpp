// attn_kernels.hpp -- attention of query rows over encoder keys and values of another
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
// Keys that are not allowed are never read.  With a key mask the workgroup
// lists the allowed keys of the next 4096 in LDS (their order kept) and the
// tiles are made of those, so a dropped key costs neither its bytes nor its
// products; lanes past the last key load from past the buffer, which gives
// zeros, and their scores are set to -inf.
//
// Two kernels.  tile_kernel: the waves of a workgroup hold different rows and
// share each K / V tile.  Many rows are bound by the matrix cores, and those by
// the chip's power: 24 heads of 128, 16384 rows over 4096 keys take 742 to 776 us by
// card (1060 to 1110 TFLOP/s, a plain BF16 library product 1263) at 1.5 to 1.7 GHz with the
// matrix cores busy 57% of the time; on zeros, 548.  A tile costs a wave 32 products and about
// 150 other vector operations.  slice_kernel: the waves hold the same 32 rows and
// each streams its own 32-key slices through LDS of its own, without a barrier:
// few rows are bound by HBM (one token over 131072 keys, 537 MB: 84 to 86 us, 6.2
// to 6.4 TB/s) or, over few keys, by latency (512 keys: 7.4 us).  Either may split the
// keys over several workgroups; the unnormalised FP32 partial results then go to
// the workspace and join_kernel adds them in a fixed order (3 to 4.5 us).
#pragma once
#include "attn.hpp"

namespace ck {
namespace attn {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

#if defined(__HIP_DEVICE_COMPILE__)

// s_waitcnt vmcnt(N) alone
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    asm volatile("" ::: "memory");
}

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
// LDS reads; the caller waits (wait_vmcnt) before the data's first use.  NT:
// nontemporal.
template <bool NT>
__device__ __forceinline__ void lds_dma_b128(v4i rsrc, uint32_t voff, uint32_t lds)
{
    if constexpr (NT)
        asm volatile(
            "s_mov_b32 m0, %2\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %0, %1, 0 offen nt lds"
            :
            : "v"(voff), "s"(rsrc), "s"(lds)
            : "memory", "m0");
    else
        asm volatile(
            "s_mov_b32 m0, %2\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %0, %1, 0 offen lds"
            :
            : "v"(voff), "s"(rsrc), "s"(lds)
            : "memory", "m0");
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

// What one lane knows of its row and its workgroup's keys.
struct Place {
    uint32_t half, col;        // lane / 32, lane % 32
    uint32_t bh, hk, eb;       // key head of the call, of its sequence; encoder sequence
    uint32_t split, row;       // row: of the key head's list, may be past the last
    uint32_t first, last;      // this workgroup's keys
    int64_t q_at, o_at;        // element offsets of the row
};

// Workgroup index -> (key head, split, row tile), the row tiles of one split
// next to each other.  Workgroups go to the 8 XCDs (each with an L2 of its own)
// in turn: without lengths each XCD takes a contiguous eighth of the order, so
// the row tiles that read the same keys share an L2.  With lengths the plain
// order stays, which spreads a long sequence over the XCDs, and with LONGEST
// the longest of up to 16 sequences come first (333 rows of 7 sequences of up to
// 1023 keys: 22.3 us, 23.9 shortest first; ranking 64 sequences takes 3 us).
// Plain order against contiguous eighths, both with lengths: those 333 rows 22.3
// and 27.9 us, 1024 rows of 16 sequences of 128 to 2048 keys, 16 heads of 64: 95
// and 129, 2 x 4096 rows of 512 and 300 keys, 24 heads of 128: 56.6 and 61.6; but
// both of 512 keys: 66.8 and 64.9, and one sequence of 16384 rows and 4096 keys:
// 768 and 766.
template <bool LONGEST>
__device__ __forceinline__ Place place_of(const Params& p, uint32_t row_in_tile, uint32_t tile_rows)
{
    Place w;
    const uint32_t lane = threadIdx.x & 63;
    w.half = lane >> 5, w.col = lane & 31;
    uint32_t at = blockIdx.x;
    if (!p.kv_len) {
        const uint32_t x = at & 7u, all = gridDim.x;
        at = x * (all >> 3) + min(x, all & 7u) + (at >> 3);
    }
    const uint32_t rest = p.by_tiles.div(at);
    const uint32_t mt = at - rest * p.m_tiles;
    const uint32_t order = p.by_splits.div(rest);
    w.split = rest - order * p.splits;
    w.eb = p.by_hkv.div(order);
    w.hk = order - w.eb * p.heads_kv;
    uint32_t len = p.tk;
    if (LONGEST && p.kv_len && p.kv_batch <= 16) {   // a sequence a lane
        const int mine = lane < p.kv_batch ? min(max(p.kv_len[lane], 0), (int)p.tk) : -1;
        uint32_t rank = 0;   // sequences before this lane's
        for (uint32_t i = 0; i < p.kv_batch; ++i) {
            const int other = __builtin_amdgcn_readlane(mine, i);
            rank += other > mine || (other == mine && i < lane);
        }
        w.eb = __builtin_ctzll(__ballot(rank == w.eb && lane < p.kv_batch));
        len = __builtin_amdgcn_readlane(mine, w.eb);
    } else if (p.kv_len) {
        // through the scalar cache: nothing in this launch writes lengths
        typedef const __attribute__((address_space(4))) int32_t* Lens;
        len = min(max(((Lens)p.kv_len)[w.eb], 0), (int)p.tk);
    }
    w.bh = w.eb * p.heads_kv + w.hk;
    w.row = mt * tile_rows + row_in_tile + w.col;
    const uint32_t r = w.row < p.rows ? w.row : p.rows - 1;   // rows past the last compute the last, and store nothing
    const uint32_t rt = p.by_g.div(r);
    const uint32_t head = w.hk * p.by_g.d + (r - rt * p.by_g.d);
    const uint32_t si = p.by_tq.div(rt);
    const uint32_t tok = rt - si * p.by_tq.d;
    const int64_t seq = (int64_t)w.eb * p.share + si;
    w.q_at = seq * p.q_sb + (int64_t)tok * p.q_st + (int64_t)head * p.q_sh;
    w.o_at = seq * p.o_sb + (int64_t)tok * p.o_st + (int64_t)head * p.o_sh;
    w.first = min(w.split * p.split_keys, len);
    w.last = min(w.first + p.split_keys, len);
    return w;
}

// The row's fragments.  Chunks past d hold channels of the last one again: K is
// zero there.  (An infinity or NaN in q makes the row NaN with or without them.)
template <int DP>
__device__ __forceinline__ void load_q(const Params& p, const Place& w, v4u (&q)[DP / 16])
{
#pragma unroll
    for (int s = 0; s < DP / 16; ++s)
        q[s] = *reinterpret_cast<const v4u*>(p.q + w.q_at + min(16 * s + 8 * w.half, p.d - 8));
}

// The indices (from `from`) of the allowed keys among [from, from + n), n <=
// kList, in order; returns their number.  All NT threads of the workgroup
// call it together; counts: one word per wave of LDS.
template <int NT>
__device__ uint32_t list_keys(const uint8_t* mask, uint32_t from, uint32_t n, uint16_t* list, uint32_t* counts)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t total = 0;
    for (uint32_t r = 0; r < n; r += NT * 8) {
        const uint32_t j = r + tid * 8;
        uint32_t keep = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (j + e < n && mask[(uint64_t)from + j + e]) keep |= 1u << e;
        const uint32_t mine = __popc(keep);
        uint32_t upto = mine;   // inclusive count over the wave
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t x = __shfl_up(upto, s);
            if (lane >= (uint32_t)s) upto += x;
        }
        __syncthreads();   // counts of the round before are read
        if (lane == 63) counts[wave] = upto;
        __syncthreads();
        uint32_t at = total + upto - mine;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) {
            const uint32_t c = counts[w];
            if ((uint32_t)w < wave) at += c;
            total += c;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (keep >> e & 1) list[at++] = (uint16_t)(j + e);
    }
    __syncthreads();
    return total;
}

// A wave's loads of a K or V tile of NK keys into LDS: CNT of its NK DP / 512
// one-KB pieces, from piece `first` on, a 16-byte chunk per lane.  LISTED: the
// keys come through a list of their indices.
template <int DP, int NK, int CNT, bool LISTED, bool NT>
struct Loader {
    static constexpr int CH = DP / 8;
    const char* base;      // key 0 of the head
    uint32_t pitch;        // bytes from key to key
    uint32_t first, lane;
    uint32_t off[CNT];     // of this lane's chunk: in its row (LISTED) or in the tile

    // key of the tile that this lane reads in piece first + i
    __device__ __forceinline__ uint32_t row(int i) const
    {
        if constexpr (64 % CH == 0) return lane / CH + (first + i) * (64 / CH);
        return ((first + i) * 64 + lane) / CH;
    }
    __device__ __forceinline__ bool past(int i, uint32_t left) const   // row(i) >= left
    {
        if constexpr (64 % CH == 0) return (int)(lane / CH) >= (int)(left - (first + i) * (64 / CH));
        return row(i) >= left;
    }
    __device__ __forceinline__ void init(const Params& p, const Place& w, bool is_v, uint32_t first_piece)
    {
        base = reinterpret_cast<const char*>(is_v ? p.v + (int64_t)w.eb * p.v_sb + (int64_t)w.hk * p.v_sh
                                                  : p.k + (int64_t)w.eb * p.k_sb + (int64_t)w.hk * p.k_sh);
        pitch = (uint32_t)((is_v ? p.v_st : p.k_st) * 2);
        first = first_piece;
        lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < CNT; ++i) {
            const uint32_t r = row(i), at = ((first + i) * 64 + lane) % CH;
            const uint32_t c = is_v ? v_swz<CH>(r, at) : k_swz<CH>(r, at);   // both are their own inverse
            // a chunk past d: 2^31, and past the buffer with any row's offset added
            off[i] = (8 * c < p.d ? 16 * c : kBufferOutside) + (LISTED ? 0 : r * pitch);
        }
    }
    // keys key .. key + NK - 1, or key + list[0 .. NK - 1], to the tile at LDS
    // address lds; only the first `left` are there
    __device__ __forceinline__ void load(uint32_t key, const uint16_t* list, uint32_t left, uint32_t lds) const
    {
        const v4i rsrc = make_rsrc(base + (uint64_t)key * pitch);
        if (!LISTED && left >= (uint32_t)NK) {
#pragma unroll
            for (int i = 0; i < CNT; ++i) lds_dma_b128<NT>(rsrc, off[i], lds + (first + i) * 1024);
        } else {
            uint32_t at[CNT];
#pragma unroll
            for (int i = 0; i < CNT; ++i) {
                at[i] = off[i];
                // the list's entries past its end are old ones, and not used
                if constexpr (LISTED) at[i] += __umul24(list[row(i)], pitch);
                if (past(i, left)) at[i] = kBufferOutside;
            }
#pragma unroll
            for (int i = 0; i < CNT; ++i) lds_dma_b128<NT>(rsrc, at[i], lds + (first + i) * 1024);
        }
    }
};

typedef const __attribute__((address_space(3))) char* LdsPtr;

// A lane's places in a K tile (its fragment of 16 channels of row col) and in
// the V tile behind it (its 8 bytes of the transposing reads of 32 channels).
// Buffers and rows are constant offsets from these, so a tile's reads cost no
// address arithmetic.
template <int DP>
struct Reads {
    static constexpr int CH = DP / 8;
    LdsPtr k[DP / 16], v[DP / 32];
    __device__ __forceinline__ Reads(const char* base, uint32_t v_behind, uint32_t half, uint32_t col)
    {
        const LdsPtr p = (LdsPtr)base;
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) k[s] = p + (col * CH + k_swz<CH>(col, 2 * s + half)) * 16;
        const uint32_t lane = half * 32 + col, j = lane & 15;
        const uint32_t key = 4 * half + (j >> 2), c = 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
#pragma unroll
        for (int b = 0; b < DP / 32; ++b)
            v[b] = p + v_behind + (key * CH + v_swz<CH>(key, 4 * b + c)) * 16 + 8 * (j & 1);
    }
    __device__ __forceinline__ void move(int by)
    {
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) k[s] += by;
#pragma unroll
        for (int b = 0; b < DP / 32; ++b) v[b] += by;
    }
};

// The running softmax of one row (m: of the raw scores) and its accumulators.
// FP16 probabilities are scaled by 2^kLift, so that small ones keep their bits:
// with the deferred maximum below they reach at most 2^14.
template <typename T, int DP>
struct Row {
    static constexpr int CH = DP / 8, DB = DP / 32, KS = DP / 16;
    static constexpr float kLift = __is_same(T, f16) ? 6.0f : 0.0f;
    static constexpr float kDefer = 8.0f;
    v16f o[DB];
    float m, l;

    __device__ __forceinline__ void clear()
    {
        m = -__builtin_inff();
        l = 0.0f;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[b][i] = 0.0f;
    }

    __device__ __forceinline__ static v4u k_read(LdsPtr at)
    {
        typedef const __attribute__((address_space(3))) v4u* LdsV4u;
        return *(LdsV4u)at;
    }
    __device__ __forceinline__ static v4u v_read(LdsPtr at)   // keys .. + 3 and + 8 .. + 11
    {
        typedef __attribute__((address_space(3))) v4s* LdsV4s;
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsV4s)at);
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsV4s)(at + 8 * CH * 16));
        return __builtin_bit_cast(v4u, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }

    // 32 N keys in LDS, AT bytes behind the places `rd`, the first `left` of
    // them real.  The order of the source is kept (sched_barrier): a fragment
    // is read a whole block of products before its use, the first V fragments
    // before the softmax, and the exponentials of the second 32 keys are spread
    // over the products with the first 32.
    template <int N, int AT>
    __device__ __forceinline__ void step(const Reads<DP>& rd, const v4u (&q)[KS], uint32_t left, float c, uint32_t half)
    {
        v16f s[N];
        v4u kf[KS], vf[DB];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) kf[ks] = k_read(rd.k[ks] + AT);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[n][i] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                s[n] = mfma<T>(kf[ks], q[ks], s[n]);
                if (n + 1 < N) kf[ks] = k_read(rd.k[ks] + (AT + (n + 1) * 32 * CH * 16));
                if (n + 1 == N && ks >= KS - DB) vf[ks - (KS - DB)] = v_read(rd.v[ks - (KS - DB)] + AT);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (left < 32u * N) {
            const int end = (int)left - 4 * (int)half;   // one register against constants
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n * 32 + (i & 3) + 8 * (i >> 2) >= end) s[n][i] = -__builtin_inff();
        }
        float mx = s[0][0];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[n][i]);
        mx = half_max(mx);
        // The maximum in use may lag behind the true one by up to 2^kDefer in
        // the probabilities: FP32 sums and 16-bit floats lose nothing by it, and
        // most tiles skip the rescale of the accumulators.
        if (__any((mx - m) * c > kDefer)) {
            const float mn = fmaxf(m, mx);
            const float alpha = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f((m - mn) * c);
            m = mn;
            l = l * alpha;
#pragma unroll
            for (int b = 0; b < DB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][i] *= alpha;
        }
        const float shift = (m == -__builtin_inff() ? 0.0f : -m * c) + kLift;
        float la = 0.0f, lb = 0.0f;
        uint32_t pw[N][8];   // probabilities of keys 2 w, 2 w + 1 of block n
        auto weigh = [&](int n, int w) {
            const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][2 * w], c, shift));
            const float b = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][2 * w + 1], c, shift));
            la += a;
            lb += b;
            pw[n][w] = pack2<T>(a, b);
        };
#pragma unroll
        for (int w = 0; w < 8; ++w) weigh(0, w);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < 2 * N; ++g) {
            const v4u pf = {pw[g / 2][4 * (g % 2)], pw[g / 2][4 * (g % 2) + 1], pw[g / 2][4 * (g % 2) + 2],
                            pw[g / 2][4 * (g % 2) + 3]};
#pragma unroll
            for (int b = 0; b < DB; ++b) {
                o[b] = mfma<T>(vf[b], pf, o[b]);
                if (g + 1 < 2 * N) vf[b] = v_read(rd.v[b] + (AT + (g + 1) * 16 * CH * 16));
                if (g < 2 && N > 1) {   // product g DB + b of the 2 DB: its share of the 8 pairs
                    const int i = g * DB + b;
#pragma unroll
                    for (int w = 8 * i / (2 * DB); w < 8 * (i + 1) / (2 * DB); ++w) weigh(N - 1, w);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        l += la + lb;
    }

    // After the last step: the row's whole sum, and the marks of a row without
    // finite scores: m = -inf where there was no key at all (o = 0), the lowest
    // float where there were keys and all their scores were -inf (0 / 0).
    __device__ __forceinline__ void finish(bool any)
    {
        l = half_sum(l);
        if (any && m == -__builtin_inff()) m = -3.402823466e38f;
    }
};

#endif

// DP: channels padded to 64, 96 or 128 (the chunks past d load zeros).
// KG key groups of NW waves each: a group's waves hold 32 rows each and share
// its tiles of 64 keys; the groups hold the same rows, take every KG-th tile,
// and are joined through LDS at the end.  With KG = 1 two (four for 64
// channels) workgroups share a CU; KG = 2 fills a CU by itself, for calls with
// no more workgroups than CUs.  MASK: with a key mask (its lists would cost the
// other calls registers).
template <typename T, int DP, int NW, int KG, bool MASK>
__global__ __launch_bounds__(NW * KG * 64, DP <= 64 && KG == 1 && !MASK ? 4 : 2) void tile_kernel(Params p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int NK = 64, DB = DP / 32;
    constexpr int TILE_B = NK * DP * 2;              // bytes of one K or V tile
    constexpr int CNT = TILE_B / 1024 / (NW / 2);    // loads of a tile per wave: half of a group's waves load K, half V
    static_assert(TILE_B % (1024 * NW / 2) == 0, "loads split evenly over the waves");
    constexpr int RING_B = 2 * 2 * TILE_B;           // a group's two buffers
    constexpr int ACC_B = DB * 16 * NW * 64 * 4;     // a group's accumulators
    static_assert((KG - 1) * ACC_B <= KG * RING_B, "the other groups' accumulators fit the rings");
    __shared__ __attribute__((aligned(1024))) char smem[KG * RING_B];
    __shared__ uint16_t list[MASK ? kList + 64 : 1];
    __shared__ uint32_t counts[NW * KG];
    __shared__ float2 ml[KG > 1 ? KG - 1 : 1][KG > 1 ? NW * 64 : 1];

    const int all_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t group = all_wave / NW;
    const int wave = all_wave % NW;
    const Place w = place_of<true>(p, wave * 32, NW * 32);
    Loader<DP, NK, CNT, MASK, false> ld;
    ld.init(p, w, wave >= NW / 2, wave % (NW / 2) * CNT);
    const char* ring = smem + group * RING_B;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem + group * RING_B +
                          wave / (NW / 2) * TILE_B;
    const uint8_t* mask = MASK ? p.mask + (int64_t)w.eb * p.mask_sb : nullptr;
    if constexpr (!MASK) {   // before the queries: the longer way
        const uint32_t n = w.last - w.first;
        if (group * NK < n) ld.load(w.first + group * NK, list, n - group * NK, lds0);
    }
    v4u q[DP / 16];
    load_q<DP>(p, w, q);

    Reads<DP> rd(ring, TILE_B, w.half, w.col);
    Row<T, DP> r;
    r.clear();
    bool any = false;   // whether any key was allowed (the same for all rows)
    // without a mask one pass over all keys; with one, a pass for each list
    for (uint32_t from = w.first; from < w.last;) {
        uint32_t n = w.last - from;
        const uint32_t upto = MASK ? from + min(n, p.list_keys) : w.last;
        if constexpr (MASK) n = list_keys<NW * KG * 64>(mask, from, upto - from, list, counts);
        any |= n != 0;
        const uint32_t tiles = (n + NK - 1) / NK;
        // tile t of the pass to buffer `to`, if there is one
        auto load = [&](uint32_t t, uint32_t to) {
            if (t < tiles)
                ld.load(MASK ? from : from + t * NK, list + t * NK, n - t * NK, lds0 + to * 2 * TILE_B);
        };
        if constexpr (MASK) {
            load(group, 0);
            // one loop body, its places moved from buffer to buffer: with two
            // bodies in two nested loops the accumulators were held twice
            int other = 2 * TILE_B;
            for (uint32_t i = 0, t = group; i < tiles; i += KG, t += KG) {
                wait_vmcnt<0>();
                workgroup_barrier();
                load(t + KG, other > 0);
                if (KG == 1 || t < tiles) r.template step<2, 0>(rd, q, n - t * NK, p.c, w.half);
                rd.move(other);
                other = -other;
            }
            if (other < 0) rd.move(other);   // back to the first buffer
            workgroup_barrier();             // the list and the buffers are free
        } else {
            // i: the first group's tile, for an end that all groups share
            for (uint32_t i = 0, t = group;; ) {
                wait_vmcnt<0>();
                workgroup_barrier();   // tile t is in LDS, and every wave is done with the other buffer
                load(t + KG, 1);
                if (KG == 1 || t < tiles) r.template step<2, 0>(rd, q, n - t * NK, p.c, w.half);
                t += KG;
                if ((i += KG) >= tiles) break;
                wait_vmcnt<0>();
                workgroup_barrier();
                load(t + KG, 0);
                if (KG == 1 || t < tiles) r.template step<2, 2 * TILE_B>(rd, q, n - t * NK, p.c, w.half);
                t += KG;
                if ((i += KG) >= tiles) break;
            }
        }
        from = upto;
    }
    r.finish(any);
    if constexpr (KG > 1) {
        // the same lane of every group holds the same row and channels
        float* acc = reinterpret_cast<float*>(smem);
        const uint32_t lane = threadIdx.x % (NW * 64);
        __syncthreads();   // the rings are free
        if (group > 0) {
            ml[group - 1][lane] = make_float2(r.m, r.l);
#pragma unroll
            for (int b = 0; b < DB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[((group - 1) * DB * 16 + b * 16 + i) * (NW * 64) + lane] = r.o[b][i];
        }
        __syncthreads();
        if (group > 0) return;
        float m = r.m;
#pragma unroll
        for (int g = 0; g < KG - 1; ++g) m = fmaxf(m, ml[g][lane].x);
        // (-inf) - (-inf) is no weight: such a group holds nothing
        const float own = r.m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((r.m - m) * p.c);
        r.l *= own;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) r.o[b][i] *= own;
#pragma unroll
        for (int g = 0; g < KG - 1; ++g) {
            const float2 t = ml[g][lane];
            const float f = t.x == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((t.x - m) * p.c);
            r.l = __builtin_fmaf(t.y, f, r.l);
#pragma unroll
            for (int b = 0; b < DB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    r.o[b][i] = __builtin_fmaf(acc[(g * DB * 16 + b * 16 + i) * (NW * 64) + lane], f, r.o[b][i]);
        }
        r.m = m;
    }
    if (w.row >= p.rows) return;
    if (p.splits > 1) {
        const uint64_t at = ((uint64_t)w.bh * p.rows + w.row) * p.splits + w.split;
        if (w.half == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(r.m, r.l);
        float* po = p.part_o + at * p.d + 4 * w.half;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (32 * b + 2 * i + 4 * w.half < p.d)
                    *reinterpret_cast<float4*>(po + 32 * b + 2 * i) =
                        make_float4(r.o[b][i], r.o[b][i + 1], r.o[b][i + 2], r.o[b][i + 3]);
        return;
    }
    // o[b][i] is channel 32 b + (i % 4) + 8 (i / 4) + 4 half of row col: pairs
    // of 4-channel groups are exchanged between the halves for 16-byte stores.
    const float inv = r.m == -__builtin_inff() ? 0.0f : 1.0f / r.l;   // no allowed key: o is zero
    uint16_t* op = p.o + w.o_at;
#pragma unroll
    for (int b = 0; b < DB; ++b) {
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            const uint32_t x0 = pack2<T>(r.o[b][i] * inv, r.o[b][i + 1] * inv);
            const uint32_t x1 = pack2<T>(r.o[b][i + 2] * inv, r.o[b][i + 3] * inv);
            const uint32_t y0 = pack2<T>(r.o[b][i + 4] * inv, r.o[b][i + 5] * inv);
            const uint32_t y1 = pack2<T>(r.o[b][i + 6] * inv, r.o[b][i + 7] * inv);
            const auto r0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
            const auto r1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
            const uint32_t c = 32 * b + 2 * i + 8 * w.half;
            if (c < p.d) *reinterpret_cast<v4u*>(op + c) = v4u{r0[0], r1[0], r0[1], r1[1]};
        }
    }
#endif
}

// Few rows: 4 waves on the same 32 rows, each streaming every fourth slice of
// 32 keys through two buffers of its own.  NT: nontemporal loads of K and V, for
// calls that read them once and past the Infinity Cache (one token over 131072
// keys, 8 key heads of 128, 537 MB: 89 us, 99 without; over 67 MB of keys 17.2,
// 16.6 without).
template <typename T, int DP, bool MASK, bool NT>
__global__ __launch_bounds__(256, 1) void slice_kernel(Params p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int NW = 4, NK = 32, DB = DP / 32;
    constexpr int SLICE_B = NK * DP * 2;             // bytes of one K or V slice
    constexpr int CNT = SLICE_B / 1024;              // loads per slice
    constexpr int PITCH = DP + 4;                    // floats per row of the joined accumulators
    constexpr int RING_B = NW * 2 * 2 * SLICE_B;
    static_assert(RING_B >= NW * 32 * PITCH * 4, "the accumulators of all waves fit the ring");
    __shared__ __attribute__((aligned(1024))) char smem[RING_B];
    __shared__ uint16_t list[MASK ? kList + 64 : 1];
    __shared__ uint32_t counts[NW];
    __shared__ float2 ml[NW][32];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place w = place_of<false>(p, 0, 32);
    v4u q[DP / 16];
    load_q<DP>(p, w, q);
    Loader<DP, NK, CNT, MASK, NT> lk, lv;
    lk.init(p, w, false, 0);
    lv.init(p, w, true, 0);
    const Reads<DP> rd(smem + wave * (2 * 2 * SLICE_B), SLICE_B, w.half, w.col);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem + wave * (2 * 2 * SLICE_B);
    const uint8_t* mask = MASK ? p.mask + (int64_t)w.eb * p.mask_sb : nullptr;

    Row<T, DP> r;
    r.clear();
    bool any = false;
    for (uint32_t from = w.first; from < w.last;) {
        uint32_t n = w.last - from;
        const uint32_t upto = MASK ? from + min(n, p.list_keys) : w.last;
        if constexpr (MASK) n = list_keys<NW * 64>(mask, from, upto - from, list, counts);
        any |= n != 0;
        const uint32_t slices = (n + NK - 1) / NK;
        auto load = [&](uint32_t t) {
            const uint32_t lds = lds0 + ((t - wave) / NW & 1) * 2 * SLICE_B;
            lk.load(MASK ? from : from + t * NK, list + t * NK, n - t * NK, lds);
            lv.load(MASK ? from : from + t * NK, list + t * NK, n - t * NK, lds + SLICE_B);
        };
        auto wait = [&](uint32_t t) {   // slice t is in LDS; the next one is on its way
            if (t + NW < slices) {
                load(t + NW);
                wait_vmcnt<2 * CNT>();  // all but the loads just issued
            } else {
                wait_vmcnt<0>();
            }
        };
        if (wave < slices) load(wave);
        for (uint32_t t = wave; t < slices; t += NW) {
            wait(t);
            r.template step<1, 0>(rd, q, n - t * NK, p.c, w.half);
            asm volatile("" ::: "memory");   // its LDS reads end before the next load into this buffer
            if ((t += NW) >= slices) break;
            wait(t);
            r.template step<1, 2 * SLICE_B>(rd, q, n - t * NK, p.c, w.half);
            asm volatile("" ::: "memory");
        }
        if constexpr (MASK) __syncthreads();   // the list is free
        from = upto;
    }
    r.finish(any);
    __syncthreads();       // every wave is done with the ring

    float* acc = reinterpret_cast<float*>(smem);
    if (w.half == 0) ml[wave][w.col] = make_float2(r.m, r.l);
    if (w.row < p.rows) {
        float* a = acc + (wave * 32 + w.col) * PITCH + 4 * w.half;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(a + 32 * b + 2 * i) =
                    make_float4(r.o[b][i], r.o[b][i + 1], r.o[b][i + 2], r.o[b][i + 3]);
    }
    __syncthreads();

    // joined: 8 channels of a row a thread
    constexpr int CH = DP / 8;
    const uint32_t row0 = w.row - w.col;   // the tile's first row
    for (uint32_t e = threadIdx.x; e < 32 * CH; e += 256) {
        const uint32_t row = e / CH, c = e % CH * 8;
        if (row0 + row >= p.rows || c >= p.d) continue;
        float m = ml[0][row].x;
#pragma unroll
        for (int i = 1; i < NW; ++i) m = fmaxf(m, ml[i][row].x);
        float l = 0.0f, x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const float2 t = ml[i][row];
            // (-inf) - (-inf) is no weight: such a wave holds nothing
            const float f = t.x == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((t.x - m) * p.c);
            const float* a = acc + (i * 32 + row) * PITCH + c;
            l = __builtin_fmaf(t.y, f, l);
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = __builtin_fmaf(a[u], f, x[u]);
        }
        if (p.splits > 1) {
            const uint64_t at = ((uint64_t)w.bh * p.rows + row0 + row) * p.splits + w.split;
            if (c == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, l);
            float* po = p.part_o + at * p.d + c;
            *reinterpret_cast<float4*>(po) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(po + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            const float inv = m == -__builtin_inff() ? 0.0f : 1.0f / l;
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] *= inv;
            const uint32_t rt = p.by_g.div(row0 + row);
            const uint32_t head = w.hk * p.by_g.d + (row0 + row - rt * p.by_g.d);
            const uint32_t si = p.by_tq.div(rt);
            const int64_t seq = (int64_t)w.eb * p.share + si;
            uint16_t* op = p.o + seq * p.o_sb + (int64_t)(rt - si * p.by_tq.d) * p.o_st + (int64_t)head * p.o_sh;
            *reinterpret_cast<uint4*>(op + c) = pack8<T>(x);
        }
    }
#endif
}

// The splits of a row joined, in a fixed order, 4 channels a lane.  TEAMS teams
// of 32 lanes share a row: one where there are many rows of few splits, eight
// (each every eighth split, then added) where there are few rows or many splits.
template <typename T, int TEAMS>
__global__ __launch_bounds__(256) void join_kernel(Params p, uint32_t all_rows)
{
    constexpr int ROWS = 8 / TEAMS;   // per workgroup
    __shared__ float4 acc[TEAMS == 1 ? 1 : 8][32];
    __shared__ float sums[8];
    const uint32_t team = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t at = blockIdx.x * ROWS + team / TEAMS, own = team % TEAMS;
    const bool there = lane * 4 < p.d && at < all_rows;
    const uint64_t first = (uint64_t)min(at, all_rows - 1) * p.splits;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + first;
    float m = -__builtin_inff();
    for (uint32_t s = lane; s < p.splits; s += 32) m = fmaxf(m, ml[s].x);
    m = fmaxf(m, dpp_xor<1>(m));
    m = fmaxf(m, dpp_xor<2>(m));
    m = fmaxf(m, swizzle_xor<4>(m));
    m = fmaxf(m, swizzle_xor<8>(m));
    m = fmaxf(m, swizzle_xor<16>(m));
    float l = 0.0f;
    float4 x = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (uint32_t s = own; s < p.splits; s += TEAMS) {
        const float2 t = ml[s];
        float4 v = make_float4(0, 0, 0, 0);
        // a split without keys has written its m (-inf) and l, and zeros
        if (there) v = *reinterpret_cast<const float4*>(p.part_o + (first + s) * p.d + lane * 4);
        const float f = t.x == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((t.x - m) * p.c);
        l = __builtin_fmaf(t.y, f, l);
        x.x = __builtin_fmaf(v.x, f, x.x), x.y = __builtin_fmaf(v.y, f, x.y);
        x.z = __builtin_fmaf(v.z, f, x.z), x.w = __builtin_fmaf(v.w, f, x.w);
    }
    if constexpr (TEAMS > 1) {
        acc[team][lane] = x;
        if (lane == 0) sums[team] = l;
        __syncthreads();
        if (team != 0) return;
        l = sums[0];
#pragma unroll
        for (int i = 1; i < TEAMS; ++i) {
            const float4 v = acc[i][lane];
            l += sums[i];
            x.x += v.x, x.y += v.y, x.z += v.z, x.w += v.w;
        }
    }
    if (!there) return;
    const float inv = m == -__builtin_inff() ? 0.0f : 1.0f / l;
    const uint32_t bh = p.by_tiles.div(at), row = at - bh * p.rows;   // by_tiles: by rows here
    const uint32_t eb = p.by_hkv.div(bh), hk = bh - eb * p.heads_kv;
    const uint32_t rt = p.by_g.div(row), head = hk * p.by_g.d + (row - rt * p.by_g.d);
    const uint32_t si = p.by_tq.div(rt);
    const int64_t seq = (int64_t)eb * p.share + si;
    uint16_t* op = p.o + seq * p.o_sb + (int64_t)(rt - si * p.by_tq.d) * p.o_st + (int64_t)head * p.o_sh;
    *reinterpret_cast<uint2*>(op + lane * 4) = make_uint2(pack2<T>(x.x * inv, x.y * inv), pack2<T>(x.z * inv, x.w * inv));
}

template <typename T, int DP, bool MASK>
hipError_t launch_padded(Params& p, const Plan& plan, uint32_t bh, hipStream_t st)
{
    const dim3 grid(bh * plan.m_tiles * plan.splits);
    if (plan.slices && plan.streamed)
        slice_kernel<T, DP, MASK, true><<<grid, dim3(256), 0, st>>>(p);
    if (plan.slices && !plan.streamed)
        slice_kernel<T, DP, MASK, false><<<grid, dim3(256), 0, st>>>(p);
    if (!plan.slices && plan.two_groups)
        tile_kernel<T, DP, kTileWaves, 2, MASK><<<grid, dim3(2 * kTileWaves * 64), 0, st>>>(p);
    if (!plan.slices && !plan.two_groups)
        tile_kernel<T, DP, kTileWaves, 1, MASK><<<grid, dim3(kTileWaves * 64), 0, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || plan.splits == 1) return e;
    p.by_tiles = FastDiv(p.rows);
    const uint32_t rows = bh * p.rows;
    // 160 rows of 6 splits: 7.9 us a call with eight teams a row, 8.6 with one;
    // 4096 rows of 4: 21.3 and 19.4
    if (plan.splits >= 16 || rows <= 512)
        join_kernel<T, 8><<<dim3(rows), dim3(256), 0, st>>>(p, rows);
    else
        join_kernel<T, 1><<<dim3((rows + 7) / 8), dim3(256), 0, st>>>(p, rows);
    return hipGetLastError();
}

template <typename T, bool MASK>
hipError_t launch_masked(Params& p, const Plan& plan, uint32_t bh, hipStream_t st)
{
    if (p.d <= 64) return launch_padded<T, 64, MASK>(p, plan, bh, st);
    if (p.d <= 96) return launch_padded<T, 96, MASK>(p, plan, bh, st);
    return launch_padded<T, 128, MASK>(p, plan, bh, st);
}

template <typename T>
hipError_t launch(Params& p, const Plan& plan, uint32_t bh, hipStream_t st)
{
    return p.mask ? launch_masked<T, true>(p, plan, bh, st) : launch_masked<T, false>(p, plan, bh, st);
}

}  // namespace attn
}  // namespace ck
