// mx4_gemm.hip -- the product of microscaled 4-bit operands (include/ck.h, "MX
// FP4 linears"): y[m, n] = bf16(sum_k x[m, k] w[n, k] (+ bias[n]) (+ residual[m, n])),
// both operands in the blocked layout.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 x 64 by 64 x 32 values of 4
// bits, each lane's 32 with a scale of its own, and adds in FP32.  W is its A
// operand and x its B operand, so a lane ends with four consecutive n of one m.
// A k-slice is 64 values, 32 bytes of a row, and one 1 KB block of a 32-row
// block is an operand in lane order.
//
// The matrix cores set the pace of large products: random codes reach 6.5 of
// the nominal 10 PFLOP/s in a loop of nothing but these instructions (the clock
// falls under their power).  So the kernel keeps them fed:
//  * A workgroup of 4 waves (2 x 2) owns a BM x BN tile; a wave's part is FM x FN
//    fragments of 32 x 32, accumulated in AGPRs.  It reads FM + FN blocks from
//    LDS for FM FN products.
//  * K advances 2 KSL slices a stage; stages go through a ring of LDS slots by
//    DMA (buffer_load ... lds), P of them ahead.  A stage is two halves around
//    one barrier: each multiplies KSL slices while it reads the other half's
//    fragments, so products never wait for LDS.  Reads and loads are placed
//    between the products in source order.
//  * Scales come with the codes: 256 bytes for 32 rows and 256 k (4 slices), one
//    DMA instruction a wave, read as one register a fragment for 4 slices.
//  * Workgroups stay and take tiles in turn; the stages run on from a tile to the
//    next, whose loads so overlap the epilogue.  The workgroups of an XCD take
//    consecutive tiles and share operands in its L2.
//  * Few tiles: k is split over several workgroups, which write FP32 partial sums
//    that a second kernel adds in a fixed order.
#include "ck_internal.hpp"
#include "mx4.hpp"

#include <algorithm>
#include <type_traits>

namespace ck {
namespace mx4 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void_t;

// s_waitcnt encodings (gfx9: vmcnt[3:0] and [15:14], expcnt[6:4], lgkmcnt[11:8])
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// s_barrier without a memory fence: loads for later stages stay in flight.
__device__ __forceinline__ void workgroup_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 16 bytes a lane from memory to LDS address lds + 16 lane, not tracked by the
// compiler (which would wait for all of them before any LDS read): the waits are
// counted by hand.
__device__ __forceinline__ void lds_dma_b128(v4i rsrc, uint32_t voff, uint32_t soff, uint32_t lds)
{
    asm volatile(
        "s_mov_b32 m0, %3\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, %2 offen lds"
        :
        : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds)
        : "memory", "m0");
}
__device__ __forceinline__ void lds_dma_b128(const uint8_t* at, uint32_t lds)
{
    asm volatile(
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %0, off"
        :
        : "v"(at), "s"(lds)
        : "memory", "m0");
}

__device__ __forceinline__ v4i make_rsrc(const void* base, int64_t bytes)
{
    const uint64_t a = (uint64_t)base;
    return v4i{(int)(uint32_t)a, (int)(uint32_t)((a >> 32) & 0xffffu),
               (int)(bytes < 0x7fffffff ? bytes : 0x7fffffff), 0x00020000};
}

template <int Q>
__device__ __forceinline__ v16f product(v4i a, v4i b, v16f c, int sa, int sb)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                           v8i{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, Q, sa, Q,
                                                           sb);
}

template <int BM_, int BN_, int KSL_>
struct Cfg {
    static constexpr int BM = BM_, BN = BN_, KSL = KSL_;
    static constexpr int KS2 = 2 * KSL;                 // slices a stage
    static constexpr int FM = BM / 64, FN = BN / 64;    // a wave's fragments
    static constexpr int A_BLK = (BN / 32) * KS2, B_BLK = (BM / 32) * KS2;
    static constexpr int AW = A_BLK / 4, XW = B_BLK / 4, L = AW + XW;   // blocks a wave loads for a stage
    static constexpr int CODES = (A_BLK + B_BLK) * 1024;
    static constexpr int CHUNKS = (BM + BN) / 32;       // of scales (32 rows, 256 k)
    static constexpr int CPW = (CHUNKS + 3) / 4;        // chunks a wave loads, into its own KB
    static constexpr int NBUF = 4, P = NBUF - 1;
    static constexpr int SBUF = KSL == 1 ? 2 : NBUF;    // a slot of scales lasts 4 slices
    static constexpr int LDS = NBUF * CODES + SBUF * 4096;
    static_assert(KSL == 1 || KSL == 2, "a stage is half of a scale chunk's k, or all of it");
    static_assert(LDS <= 160 * 1024, "LDS");
    static_assert(A_BLK % 4 == 0 && B_BLK % 4 == 0, "blocks split evenly over 4 waves");
};

struct Args {
    const uint8_t *xc, *xs, *wc, *ws;
    void* out;          // BF16 [M, N], or the FP32 partial sums [splits][M][N]
    EpiExtra ex;
    int M, N;
    int kb;             // 1 KB blocks (slices) of a 32-row block: kp / 64
    int xb, wb;         // 32-row blocks of x and w
    int tiles_m, tiles_n, group_m;
    int splits, stages; // stages of one unit (a tile and one of the splits of k)
};

// Tile j of the grouped order -> (tm, tn): columns of `group_m` tile-rows.
__device__ __forceinline__ void tile_coords(int j, int tiles_m, int tiles_n, int group_m, int& tm, int& tn)
{
    const int width = group_m * tiles_n;
    const int grp = j / width;
    const int first_m = grp * group_m;
    const int gm = min(tiles_m - first_m, group_m);
    tm = first_m + (j % width) % gm;
    tn = (j % width) / gm;
}

// PART: FP32 partial sums out.  EXTRA: bias and / or residual.
template <int BM, int BN, int KSL, bool PART, bool EXTRA>
__global__ __launch_bounds__(256) void mx4_gemm_kernel(Args g)
{
    // The body uses AMDGPU-only types; the host pass only needs the launch stub.
#if defined(__HIP_DEVICE_COMPILE__)
    using C = Cfg<BM, BN, KSL>;
    __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
    constexpr int NMF = C::FN * C::FM;                  // products of a slice
    constexpr int NDS = C::FN + C::FM;                  // fragment reads of a slice
    // Large tiles spread a stage's loads over both halves: a burst of them fills
    // the address unit's queue and holds up the products behind it.
    constexpr bool SPREAD = KSL == 1;
    constexpr int HL = SPREAD ? C::L / 2 : C::L;        // loads of the first half
    constexpr int NST = PART ? 0 : 2 * NMF;             // stores of an epilogue (PART: too many to count, waited for)
    // Loads issued after the last of stage s + 1 at the middle of stage s: those of
    // the stages up to s + P but for the second half's, with their scales (KSL 1:
    // one of any two consecutive stages has some).
    constexpr int OUTS = SPREAD ? (C::P - 2) * C::L + HL + 1 : (C::P - 1) * (C::L + 1);
    static_assert(!SPREAD || C::P == 3, "the count above");
    static_assert(OUTS + NST < 64, "vmcnt range");

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = gridDim.x, b = blockIdx.x;
    const int tiles = g.tiles_m * g.tiles_n;
    const int units = tiles * g.splits;                 // split-major
    const int KT = g.stages;
    const int my_units = (units - b + G - 1) / G;
    const int total = my_units * KT;

    // Within a full round the workgroups of one XCD (b % 8) take consecutive units.
    const bool xcd_order = (G & 7) == 0;
    const int b_xcd = (b & 7) * (G >> 3) + (b >> 3);
    auto unit_of = [&](int q) {
        const bool full = xcd_order & ((q + 1) * G <= units);
        return q * G + (full ? b_xcd : b);
    };
    const uint32_t smem_addr = (uint32_t)(uintptr_t)(lds_void_t*)smem;
    const uint32_t lane16 = (uint32_t)lane * 16u;

    // ---- the load cursor: the stage to be loaded next (it stays at the last one,
    // whose repeated loads go to slots that nobody reads again, so that the number
    // of loads of a stage is constant) ----
    int ls = 0, lq = 0, lkt = 0;
    v4i rs_w, rs_x;                                     // the tile's rows of codes, from the unit's first slice
    const uint8_t* sp;                                  // this lane's scales of the unit's first 256 k
    auto set_unit = [&](int q) {
        const int u = unit_of(q), k0 = (u / tiles) * KT * C::KS2;
        int tm, tn;
        tile_coords(u % tiles, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
        const int64_t wb0 = (int64_t)tn * (BN / 32), xb0 = (int64_t)tm * (BM / 32);
        const int64_t w0 = (wb0 * g.kb + k0) * 1024, x0 = (xb0 * g.kb + k0) * 1024;
        // blocks past the operand's end are outside the buffer and read as zero
        rs_w = make_rsrc(g.wc + w0, (int64_t)g.wb * g.kb * 1024 - w0);
        rs_x = make_rsrc(g.xc + x0, (int64_t)g.xb * g.kb * 1024 - x0);
        // a chunk past the end takes the last block's scales (for products that are not stored)
        const int c = min(wave * C::CPW + min(lane >> 4, C::CPW - 1), C::CHUNKS - 1);
        const bool w = c < BN / 32;
        const int64_t rb = w ? min((int64_t)g.wb - 1, wb0 + c) : min((int64_t)g.xb - 1, xb0 + c - BN / 32);
        sp = (w ? g.ws : g.xs) + (rb * (g.kb / 4) + k0 / 4) * 256 + (lane & 15) * 16;
    };
    auto advance = [&]() {
        if (ls + 1 < total) {
            ++ls;
            if (++lkt == KT) {
                lkt = 0;
                set_unit(++lq);
            }
        }
    };
    // Block a of this wave's share of a stage: block ai covers row block ai / KS2, slice ai % KS2.
    auto issue_one = [&](int a, uint32_t slot) {
        const bool w = a < C::AW;
        const int ai = w ? wave * C::AW + a : wave * C::XW + (a - C::AW);
        const uint32_t off = (uint32_t)(lkt * C::KS2 + (ai / (unsigned)C::KS2) * g.kb + (ai % (unsigned)C::KS2)) * 1024u;
        if (w)
            lds_dma_b128(rs_w, lane16, off, slot + (uint32_t)ai * 1024u);
        else
            lds_dma_b128(rs_x, lane16, off, slot + (uint32_t)(C::A_BLK + ai) * 1024u);
    };
    auto issue_scales = [&](int d) {   // d: counts the slots of scales
        lds_dma_b128(sp + (lkt * C::KS2 / 4) * 256,
                     smem_addr + (uint32_t)(C::NBUF * C::CODES + (d % C::SBUF) * 4096 + wave * 1024));
    };

    v16f acc[C::FN][C::FM];
    const int lr = lane & 31, lh = lane >> 5;
    const int wm0 = (wave & 1) * (BM / 2), wn0 = (wave >> 1) * (BN / 2);
    auto frag_a = [&](int buf, int i, int ks) {
        return *reinterpret_cast<const v4i*>(smem + buf * C::CODES + (((wn0 >> 5) + i) * C::KS2 + ks) * 1024 + lane * 16);
    };
    auto frag_b = [&](int buf, int j, int ks) {
        return *reinterpret_cast<const v4i*>(smem + buf * C::CODES + (C::A_BLK + ((wm0 >> 5) + j) * C::KS2 + ks) * 1024 +
                                             lane * 16);
    };
    auto scale = [&](int d, int c) {
        return *reinterpret_cast<const int*>(smem + C::NBUF * C::CODES + (d % C::SBUF) * 4096 + (c / C::CPW) * 1024 +
                                             (c % C::CPW) * 256 + lane * 4);
    };

    set_unit(0);
#pragma unroll
    for (int p = 0; p < C::P; ++p) {
        if (KSL == 2 || p % 2 == 0) issue_scales(KSL == 2 ? p : p / 2);
#pragma unroll
        for (int a = 0; a < C::L; ++a) issue_one(a, smem_addr + (uint32_t)(p * C::CODES));
        advance();
    }
    wait_vmcnt<(C::P - 1) * C::L + (KSL == 2 ? C::P - 1 : 1)>();
    workgroup_barrier();
    v4i fa[KSL][C::FN], fb[KSL][C::FM], ga[KSL][C::FN], gb[KSL][C::FM];
    int sa[C::FN], sb[C::FM], na[C::FN], nb[C::FM];     // scales of 4 slices, and the next ones
#pragma unroll
    for (int ks = 0; ks < KSL; ++ks) {
#pragma unroll
        for (int i = 0; i < C::FN; ++i) fa[ks][i] = frag_a(0, i, ks);
#pragma unroll
        for (int j = 0; j < C::FM; ++j) fb[ks][j] = frag_b(0, j, ks);
    }
#pragma unroll
    for (int i = 0; i < C::FN; ++i) sa[i] = scale(0, (wn0 >> 5) + i);
#pragma unroll
    for (int j = 0; j < C::FM; ++j) sb[j] = scale(0, BN / 32 + (wm0 >> 5) + j);

    // Product k of a half whose first slice is slice Q0 of the scales' four.
    auto mfma_step = [&](int k, auto q0, const v4i (&w)[KSL][C::FN], const v4i (&x)[KSL][C::FM], bool zero) {
        constexpr int Q0 = decltype(q0)::value;
        const int ks = k / NMF, i = (k % NMF) / C::FM, j = (k % NMF) % C::FM;
        const v16f c = (zero && ks == 0) ? v16f{} : acc[i][j];
        if (ks == 0)
            acc[i][j] = product<Q0>(w[0][i], x[0][j], c, sa[i], sb[j]);
        else
            acc[i][j] = product<(Q0 + 1) & 3>(w[KSL - 1][i], x[KSL - 1][j], c, sa[i], sb[j]);
    };
    auto read_step = [&](int r, int buf, int ks0, v4i (&w)[KSL][C::FN], v4i (&x)[KSL][C::FM]) {
        if (r >= KSL * NDS) return;
        const int ks = r / NDS, rr = r % NDS;
        if (rr < C::FN) w[ks][rr] = frag_a(buf, rr, ks0 + ks);
        else x[ks][rr - C::FN] = frag_b(buf, rr - C::FN, ks0 + ks);
    };
    auto read_scale = [&](int r, int d) {
        if (r < C::FN) na[r] = scale(d, (wn0 >> 5) + r);
        else if (r < NDS) nb[r - C::FN] = scale(d, BN / 32 + (wm0 >> 5) + r - C::FN);
    };

    constexpr int STEPS = KSL * (NMF > NDS ? NMF : NDS);
    constexpr int STEPS0 = !SPREAD && C::L > STEPS ? C::L : STEPS;
    constexpr int STEPS1 = STEPS > NDS ? STEPS : NDS;
    // Stage s, of parity PAR in its unit (KSL 1: which half of the scales' k).
    auto stage = [&](int s, int kt, auto first, auto par, bool after_epilogue) {
        constexpr int PAR = decltype(par)::value;
        constexpr bool LOADS_SCALES = KSL == 2 || PAR == 1;   // the stage P = 3 ahead begins a chunk
        constexpr bool READS_SCALES = KSL == 2 || PAR == 1;   // so does the next one
        const int buf = (int)((unsigned)s % C::NBUF), nbuf = (int)((unsigned)(s + 1) % C::NBUF);
        const uint32_t lslot = smem_addr + (uint32_t)(((unsigned)(s + C::P) % C::NBUF) * C::CODES);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (LOADS_SCALES) issue_scales(KSL == 2 ? s + C::P : (s + C::P) / 2);
#pragma unroll
        for (int k = 0; k < STEPS0; ++k) {
            if (k < KSL * NMF) mfma_step(k, std::integral_constant<int, KSL == 2 ? 0 : 2 * PAR>{}, fa, fb, decltype(first)::value);
            read_step(k, buf, KSL, ga, gb);
            if constexpr (SPREAD) {
                constexpr int SP = STEPS / HL;
                if (k % SP == SP / 2 && k / SP < HL) issue_one(k / SP, lslot);
            } else {
                if (k < C::L) issue_one(k, lslot);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!SPREAD) advance();

        wait_lgkmcnt0();              // this wave's fragments of the second half are in registers
        if (kt <= C::P - 2 && after_epilogue) wait_vmcnt<OUTS + NST>();
        else wait_vmcnt<OUTS>();
        workgroup_barrier();          // every wave's; stage s + 1 is in LDS, and slot s is read no more
#pragma unroll
        for (int k = 0; k < STEPS1; ++k) {
            if (k < KSL * NMF) mfma_step(k, std::integral_constant<int, KSL == 2 ? 2 : 2 * PAR + 1>{}, ga, gb, false);
            read_step(k, nbuf, 0, fa, fb);
            if constexpr (READS_SCALES) read_scale(k, KSL == 2 ? s + 1 : (s + 1) / 2);
            if constexpr (SPREAD) {
                constexpr int SP = STEPS / (C::L - HL);
                if (k % SP == SP / 2 && k / SP < C::L - HL) issue_one(HL + k / SP, lslot);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (SPREAD) advance();
        if constexpr (READS_SCALES) {
#pragma unroll
            for (int i = 0; i < C::FN; ++i) sa[i] = na[i];
#pragma unroll
            for (int j = 0; j < C::FM; ++j) sb[j] = nb[j];
        }
    };

    // D fragment (32 x 32): lane l holds column l % 32 (output row m) and, in
    // registers 4 qd .. 4 qd + 3, rows 8 qd + 4 (l / 32) + 0..3 (four consecutive
    // n).  Lanes l and l + 32 exchange halves so that each has 8 consecutive n.
    // Rows past M lie outside the buffer of the tile's rows, columns past N are
    // given an offset outside it: both stores are dropped.
    auto epilogue = [&](int u) {
        int tm, tn;
        tile_coords(u % tiles, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
        const int64_t row0 = (int64_t)tm * BM;
        const int rows = (int)min((int64_t)BM, g.M - row0);
        constexpr int B = PART ? 4 : 2;
        char* base = static_cast<char*>(g.out) + ((PART ? (int64_t)(u / tiles) * g.M : 0) + row0) * g.N * B;
        const __amdgpu_buffer_rsrc_t rs_o = __builtin_amdgcn_make_buffer_rsrc(base, (short)0, rows * g.N * B, 0x00020000);
        const int n_base = tn * BN + wn0 + 8 * lh;
#pragma unroll
        for (int j = 0; j < C::FM; ++j) {
            const int r = wm0 + 32 * j + lr;
            const uint32_t row = (uint32_t)r * (uint32_t)g.N;
#pragma unroll
            for (int i = 0; i < C::FN; ++i) {
                // one fragment out of the accumulators here, not all of them up front
                asm volatile("" : "+a"(acc[i][j]));
                v16f f = acc[i][j];
                asm volatile("" : "+v"(f));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int n = n_base + 32 * i + 16 * h;
                    const bool ok = n < g.N;
                    if constexpr (!PART && !EXTRA) {
                        const auto r0 = __builtin_amdgcn_permlane32_swap(
                            pack_bf16x2(f[8 * h], f[8 * h + 1]), pack_bf16x2(f[8 * h + 4], f[8 * h + 5]), false, false);
                        const auto r1 = __builtin_amdgcn_permlane32_swap(
                            pack_bf16x2(f[8 * h + 2], f[8 * h + 3]), pack_bf16x2(f[8 * h + 6], f[8 * h + 7]), false, false);
                        const v4i d = {(int)r0[0], (int)r1[0], (int)r0[1], (int)r1[1]};
                        __builtin_amdgcn_raw_buffer_store_b128(d, rs_o, ok ? (row + (uint32_t)n) * 2u : kBufferOutside, 0, 0);
                    } else {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(f[8 * h + e]),
                                                                            __float_as_uint(f[8 * h + 4 + e]), false, false);
                            v[e] = __uint_as_float(t[0]);
                            v[4 + e] = __uint_as_float(t[1]);
                        }
                        if constexpr (PART) {
                            const uint32_t o = ok ? (row + (uint32_t)n) * 4u : kBufferOutside;
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, v4f{v[0], v[1], v[2], v[3]}), rs_o,
                                                                   r < rows ? o : kBufferOutside, 0, 0);
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, v4f{v[4], v[5], v[6], v[7]}), rs_o,
                                                                   r < rows && ok ? o + 16u : kBufferOutside, 0, 0);
                        } else {
                            const int nn = min(n, g.N - 8);
                            if (g.ex.bias) {
                                float bias[8];
                                *reinterpret_cast<float4*>(bias) = *reinterpret_cast<const float4*>(g.ex.bias + nn);
                                *reinterpret_cast<float4*>(bias + 4) = *reinterpret_cast<const float4*>(g.ex.bias + nn + 4);
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] = v[e] + bias[e];
                            }
                            if (g.ex.res) {
                                float res[8];
                                unpack8<bf16>(*reinterpret_cast<const uint4*>(
                                                  g.ex.res + (row0 + min(r, rows - 1)) * g.N + nn), res);
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] = v[e] + res[e];
                            }
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, pack8<bf16>(v)), rs_o,
                                                                   ok ? (row + (uint32_t)n) * 2u : kBufferOutside, 0, 0);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    int s = 0;
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    for (int q = 0; q < my_units; ++q) {
        if constexpr (KSL == 1) {   // KT is even: a padded row holds whole chunks of scales
            stage(s++, 0, std::true_type{}, even, q > 0);
            stage(s++, 1, std::false_type{}, odd, q > 0);
            for (int kt = 2; kt < KT; kt += 2) {
                stage(s++, kt, std::false_type{}, even, q > 0);
                stage(s++, kt + 1, std::false_type{}, odd, q > 0);
            }
        } else {
            stage(s++, 0, std::true_type{}, even, q > 0);
            for (int kt = 1; kt < KT; ++kt) stage(s++, kt, std::false_type{}, even, q > 0);
        }
        epilogue(unit_of(q));
    }
    wait_vmcnt<0>();   // no LDS load may land after the workgroup retires
#endif  // __HIP_DEVICE_COMPILE__
}

// y from `splits` FP32 partial sums [splits][M][N], added in order; 8 outputs a thread.
__global__ __launch_bounds__(256) void mx4_join_kernel(const float* __restrict__ part, int splits, int64_t M, int N,
                                                       EpiExtra ex, uint16_t* __restrict__ y)
{
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= M * N) return;
    float v[8] = {};
    for (int s = 0; s < splits; ++s) {
        const float4* p = reinterpret_cast<const float4*>(part + s * M * N + at);
        const float4 a = p[0], b = p[1];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    if (ex.bias) {
        const int n = (int)(at % N);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] + ex.bias[n + e];
    }
    if (ex.res) {
        float r[8];
        unpack8<bf16>(*reinterpret_cast<const uint4*>(ex.res + at), r);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] + r[e];
    }
    *reinterpret_cast<uint4*>(y + at) = pack8<bf16>(v);
}

template <int BM, int BN, int KSL>
hipError_t launch(Args g, int num_cu, hipStream_t st)
{
    using C = Cfg<BM, BN, KSL>;
    const bool part = g.splits > 1, extra = g.ex.bias || g.ex.res;
    g.tiles_m = (g.M + BM - 1) / BM;
    g.tiles_n = (g.N + BN - 1) / BN;
    g.group_m = std::min(g.tiles_m, 4);
    g.stages = g.kb / C::KS2 / g.splits;
    const int units = g.tiles_m * g.tiles_n * g.splits;
    const int slots = num_cu * (160 * 1024 / C::LDS);
    const dim3 grid(std::min(units, slots)), block(256);
    if (part)
        mx4_gemm_kernel<BM, BN, KSL, true, false><<<grid, block, 0, st>>>(g);
    else if (extra)
        mx4_gemm_kernel<BM, BN, KSL, false, true><<<grid, block, 0, st>>>(g);
    else
        mx4_gemm_kernel<BM, BN, KSL, false, false><<<grid, block, 0, st>>>(g);
    return hipGetLastError();
}

// How a product runs: which tiles, over how many splits of k.
struct Plan {
    int bm, bn, splits;
};

Plan plan_of(int64_t m, int64_t n, int64_t k, int num_cu)
{
    auto tiles = [&](int bm, int bn) { return ((m + bm - 1) / bm) * ((n + bn - 1) / bn); };
    const int64_t units = pad_cols(k) / 256;
    if (tiles(256, 256) >= num_cu) return {256, 256, 1};
    if (tiles(128, 128) >= num_cu / 2) return {128, 128, 1};
    Plan p{64, 64, 1};
    while (tiles(64, 64) * p.splits * 2 <= num_cu && units % (p.splits * 2) == 0 && units / (p.splits * 2) >= 4) p.splits *= 2;
    return p;
}

}  // namespace mx4

size_t mx4_gemm_workspace(int64_t m, int64_t n, int64_t k)
{
    const mx4::Plan p = mx4::plan_of(m, n, k, num_cus());
    return p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)n * 4 : 0;
}

hipError_t launch_mx4_gemm(const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* ws, int64_t m,
                           int64_t n, int64_t k, uint16_t* y, EpiExtra ex, void* workspace, hipStream_t st)
{
    const int num_cu = num_cus();
    const mx4::Plan p = mx4::plan_of(m, n, k, num_cu);
    mx4::Args g{};
    g.xc = xc, g.xs = xs, g.wc = wc, g.ws = ws;
    g.M = (int)m, g.N = (int)n, g.kb = (int)(mx4::pad_cols(k) / 64);
    g.xb = (int)(mx4::pad_rows(m) / 32), g.wb = (int)(mx4::pad_rows(n) / 32);
    g.splits = p.splits;
    g.out = p.splits > 1 ? workspace : y;
    if (p.splits == 1) g.ex = ex;
    hipError_t e = p.bm == 256   ? mx4::launch<256, 256, 1>(g, num_cu, st)
                   : p.bm == 128 ? mx4::launch<128, 128, 2>(g, num_cu, st)
                                 : mx4::launch<64, 64, 2>(g, num_cu, st);
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t threads = m * n / 8;
    mx4::mx4_join_kernel<<<dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st>>>(
        static_cast<const float*>(workspace), p.splits, m, (int)n, ex, y);
    return hipGetLastError();
}

}  // namespace ck
