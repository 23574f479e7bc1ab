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
// The matrix cores set the pace of large products: random codes reach 6.2 to 6.6,
// by card, of the nominal 10 PFLOP/s in a loop of nothing but these instructions
// (the clock falls under their power).  A wave issues a product every 32 cycles and
// some 4 other instructions in its shadow; past that each one more costs 7 or 8 cycles
// (in a loop, at the nominal clock: 37 cycles a product alone or with 2 scalar ones,
// 42 with 4, 57 with 6, 73 with 8).  So the kernel is built for few instructions a
// product:
//  * A group of 4 waves (2 x 2) owns a BM x BN tile; a wave's part is FM x FN
//    fragments of 32 x 32, accumulated in AGPRs.  It reads FM + FN blocks from
//    LDS for FM FN products.
//  * K advances two slices (128 values) a stage.  Stages go through a ring of LDS
//    slots by DMA (buffer_load ... lds, two for one LDS address), 3 ahead.  A stage is
//    two halves around one barrier: each multiplies one slice while it
//    reads the next one's fragments, so products never wait for LDS.  Reads and
//    loads are placed between the products in source order.
//  * Two stages make a pair: 256 values, one chunk of scales (256 bytes for 32
//    rows; one DMA instruction a wave, one register a fragment).  Slots, scale
//    selects and the ends of tiles are constants of a stage's place in its pair.
//  * Tiles of 256 columns, one group a CU: workgroups stay and take tiles in turn; the
//    stages run on from a tile to the next, whose loads so overlap the epilogue.
//    The workgroups of an XCD take consecutive tiles and share operands in its L2.
//  * Smaller tiles, two groups a workgroup, each with half of k: their waves fill
//    each other's gaps, and their sums meet in LDS.
// Small products take mx4_few.hip instead.
// Measured, cards differing by 4%: 4096 x 4096 -> 24576 197 to 201 us (4.1 PFLOP/s),
// 16384 x 12288 -> 4096 331 to 355 us (5.0 to 4.65), with a residual of 134 MB 370 to
// 382.  The matrix cores are busy 55 and 62% of the cycles at 1.8 and 1.65 GHz.  Codes
// of zero, whose products cost little power, take 163 and 265 us: a fifth of the time
// is the power's, the rest beyond the products is the schedule's.
#include "ck_internal.hpp"
#include "mx4.hpp"
#include "mx4_stage.hpp"

#include <algorithm>
#include <type_traits>
#include <utility>

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

// 16 bytes a lane from memory to LDS, not tracked by the compiler (which would
// wait for all of them before any LDS read): the waits are counted by hand.  Lane
// l's bytes land at lds + OFF + 16 l.  TWO: and those 1 KB on at 1 KB on (the
// instruction's offset counts in memory and in LDS).
template <int OFF, bool TWO>
__device__ __forceinline__ void lds_dma(v4i rsrc, uint32_t voff, uint32_t soff, uint32_t lds)
{
    if constexpr (TWO)
        asm volatile(
            "s_add_u32 m0, %3, %4\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %0, %1, %2 offen lds\n\t"
            "buffer_load_dwordx4 %0, %1, %2 offen offset:1024 lds"
            :
            : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds), "n"(OFF)
            : "memory", "m0", "scc");
    else
        asm volatile(
            "s_add_u32 m0, %3, %4\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %0, %1, %2 offen lds"
            :
            : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds), "n"(OFF)
            : "memory", "m0", "scc");
}
__device__ __forceinline__ void lds_dma(const uint8_t* at, uint32_t lds)
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

// f(0), f(1), ... f(N - 1) with constants as arguments.
template <typename F, int... I>
__device__ __forceinline__ void for_each_in(F&& f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void for_each(F&& f)
{
    for_each_in(f, std::make_integer_sequence<int, N>{});
}

template <int BM_, int BN_, int GROUPS_>
struct Cfg {
    static constexpr int BM = BM_, BN = BN_, GROUPS = GROUPS_;
    // Pairs of stages in the ring, and stages ahead (3 and 4 pairs, where they fit, were
    // no faster).
    static constexpr int R = 2, P = 2 * R - 1;
    static constexpr int FM = BM / 64, FN = BN / 64;    // a wave's fragments
    static constexpr int A_BLK = BN / 16, B_BLK = BM / 16;              // 1 KB blocks of a stage
    static constexpr int AW = A_BLK / 4, XW = B_BLK / 4, L = AW + XW;   // a wave's share
    static constexpr int AP = (AW + 1) / 2, XP = (XW + 1) / 2;          // as loads of one row block: both slices, or one
    static constexpr int CODES = (A_BLK + B_BLK) * 1024;
    static constexpr int CHUNKS = (BM + BN) / 32;       // of scales (32 rows, 256 k)
    static constexpr int CPW = (CHUNKS + 3) / 4;        // chunks a wave loads, into its own KB
    static constexpr int RING = R * (2 * CODES + 4096); // slots of codes, then of scales
    static constexpr int LDS = GROUPS * RING;
    // the groups' sums: group o keeps fragments j of its share (all of them in group
    // 0 where there are fewer than groups), the others give theirs in LDS
    static constexpr int OWNERS = FM >= GROUPS ? GROUPS : 1, SHARE = FM / OWNERS;
    static constexpr int SUMS = 4 * OWNERS * (GROUPS - 1) * FN * SHARE * 4096;
    static_assert(FM % OWNERS == 0, "shares");
    static_assert(LDS <= 160 * 1024, "LDS");
    static_assert(A_BLK % 4 == 0 && B_BLK % 4 == 0, "blocks split evenly over 4 waves");
};

struct Args {
    const uint8_t *xc, *xs, *wc, *ws;
    uint16_t* y;
    EpiExtra ex;
    int M, N;
    int kb;             // 1 KB blocks (slices) of a 32-row block: kp / 64
    int xb, wb;         // 32-row blocks of x and w
    int tiles_m, tiles_n, group_m;
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

// EXTRA: bias and / or residual.
template <int BM, int BN, int GROUPS, bool EXTRA>
__global__ __launch_bounds__(256 * GROUPS) void mx4_gemm_kernel(Args g)
{
    // The body uses AMDGPU-only types; the host pass only needs the launch stub.
#if defined(__HIP_DEVICE_COMPILE__)
    using C = Cfg<BM, BN, GROUPS>;
    constexpr int R = C::R;
    // the rings; then the tile's bias, or (GROUPS > 1) the groups' sums and the bias in place of the rings
    constexpr int SUMS = GROUPS > 1 ? C::SUMS : C::LDS;
    static_assert(GROUPS == 1 || SUMS + BN * 4 <= C::LDS, "LDS of the sums");
    __shared__ __attribute__((aligned(1024))) char smem[C::LDS + (GROUPS == 1 && EXTRA ? BN * 4 : 0)];
    constexpr int NMF = C::FN * C::FM;                  // products of a slice
    constexpr int NDS = C::FN + C::FM;                  // fragment reads of a slice
    constexpr int NPAIR = C::AP + C::XP;                // loads (of one or two KB) of a stage
    constexpr int H0 = NPAIR / 2;                       // of them, in the first half
    constexpr int L0 = (H0 < C::AP ? H0 : C::AP) * (C::AW > 1 ? 2 : 1) +
                       (H0 > C::AP ? H0 - C::AP : 0) * (C::XW > 1 ? 2 : 1);   // as instructions
    constexpr int NST = 2 * NMF;                        // stores of an epilogue
    // Loads issued after the last of stage s + 1 at the middle of stage s: those of
    // s + 2 .. s + P - 1, the first half's of s + P, and the scales with every second one of these.
    constexpr int OUTS = (C::P - 2) * C::L + L0 + R - 1;
    static_assert(OUTS + NST < 64, "vmcnt range");

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
    const int group = GROUPS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) : 0;
    const int G = gridDim.x, b = blockIdx.x;
    const int tiles = g.tiles_m * g.tiles_n;
    const int my_tiles = (tiles - b + G - 1) / G;       // one with several groups
    const int all_pairs = g.kb / 4;

    // Within a full round the workgroups of one XCD (b % 8) take consecutive tiles.
    const bool xcd_order = (G & 7) == 0;
    const int b_xcd = (b & 7) * (G >> 3) + (b >> 3);
    auto tile_of = [&](int q) {
        const bool full = xcd_order & ((q + 1) * G <= tiles);
        return q * G + (full ? b_xcd : b);
    };
    // this group's range of pairs (of two or more groups at least two pairs each)
    const int pair0 = group * all_pairs / GROUPS;
    const int pairs = (group + 1) * all_pairs / GROUPS - pair0;
    const int most_pairs = (all_pairs + GROUPS - 1) / GROUPS;
    const uint32_t ring = (uint32_t)(uintptr_t)(lds_void_t*)smem + (uint32_t)(group * C::RING);
    const uint32_t lane16 = (uint32_t)lane * 16u;

    // ---- the load cursor: the stage to be loaded next.  After the last tile it
    // starts over on it: those loads go to slots that nobody reads again, and the
    // number of loads of a stage stays constant. ----
    int lq = 0, lpairs = pairs;
    v4i rs_w, rs_x;                                     // the tile's rows of codes
    uint32_t so_w[C::AP], so_x[C::XP];                  // where in them this wave's loads of the stage are
    const uint8_t* sp;                                  // this lane's scales of the pair
    auto set_tile = [&](int q) {
        int tm, tn;
        tile_coords(tile_of(q), g.tiles_m, g.tiles_n, g.group_m, tm, tn);
        // quotients are computed in lanes; what follows from them here are scalar operands
        tm = __builtin_amdgcn_readfirstlane(tm), tn = __builtin_amdgcn_readfirstlane(tn);
        const int64_t wb0 = (int64_t)tn * (BN / 32), xb0 = (int64_t)tm * (BM / 32);
        const int64_t w0 = wb0 * g.kb * 1024, x0 = xb0 * g.kb * 1024;
        rs_w = make_rsrc(g.wc + w0, (int64_t)g.wb * g.kb * 1024 - w0);
        rs_x = make_rsrc(g.xc + x0, (int64_t)g.xb * g.kb * 1024 - x0);
#pragma unroll
        for (int p = 0; p < C::AP; ++p)
            so_w[p] = stage_offset(wave * C::AW + 2 * p, g.kb, pair0 * 4, g.wb - (int)wb0);
#pragma unroll
        for (int p = 0; p < C::XP; ++p)
            so_x[p] = stage_offset(wave * C::XW + 2 * p, g.kb, pair0 * 4, g.xb - (int)xb0);
        // past the operand's end the last block's scales, as with its codes
        const int c = min(wave * C::CPW + min(lane >> 4, C::CPW - 1), C::CHUNKS - 1);
        const bool w = c < BN / 32;
        const int64_t rb = w ? min((int64_t)g.wb - 1, wb0 + c) : min((int64_t)g.xb - 1, xb0 + c - BN / 32);
        sp = (w ? g.ws : g.xs) + (rb * (g.kb / 4) + pair0) * 256 + (lane & 15) * 16;
    };
    // Load p of a stage into the slot whose share of this wave begins at LDS address `at`.
    auto issue = [&](auto p_, uint32_t at) {
        constexpr int p = decltype(p_)::value;
        if constexpr (p < C::AP)
            lds_dma<p * 2048, (C::AW > 1)>(rs_w, lane16, so_w[p], at + (uint32_t)(wave * C::AW * 1024));
        else
            lds_dma<C::A_BLK * 1024 + (p - C::AP) * 2048, (C::XW > 1)>(rs_x, lane16, so_x[p - C::AP],
                                                                     at + (uint32_t)(wave * C::XW * 1024));
    };
    auto issue_scales = [&](uint32_t slot) {
        lds_dma(sp, ring + 2 * R * C::CODES + slot * 4096 + (uint32_t)wave * 1024);
        sp += 256;
    };
    auto next_stage = [&]() {
#pragma unroll
        for (int p = 0; p < C::AP; ++p) so_w[p] += 2048;
#pragma unroll
        for (int p = 0; p < C::XP; ++p) so_x[p] += 2048;
    };
    auto next_pair = [&]() {   // after an odd stage
        if (--lpairs == 0) {
            asm volatile("" ::: "memory");   // a branch, not its ~100 scalar operations in every pair
            lpairs = pairs;
            lq = min(lq + 1, my_tiles - 1);
            set_tile(lq);
        }
    };

    v16f acc[C::FN][C::FM];
    const int lr = lane & 31, lh = lane >> 5;
    const int wm0 = (wave & 1) * (BM / 2), wn0 = (wave >> 1) * (BN / 2);
    // this lane's places in the pair's first slot
    const char* pa = smem + group * C::RING + (wn0 / 32) * 2048 + lane * 16;
    const char* pb = smem + group * C::RING + C::A_BLK * 1024 + (wm0 / 32) * 2048 + lane * 16;
    const char* const ps = smem + group * C::RING + 2 * R * C::CODES + lane * 4;
    int cur = 0;                                        // the pair's place in the ring
    auto frag_a = [&](int off, int i) { return *reinterpret_cast<const v4i*>(pa + off + i * 2048); };
    auto frag_b = [&](int off, int j) { return *reinterpret_cast<const v4i*>(pb + off + j * 2048); };
    auto scale = [&](uint32_t slot, int c) {
        return *reinterpret_cast<const int*>(ps + slot * 4096 + (c / C::CPW) * 1024 + (c % C::CPW) * 256);
    };

    set_tile(0);
#pragma unroll
    for (int p = 0; p < C::P; ++p) {
        if (p % 2 == 0) issue_scales(p / 2);
        for_each<NPAIR>([&](auto i) { issue(i, ring + (uint32_t)(p * C::CODES)); });
        next_stage();
        if (p % 2 == 1) next_pair();
    }
    wait_vmcnt<(C::P - 1) * C::L + R - 1>();
    workgroup_barrier();
    v4i fa[C::FN], fb[C::FM], ga[C::FN], gb[C::FM];
    int sa[C::FN], sb[C::FM], na[C::FN], nb[C::FM];     // the pair's scales, and the next one's
#pragma unroll
    for (int i = 0; i < C::FN; ++i) fa[i] = frag_a(0, i), sa[i] = scale(0, (wn0 >> 5) + i);
#pragma unroll
    for (int j = 0; j < C::FM; ++j) fb[j] = frag_b(0, j), sb[j] = scale(0, BN / 32 + (wm0 >> 5) + j);

    // Product k of a slice, slice Q of the pair.
    auto mfma_step = [&](int k, auto q, const v4i (&w)[C::FN], const v4i (&x)[C::FM], bool zero) {
        // back and forth over j, so that consecutive products share an operand (the
        // operands' switching is power, and power is speed: 0.5% on large products)
        const int i = k / C::FM, j = i % 2 ? C::FM - 1 - k % C::FM : k % C::FM;
        const v16f c = zero ? v16f{} : acc[i][j];
        acc[i][j] = product<decltype(q)::value>(w[i], x[j], c, sa[i], sb[j]);
        // here and nowhere else: the compiler takes this instruction for one that it
        // may sink, and would gather all products behind the stage's last branch
        asm volatile("" : "+a"(acc[i][j]));
    };
    auto read_step = [&](int r, int off, v4i (&w)[C::FN], v4i (&x)[C::FM]) {
        if (r < C::FN) w[r] = frag_a(off, r);
        else if (r < NDS) x[r - C::FN] = frag_b(off, r - C::FN);
    };
    auto read_scale = [&](int r, uint32_t slot) {
        if (r < C::FN) na[r] = scale(slot, (wn0 >> 5) + r);
        else if (r < NDS) nb[r - C::FN] = scale(slot, BN / 32 + (wm0 >> 5) + r - C::FN);
    };
    constexpr int STEPS = NMF > NDS ? NMF : NDS;
    // loads [P0, P1) of the stage ahead, spread over the steps of a half (a burst of
    // them fills the address unit's queue and holds up the products behind it)
    auto spread = [&](int k, auto p0, auto p1, uint32_t at) {
        constexpr int P0 = decltype(p0)::value, P1 = decltype(p1)::value;
        if constexpr (P1 > P0) {
            constexpr int EVERY = STEPS / (P1 - P0);
            for_each<P1 - P0>([&](auto i) {
                if (k == i * EVERY + EVERY / 2) issue(std::integral_constant<int, P0 + decltype(i)::value>{}, at);
            });
        }
    };
    // One stage, of parity PAR in its pair.  It loads the stage P ahead into the slot
    // of the one before it: the pair's own first slot when odd, the second one of the
    // pair before when even.  `stores`: an epilogue's may still be counted.  LEFT: the
    // stages after it, 3 for more than that; the last three load nothing.
    auto stage = [&](auto first, auto par, auto left, bool stores) {
        constexpr int PAR = decltype(par)::value, LEFT = decltype(left)::value;
        const int next = cur + 1 == R ? 0 : cur + 1, before = cur == 0 ? R - 1 : cur - 1;
        const uint32_t at = ring + (uint32_t)((PAR ? cur : before) * (2 * C::CODES) + (PAR ? 0 : C::CODES));
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (PAR == 1 && LEFT == 3) issue_scales((uint32_t)cur);
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            if (k < NMF) mfma_step(k, std::integral_constant<int, 2 * PAR>{}, fa, fb, decltype(first)::value);
            read_step(k, PAR * C::CODES + 1024, ga, gb);
            if constexpr (LEFT == 3) spread(k, std::integral_constant<int, 0>{}, std::integral_constant<int, H0>{}, at);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (LEFT > 0) {
            wait_lgkmcnt0();          // this wave's fragments of the second half are in registers
            if constexpr (LEFT == 1) wait_vmcnt<0>();
            else if constexpr (LEFT == 2) wait_vmcnt<C::L>();   // of the last stage
            else if (stores) wait_vmcnt<OUTS + NST>();
            else wait_vmcnt<OUTS>();
            workgroup_barrier();      // every wave's; the next stage is in LDS, and this one's slot is read no more
        }
        if constexpr (PAR == 1 && LEFT > 0) pa += (next - cur) * (2 * C::CODES), pb += (next - cur) * (2 * C::CODES);
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            if (k < NMF) mfma_step(k, std::integral_constant<int, 2 * PAR + 1>{}, ga, gb, false);
            if constexpr (LEFT > 0) read_step(k, PAR ? 0 : C::CODES, fa, fb);
            if constexpr (PAR == 1 && LEFT > 0) read_scale(k, (uint32_t)next);
            if constexpr (LEFT == 3) spread(k, std::integral_constant<int, H0>{}, std::integral_constant<int, NPAIR>{}, at);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (LEFT == 3) {
            next_stage();
            if constexpr (PAR == 0) next_pair();
        }
        if constexpr (PAR == 1 && LEFT > 0) {
            cur = next;
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
    // given an offset outside it: both stores are dropped.  Fragments j0 <= j < j1.
    auto stage_bias = [&](int tn) {
        const int t = (int)threadIdx.x;
        if (t < BN) reinterpret_cast<float*>(smem + SUMS)[t] = g.ex.bias[min(tn * BN + t, g.N - 1)];
    };
    auto epilogue = [&](int tile, int j0, int j1) {
        int tm, tn;
        tile_coords(tile, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
        const int64_t row0 = (int64_t)tm * BM;
        const int rows = (int)min((int64_t)BM, g.M - row0);
        const __amdgpu_buffer_rsrc_t rs_o =
            __builtin_amdgcn_make_buffer_rsrc(g.y + row0 * g.N, (short)0, rows * g.N * 2, 0x00020000);
        const int n_base = tn * BN + wn0 + 8 * lh;
        // The residual's row j is loaded while row j - 1 is stored; the bias, which
        // every row needs, waits in LDS.  (Where groups share a tile's rows j0 is no
        // constant, and in tiles of 128 x 128 these rows lie in scratch, 144 bytes a lane.)
        constexpr int PER_ROW = EXTRA ? C::FN * 2 : 1;
        uint4 res[2][PER_ROW];
        auto load_residual = [&](int j) {
            const int64_t row = (row0 + min(wm0 + 32 * j + lr, rows - 1)) * g.N;
#pragma unroll
            for (int t = 0; t < PER_ROW; ++t)
                res[j & 1][t] = *reinterpret_cast<const uint4*>(g.ex.res + row + min(n_base + 16 * t, g.N - 8));
        };
        if constexpr (EXTRA) {
            if (g.ex.res) load_residual(j0);
            if (GROUPS == 1 && g.ex.bias) {   // the last tile's readers have passed the stages' barriers
                stage_bias(tn);
                wait_lgkmcnt0();
                workgroup_barrier();
            }
        }
#pragma unroll
        for (int j = 0; j < C::FM; ++j) {
            if (j < j0 || j >= j1) continue;
            const int r = wm0 + 32 * j + lr;
            const uint32_t row = (uint32_t)r * (uint32_t)g.N;
            if constexpr (EXTRA) {
                if (g.ex.res && j + 1 < j1) load_residual(j + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
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
                    if constexpr (!EXTRA) {
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
                        if (g.ex.bias) {
                            const float* lb = reinterpret_cast<const float*>(smem + SUMS) + wn0 + 8 * lh + 32 * i + 16 * h;
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = v[e] + lb[e];
                        }
                        if (g.ex.res) {
                            float x[8];
                            unpack8<bf16>(res[j & 1][2 * i + h], x);
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = v[e] + x[e];
                        }
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, pack8<bf16>(v)), rs_o,
                                                               ok ? (row + (uint32_t)n) * 2u : kBufferOutside, 0, 0);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    constexpr std::integral_constant<int, 0> even{}, last{};
    constexpr std::integral_constant<int, 1> odd{}, one_left{};
    constexpr std::integral_constant<int, 2> two_left{};
    constexpr std::integral_constant<int, 3> more{};
    constexpr std::true_type first{};
    constexpr std::false_type later{};
    if constexpr (GROUPS == 1) {
        for (int q = 0; q < my_tiles; ++q) {
            stage(first, even, more, q > 0);
            stage(later, odd, more, q > 0);
            for (int p = 1; p < pairs; ++p) {
                stage(later, even, more, false);
                stage(later, odd, more, false);
            }
            epilogue(tile_of(q), 0, C::FM);
        }
        wait_vmcnt<0>();   // no LDS load may land after the workgroup retires
    } else {
        stage(first, even, more, false);
        for (int p = 2; p < pairs; ++p) {
            stage(later, odd, more, false);
            stage(later, even, more, false);
        }
        stage(later, odd, two_left, false);
        stage(later, even, one_left, false);
        stage(later, odd, last, false);
        if (pairs < most_pairs) {   // as many barriers in every group
            workgroup_barrier();
            workgroup_barrier();
        }
        wait_vmcnt<0>();
        wait_lgkmcnt0();
        workgroup_barrier();        // the rings are read no more and nothing lands in them
        constexpr int OWNERS = C::OWNERS, SHARE = C::SHARE;
        // [owner][giver, but the owner][wave][i][j of the share][4 registers][lane]
        auto place = [&](int owner, int giver, int i, int j) {
            const int slot = giver < owner ? giver : giver - 1;
            return smem + ((((owner * (GROUPS - 1) + slot) * 4 + wave) * C::FN + i) * SHARE + j) * 4096 + lane * 16;
        };
#pragma unroll
        for (int j = 0; j < C::FM; ++j) {
            const int owner = j / SHARE;
            if (owner == group) continue;
#pragma unroll
            for (int i = 0; i < C::FN; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<v4f*>(place(owner, group, i, j % SHARE) + q * 1024) =
                        v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        }
        if (EXTRA && g.ex.bias) {
            int tm, tn;
            tile_coords(tile_of(0), g.tiles_m, g.tiles_n, g.group_m, tm, tn);
            stage_bias(tn);
        }
        __syncthreads();
        if (group >= OWNERS) return;
#pragma unroll
        for (int j = 0; j < C::FM; ++j) {
            if (j / SHARE != group) continue;
#pragma unroll
            for (int o = 0; o < GROUPS; ++o) {
                if (o == group) continue;
#pragma unroll
                for (int i = 0; i < C::FN; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const v4f t = *reinterpret_cast<const v4f*>(place(group, o, i, j % SHARE) + q * 1024);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += t[e];
                    }
            }
        }
        epilogue(tile_of(0), group * SHARE, (group + 1) * SHARE);
    }
#endif  // __HIP_DEVICE_COMPILE__
}

template <int BM, int BN, int GROUPS>
hipError_t launch(Args g, int num_cu, hipStream_t st)
{
    const bool extra = g.ex.bias || g.ex.res;
    g.tiles_m = (g.M + BM - 1) / BM;
    g.tiles_n = (g.N + BN - 1) / BN;
    g.group_m = std::min(g.tiles_m, 4);
    const int tiles = g.tiles_m * g.tiles_n;
    const dim3 grid(GROUPS > 1 ? tiles : std::min(tiles, num_cu)), block(256 * GROUPS);
    if (extra)
        mx4_gemm_kernel<BM, BN, GROUPS, true><<<grid, block, 0, st>>>(g);
    else
        mx4_gemm_kernel<BM, BN, GROUPS, false><<<grid, block, 0, st>>>(g);
    return hipGetLastError();
}

// Tiles, and what a call on them takes in us: start + rounds (unit + pair pairs), a
// round being a tile a CU and a pair 256 of k.  The last two are mx4_few.hip's.
// Measured: 4096 x 4096 -> 24576, 6 rounds of 256 x 256 tiles, 200 us (128 x 256:
// 226); 2048 x 4096 -> 4096 22 us on 128 x 256 (128 x 128: 28, 256 x 256 on half of
// the CUs: 28); 1024 x 4096 -> 4096 14 us on 128 x 128 (64 x 128: 19, 128 x 256: 17);
// 512 x 4096 -> 4096 10.0 us on 64 x 128 (128 x 128: 11.5, 64 x 64: 12.0); 256 x 4096
// -> 4096 6.8 us on 64 x 64 (32 x 32: 8.6, 64 x 128: 8.9), with k = 12288 13.3 (64 x
// 128: 17); 333 x 2112 -> 1040 4.4 us on 32 x 32 (64 x 64: 5.0, 64 x 128: 6.8).
struct Shape {
    int bm, bn, groups;
    float start, unit, pair;
};
constexpr Shape kShapes[] = {{256, 256, 1, 3.0f, 9.0f, 1.5f}, {128, 256, 1, 4.0f, 4.0f, 0.93f},
                             {128, 128, 2, 2.5f, 4.0f, 0.5f}, {64, 128, 2, 1.5f, 3.4f, 0.33f},
                             {64, 64, 1, 2.6f, 0.6f, 0.222f}, {32, 32, 1, 2.6f, 0.3f, 0.079f}};

const Shape& shape_of(int64_t m, int64_t n, int64_t k, int num_cu)
{
    const int64_t pairs = pad_cols(k) / 256;
    const Shape* best = nullptr;
    double least = 0;
    for (const Shape& c : kShapes) {
        if (c.groups > 1 && pairs < 2 * c.groups) continue;   // two pairs a group
        const int64_t tiles = ((m + c.bm - 1) / c.bm) * ((n + c.bn - 1) / c.bn), rounds = (tiles + num_cu - 1) / num_cu;
        // a workgroup a tile: kept to half of a launch's 2^32 threads
        if (c.bn < 256 && tiles > 1 << 22) continue;
        const double t = c.start + (double)rounds * (c.unit + c.pair * (double)pairs);
        if (!best || t < least) best = &c, least = t;
    }
    return *best;
}

}  // namespace mx4

hipError_t launch_mx4_gemm(const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* ws, int64_t m,
                           int64_t n, int64_t k, uint16_t* y, EpiExtra ex, hipStream_t st)
{
    if (m <= 16) return launch_mx4_few(xc, xs, wc, ws, m, n, k, 16, y, ex, st);
    const int num_cu = num_cus();
    const mx4::Shape& c = mx4::shape_of(m, n, k, num_cu);
    if (c.bn <= 64) return launch_mx4_few(xc, xs, wc, ws, m, n, k, c.bm, y, ex, st);
    mx4::Args g{};
    g.xc = xc, g.xs = xs, g.wc = wc, g.ws = ws, g.y = y, g.ex = ex;
    g.M = (int)m, g.N = (int)n, g.kb = (int)(mx4::pad_cols(k) / 64);
    g.xb = (int)(mx4::pad_rows(m) / 32), g.wb = (int)(mx4::pad_rows(n) / 32);
    if (c.bm == 256) return mx4::launch<256, 256, 1>(g, num_cu, st);
    if (c.bn == 256) return mx4::launch<128, 256, 1>(g, num_cu, st);
    return c.bm == 128 ? mx4::launch<128, 128, 2>(g, num_cu, st) : mx4::launch<64, 128, 2>(g, num_cu, st);
}

}  // namespace ck
