// attn.hpp -- what the host side of ck_cross_attn (attn.hip) shares with its
// kernels (attn_kernels.hpp, compiled for one type in attn_bf16.hip and one in
// attn_fp16.hip).
#pragma once
#include "ck_internal.hpp"
#include "heads.hpp"

namespace ck {
namespace attn {

constexpr int kTileWaves = 4;   // 32-row waves of a tile workgroup (of each of its key groups)
constexpr int kList = 4096;   // keys whose mask is listed at a time

struct Params {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* o;
    int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh, v_sb, v_st, v_sh, o_sb, o_st, o_sh;
    const int32_t* kv_len;
    const uint8_t* mask;
    int64_t mask_sb;
    uint32_t tk, d, share, kv_batch, heads_kv, rows, m_tiles;
    uint32_t splits, split_keys;    // keys [split_keys s, split_keys (s + 1)) belong to split s
    uint32_t list_keys;             // keys listed at a time: at most kList, their offsets in 32 bits
    float c;                        // scale * log2(e)
    float* part_o;                  // [key head, row][split][d]
    float* part_ml;                 // [key head, row][split] (m, l)
    FastDiv by_g, by_tq, by_hkv, by_tiles, by_splits;
};

// How a call runs: by slices (few rows; their keys streamed past the caches or
// not) or tiles, with one or two key groups a workgroup, and over how many splits.
struct Plan {
    bool slices, streamed, two_groups;
    uint32_t m_tiles, splits, split_keys;
};

// Enqueues the kernels of a call over bh key heads.
template <typename T>
hipError_t launch(Params& p, const Plan& plan, uint32_t bh, hipStream_t st);

}  // namespace attn
}  // namespace ck
