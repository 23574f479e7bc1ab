// attn.hip -- host side of ck_cross_attn: which kernel takes a call, over how
// many splits of the keys, and its workspace.
#include "attn.hpp"

#include <algorithm>

namespace ck {

namespace {

attn::Plan plan_of(int64_t bh, int64_t rows, int64_t tk, int64_t d)
{
    attn::Plan p{};
    const int64_t cus = num_cus();
    // Slices up to 96 rows, where part of a 128-row tile would idle (96 rows, 16
    // heads of 128, 2048 keys: 13.9 us, tiles 17.5; 64 rows, 64 heads of 128, 1024
    // keys: 15.2 and 17.4; 64 rows, 64 heads of 64, 4096 keys: 19.2 and 19.0), and
    // up to 512 where 32-row workgroups fill less than half of the chip (256 rows,
    // 8 heads of 128, 1024 keys: 11.3 and 16.6; but 128 rows, 64 heads of 64, 4096
    // keys: 26.8 and 22.2).
    p.slices = rows <= 96 || (rows <= 512 && bh * ((rows + 31) / 32) < cus / 2);
    const int64_t tile_rows = p.slices ? 32 : 32 * attn::kTileWaves;
    p.m_tiles = (uint32_t)((rows + tile_rows - 1) / tile_rows);
    // As many splits as keep every workgroup resident at once, one a CU (two
    // slice workgroups of up to 64 channels share one): a second round of
    // workgroups costs more than it balances, also where lengths differ (one token,
    // 8 sequences of 2048 keys, 8 heads of 128: 4 splits 16.6 us, 8 splits 20).
    // The join costs about as much as 512 keys of a slice workgroup (128 rows, 16
    // heads of 128, 512 keys: one split 8.6 us, two 10.4; one token, 8 heads, 512
    // keys: 7.4 and, with four, 7.2, but a second launch).
    const int64_t groups = bh * p.m_tiles;
    const int64_t resident = cus * (p.slices && d <= 64 ? 2 : 1), least = p.slices ? 128 : 512;
    int64_t splits = std::max<int64_t>(1, std::min(resident / groups, tk / least));
    if (p.slices && tk < 768) splits = 1;
    // Whole 128-key pieces a split, so fewer splits where that rounds up: 1500 keys
    // over 32 key heads are 6 splits of 256, 1536 are 12 of 128, and both take 7.9 us.
    const int64_t unit = 128;
    const int64_t keys = (tk + splits - 1) / splits;
    p.split_keys = (uint32_t)std::max<int64_t>(unit, (keys + unit - 1) / unit * unit);
    p.splits = (uint32_t)std::max<int64_t>(1, (tk + p.split_keys - 1) / p.split_keys);
    // two groups of waves halve a workgroup's way through its keys, for about a
    // microsecond to join them (1000 rows, 8 heads of 128, 8192 keys: 46.0 us, one
    // group 49.4; 1024 rows, 32 heads of 96, 128 keys: 8.4 and 7.1)
    p.two_groups = !p.slices && groups * p.splits <= cus && p.split_keys >= 512;
    return p;
}

}  // namespace

size_t cross_attn_workspace(int64_t batch, int64_t kv_batch, int64_t tq, int64_t tk, int64_t heads, int64_t kv_heads,
                            int64_t d)
{
    const int64_t bh = kv_batch * kv_heads, rows = batch / kv_batch * tq * (heads / kv_heads);
    const attn::Plan p = plan_of(bh, rows, tk, d);
    return p.splits == 1 ? 0 : (size_t)(bh * rows * p.splits) * (size_t)(d + 2) * sizeof(float);
}

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
    p.kv_batch = (uint32_t)a.kv_batch;
    const int64_t g = a.heads / a.kv_heads;
    p.rows = (uint32_t)(p.share * a.tq * g);
    p.c = a.scale * 1.44269504088896340736f;
    p.by_g = FastDiv((uint32_t)g);
    p.by_tq = FastDiv((uint32_t)a.tq);
    p.by_hkv = FastDiv((uint32_t)a.kv_heads);
    const int64_t bh = a.kv_batch * a.kv_heads;
    attn::Plan plan = plan_of(bh, p.rows, a.tk, a.d);
    // with lengths, whose values only the device knows, half of the keys
    plan.streamed = plan.m_tiles == 1 && bh * a.tk * a.d * 4 / (a.kv_len ? 2 : 1) >= kInfinityCacheBytes;
    p.m_tiles = plan.m_tiles;
    p.splits = plan.splits;
    p.split_keys = plan.split_keys;
    p.by_tiles = FastDiv(p.m_tiles);
    p.by_splits = FastDiv(p.splits);
    // a listed key's offset from the list's first stays below 2^31 bytes
    const int64_t pitch = std::max<int64_t>(1, std::max(a.k_st, a.v_st)) * 2;
    p.list_keys = (uint32_t)std::min<int64_t>(attn::kList, 0x7f000000LL / pitch);
    p.part_o = static_cast<float*>(a.ws);
    p.part_ml = p.part_o + (uint64_t)bh * p.rows * p.splits * p.d;
    return a.fp16 ? attn::launch<f16>(p, plan, (uint32_t)bh, st) : attn::launch<bf16>(p, plan, (uint32_t)bh, st);
}

}  // namespace ck
