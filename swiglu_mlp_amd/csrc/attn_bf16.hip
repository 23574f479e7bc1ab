// The kernels of ck_cross_attn for BF16 heads.
#include "attn_kernels.hpp"

template hipError_t ck::attn::launch<ck::bf16>(Params&, const Plan&, uint32_t, hipStream_t);
