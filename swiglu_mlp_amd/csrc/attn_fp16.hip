// The kernels of ck_cross_attn for FP16 heads.
#include "attn_kernels.hpp"

template hipError_t ck::attn::launch<ck::f16>(Params&, const Plan&, uint32_t, hipStream_t);
