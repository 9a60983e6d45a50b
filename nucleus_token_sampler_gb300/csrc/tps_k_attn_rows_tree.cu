// The 8- and 16-row attention kernels for trees of few rows over 8-bit caches.
#include "tps_attn_rows_launch.cuh"

namespace tps {

cudaError_t launch_attn_tree_rows(const AttnArgs& a, cudaStream_t stream)
{
    const bool fp8 = a.c.format == TPS_KV_FP8;
    if (a.c.head_dim == 64) return fp8 ? own<64, TPS_KV_FP8, true>(a, false, stream) : own<64, TPS_KV_INT8, true>(a, false, stream);
    return fp8 ? own<128, TPS_KV_FP8, true>(a, false, stream) : own<128, TPS_KV_INT8, true>(a, false, stream);
}

}  // namespace tps
