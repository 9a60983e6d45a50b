// The tcgen05 prefix kernel on a fp8 cache.
#include "tps_attn_prefix_launch.cuh"

namespace tps {

cudaError_t launch_attn_prefix_fp8(const AttnArgs& a, cudaStream_t stream)
{
    return launch_prefix_format<TPS_KV_FP8>(a, stream);
}

}  // namespace tps
