// The tcgen05 prefix kernel on a bf16 cache.
#include "tps_attn_prefix_launch.cuh"

namespace tps {

cudaError_t launch_attn_prefix_bf16(const AttnArgs& a, cudaStream_t stream)
{
    return launch_prefix_format<TPS_KV_BF16>(a, stream);
}

}  // namespace tps
