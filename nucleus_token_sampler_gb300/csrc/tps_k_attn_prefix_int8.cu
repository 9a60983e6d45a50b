// The tcgen05 prefix kernel on a int8 cache.
#include "tps_attn_prefix_launch.cuh"

namespace tps {

cudaError_t launch_attn_prefix_int8(const AttnArgs& a, cudaStream_t stream)
{
    return launch_prefix_format<TPS_KV_INT8>(a, stream);
}

}  // namespace tps
