// The tcgen05 tree kernel on an int8 cache.
#include "tps_attn_prefix_launch.cuh"

namespace tps {

cudaError_t launch_attn_tree_int8(const TreeArgs& a, cudaStream_t stream)
{
    return launch_prefix_format<TPS_KV_INT8, true>(a, stream);
}

}  // namespace tps
