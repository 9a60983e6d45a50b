// The tcgen05 tree kernel on an int8 cache.
#include "tps_attn_prefix_launch.cuh"

namespace tps {

cudaError_t launch_attn_tree_int8(const TreeArgs& a, cudaStream_t stream)
{
    return launch_tree_format<TPS_KV_INT8>(a, stream);
}

}  // namespace tps
