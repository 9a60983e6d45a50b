// The tcgen05 tree kernel on an fp8 cache.
#include "tps_attn_prefix_launch.cuh"

namespace tps {

cudaError_t launch_attn_tree_fp8(const TreeArgs& a, cudaStream_t stream)
{
    return launch_tree_format<TPS_KV_FP8>(a, stream);
}

}  // namespace tps
