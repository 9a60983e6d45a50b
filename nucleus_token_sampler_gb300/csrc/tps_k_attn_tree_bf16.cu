// The tcgen05 tree kernel on a bf16 cache.
#include "tps_attn_prefix_launch.cuh"

namespace tps {

cudaError_t launch_attn_tree_bf16(const TreeArgs& a, cudaStream_t stream)
{
    return launch_tree_format<TPS_KV_BF16>(a, stream);
}

}  // namespace tps
