// The 8- and 16-row attention kernels for trees of few rows.
#include "tps_attn_rows_launch.cuh"

namespace tps {

namespace {

template <int D> cudaError_t tree_rows(const AttnArgs& a, cudaStream_t stream)
{
    return a.c.format == TPS_KV_BF16  ? own<D, TPS_KV_BF16, true>(a, false, stream)
           : a.c.format == TPS_KV_FP8 ? own<D, TPS_KV_FP8, true>(a, false, stream)
                                       : own<D, TPS_KV_INT8, true>(a, false, stream);
}

}  // namespace

cudaError_t launch_attn_tree_rows(const AttnArgs& a, cudaStream_t stream)
{
    return a.c.head_dim == 64 ? tree_rows<64>(a, stream) : tree_rows<128>(a, stream);
}

}  // namespace tps
