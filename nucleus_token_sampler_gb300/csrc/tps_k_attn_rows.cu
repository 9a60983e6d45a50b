// The 8- and 16-row attention kernels for each head size and cache format, of calls with a shared prefix.
#include "tps_attn_rows_launch.cuh"

namespace tps {

namespace {

template <int D>
cudaError_t by_format(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    switch (a.c.format) {
    case TPS_KV_BF16: return own<D, TPS_KV_BF16, false>(a, after_prefix, stream);
    case TPS_KV_FP8: return own<D, TPS_KV_FP8, false>(a, after_prefix, stream);
    default: return own<D, TPS_KV_INT8, false>(a, after_prefix, stream);
    }
}

}  // namespace

cudaError_t launch_attn_own(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    return a.c.head_dim == 64 ? by_format<64>(a, after_prefix, stream) : by_format<128>(a, after_prefix, stream);
}

}  // namespace tps
