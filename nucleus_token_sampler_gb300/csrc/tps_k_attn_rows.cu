// The 16-row attention kernels for each head size and cache format, and their launches.
#include "tps_attn_rows.cuh"

namespace tps {

namespace {

template <int D, int kFormat>
cudaError_t prefix_rows(const AttnArgs& a, cudaStream_t stream)
{
    static_assert(sizeof(RowsShared<D>) <= 48 * 1024, "fits the default limit");
    attn_prefix_rows_kernel<D, kFormat><<<(unsigned)a.p.ctas, kRowsThreads, sizeof(RowsShared<D>), stream>>>(a);
    return cudaGetLastError();
}

template <int D, int kFormat>
cudaError_t suffix(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    auto k = attn_suffix_kernel<D, kFormat>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.a.B * a.c.n_heads * a.p.suffix_tiles * a.p.cluster), 1, 1);
    cfg.blockDim = dim3(kRowsThreads, 1, 1);
    cfg.dynamicSmemBytes = sizeof(RowsShared<D>);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (a.p.cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)a.p.cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (after_prefix) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <int D>
cudaError_t by_format(const AttnArgs& a, bool own, bool after_prefix, cudaStream_t stream)
{
    switch (a.c.format) {
    case TPS_KV_BF16: return own ? suffix<D, TPS_KV_BF16>(a, after_prefix, stream) : prefix_rows<D, TPS_KV_BF16>(a, stream);
    case TPS_KV_FP8: return own ? suffix<D, TPS_KV_FP8>(a, after_prefix, stream) : prefix_rows<D, TPS_KV_FP8>(a, stream);
    default: return own ? suffix<D, TPS_KV_INT8>(a, after_prefix, stream) : prefix_rows<D, TPS_KV_INT8>(a, stream);
    }
}

}  // namespace

cudaError_t launch_attn_prefix_rows(const AttnArgs& a, cudaStream_t stream)
{
    return a.c.head_dim == 64 ? by_format<64>(a, false, false, stream) : by_format<128>(a, false, false, stream);
}

cudaError_t launch_attn_suffix(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    return a.c.head_dim == 64 ? by_format<64>(a, true, after_prefix, stream) : by_format<128>(a, true, after_prefix, stream);
}

}  // namespace tps
