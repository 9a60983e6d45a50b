// The 16-row attention kernels for each head size and cache format, and their launches.
#include "tps_attn_rows.cuh"

#include <atomic>

namespace tps {

namespace {

// More than 48 KB of dynamic shared memory has to be asked for, once per kernel and device.
template <typename Kernel>
cudaError_t allow_smem(Kernel k, size_t bytes, std::atomic<uint64_t>& allowed)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (allowed.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_release);
    return e;
}

template <int D, int kFormat>
cudaError_t prefix_rows(const AttnArgs& a, cudaStream_t stream)
{
    static std::atomic<uint64_t> allowed{0};
    auto k = attn_prefix_rows_kernel<D, kFormat>;
    const cudaError_t e = allow_smem(k, sizeof(RowsShared<D, kFormat>), allowed);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)a.p.ctas, kRowsThreads, sizeof(RowsShared<D, kFormat>), stream>>>(a);
    return cudaGetLastError();
}

template <int D, int kFormat, bool kOneWarp>
cudaError_t suffix_shape(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    static std::atomic<uint64_t> allowed{0};
    auto k = attn_suffix_kernel<D, kFormat, kOneWarp>;
    const cudaError_t e = allow_smem(k, sizeof(RowsShared<D, kFormat>), allowed);
    if (e != cudaSuccess) return e;
    const int64_t items = a.a.B * a.c.n_heads * a.p.suffix_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kOneWarp ? (items + kRowsWarps - 1) / kRowsWarps : items * a.p.cluster), 1, 1);
    cfg.blockDim = dim3(kRowsThreads, 1, 1);
    cfg.dynamicSmemBytes = sizeof(RowsShared<D, kFormat>);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (a.p.cluster > 1) {  // 1 wherever kOneWarp
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

template <int D, int kFormat>
cudaError_t suffix(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    return a.p.one_warp ? suffix_shape<D, kFormat, true>(a, after_prefix, stream)
                        : suffix_shape<D, kFormat, false>(a, after_prefix, stream);
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
